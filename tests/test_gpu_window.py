"""Attention with a sliding window and sinks (fa_fwd_window, fa_bwd_window, fa_fwd_paged_window) against fp64."""
import math

import pytest
import torch

import exact_attention_114_b200 as fa
from tests.masked_ref import Ref, close, window_seen

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def make(B, Hq, Hkv, Nq, Nk, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    return rnd(B, Hq, Nq, d), rnd(B, Hkv, Nk, d), rnd(B, Hkv, Nk, d), rnd(B, Hq, Nq, d)


def grouped(t, Hkv):
    """[B, Hq, N, ...] as [B, Hkv, G * N, ...]"""
    return t.reshape(t.shape[0], Hkv, -1, *t.shape[3:])


def ref_of(q, k, v, window, sinks, dout=None):
    Hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    seen = window_seen(q.shape[2], k.shape[2], window, sinks, q.device).repeat(G, 1)
    return Ref(grouped(q, Hkv), k, v, seen, dout=None if dout is None else grouped(dout, Hkv))


def check_fwd(q, k, v, window, sinks):
    o, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    r = ref_of(q, k, v, window, sinks)
    close(o, r.o, r.o_tol, "o")
    close(lse, r.lse, r.lse_tol, "lse")
    return o, lse


# B, Hq, Hkv, Nq, Nk, d, window, sinks
TILED = [
    (1, 2, 1, 300, 300, 128, 64, 4),          # window inside a tile
    (2, 4, 2, 333, 333, 64, 100, 1),
    (1, 2, 2, 700, 700, 128, 257, 130),       # sinks past one block, not a multiple of 8
    (1, 1, 1, 600, 600, 128, 128, 125),       # the sinks' places fill a block exactly
    (1, 1, 1, 600, 600, 64, 1, 0),            # each query sees itself only
    (1, 2, 1, 520, 520, 256, 200, 7),
    (1, 2, 1, 520, 520, 160, 90, 64),
    (1, 2, 2, 400, 400, 32, 150, 16),
    (1, 1, 1, 513, 513, 96, 10000, 3),        # the window exceeds the history: causal
    (1, 1, 1, 513, 513, 128, 7, 10000),       # so do the sinks
    (1, 2, 1, 300, 1500, 128, 333, 20),       # a chunk appended to a history
    (1, 2, 2, 500, 200, 128, 60, 5),          # more queries than keys: the first rows see nothing
    (2, 8, 2, 17, 900, 128, 100, 4),          # group rows over two tiles
    (1, 32, 1, 9, 2000, 256, 300, 50),
    (1, 8, 2, 40, 5000, 64, 2000, 256),       # key split
    (1, 1, 1, 256, 20000, 128, 4096, 128),
    # two shares as a cluster: ragged last tiles, rows without keys, one share without any
    (1, 3, 3, 700, 700, 96, 300, 2), (2, 4, 2, 257, 3000, 128, 1500, 9), (1, 2, 2, 900, 500, 64, 450, 0),
    (1, 5, 1, 385, 2000, 32, 2000, 0), (3, 8, 8, 512, 1024, 128, 384, 70),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", TILED, ids=str)
def test_tiled_forward(case, dtype):
    B, Hq, Hkv, Nq, Nk, d, window, sinks = case
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, dtype, 100 + TILED.index(case))
    check_fwd(q, k, v, window, sinks)


DECODE = [
    (1, 4, 1, 1, 1, 128, 1, 0), (1, 4, 1, 1, 1, 64, 5, 5), (3, 8, 2, 1, 700, 128, 128, 4),
    (2, 16, 1, 1, 5000, 64, 1000, 100), (2, 8, 2, 4, 333, 128, 50, 3), (1, 4, 2, 8, 5, 128, 2, 1),
    (1, 2, 2, 16, 1000, 96, 1, 64), (2, 4, 4, 2, 129, 32, 64, 0), (1, 8, 1, 2, 300, 128, 1000, 1000),
    (1, 1, 1, 3, 4097, 128, 2048, 65),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(case, dtype):
    B, Hq, Hkv, Nq, Nk, d, window, sinks = case
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, dtype, 200 + DECODE.index(case))
    check_fwd(q, k, v, window, sinks)


BACKWARD = [
    (1, 2, 1, 300, 300, 128, 64, 4), (2, 4, 2, 333, 333, 64, 100, 1), (1, 2, 2, 700, 700, 128, 257, 130),
    (1, 1, 1, 600, 600, 64, 1, 0), (1, 2, 1, 520, 520, 256, 200, 7), (1, 2, 1, 300, 300, 160, 90, 64),
    (1, 2, 2, 400, 400, 32, 150, 16), (1, 1, 1, 257, 257, 96, 10000, 3), (1, 1, 1, 300, 300, 128, 7, 10000),
    (1, 2, 1, 300, 1500, 128, 333, 20),       # keys that no query sees: zero gradients
    (1, 2, 2, 500, 200, 128, 60, 5), (1, 8, 1, 1, 200, 128, 60, 5),
    (1, 2, 1, 4000, 4000, 64, 130, 4),        # the sinks' block is shared between CTAs
    (1, 2, 1, 2500, 2500, 256, 70, 200),      # and so are two of them
    (1, 8, 1, 2048, 2048, 128, 512, 0),       # few units: the others are shared too
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", BACKWARD, ids=str)
def test_backward(case, dtype):
    B, Hq, Hkv, Nq, Nk, d, window, sinks = case
    q, k, v, dout = make(B, Hq, Hkv, Nq, Nk, d, dtype, 300 + BACKWARD.index(case))
    o, lse = check_fwd(q, k, v, window, sinks)
    dq, dk, dv = fa.fa_bwd_window(q, k, v, o, dout, lse, window, sinks)
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    r = ref_of(q, k, v, window, sinks, dout)
    close(dq, r.dq, r.dq_tol, "dq")
    close(dk, r.dk, r.dk_tol, "dk")
    close(dv, r.dv, r.dv_tol, "dv")


def test_gradient_against_differences():
    """The kernel's gradient along a direction against central differences of the fp64 forward."""
    q, k, v, dout = make(1, 2, 1, 200, 200, 64, FP16, 400)
    window, sinks = 50, 3
    o, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    grads = fa.fa_bwd_window(q, k, v, o, dout, lse, window, sinks)
    r = ref_of(q, k, v, window, sinks, dout)
    seen = window_seen(200, 200, window, sinks, q.device).repeat(2, 1)

    def loss(x):
        s = torch.where(seen, grouped(x[0], 1) @ x[1].transpose(-1, -2) / 8.0, -math.inf)
        return (torch.softmax(s, -1) @ x[2] * grouped(dout, 1).double()).sum()

    x = [t.double() for t in (q, k, v)]
    g = torch.Generator(device="cuda").manual_seed(401)
    for i, (got, tol) in enumerate(zip(grads, (r.dq_tol, r.dk_tol, r.dv_tol))):
        way = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        lo, hi = (loss([t + f * h * way if j == i else t for j, t in enumerate(x)]) for f in (-1, 1))
        # bound: the elements' own, and h^2 and rounding of the differences
        bound = float((tol.reshape(way.shape) * way.abs()).sum()) + 1e-4
        assert abs(float((got.double() * way).sum() - (hi - lo) / (2 * h))) <= bound


@pytest.mark.parametrize("shared", [False, True])
def test_backward_repeats_and_workspaces(shared):
    """dk and dv repeat bitwise; a workspace without room for the partials gives the same to rounding."""
    q, k, v, dout = make(1, 4, 2, 3000, 3000, 64, BF16, 500)
    window, sinks = 200, 4
    o, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    need = fa.fa_bwd_window_workspace_size(1, 4, 2, 3000, 3000, 64, window, sinks)
    least = fa.fa_bwd_workspace_size(1, 4, 2, 64, 64, 64)   # of another shape: too small
    with pytest.raises(fa.FaError) as e:
        fa.fa_bwd_window(q, k, v, o, dout, lse, window, sinks, workspace=torch.empty(least, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fa.FA_ERR_WORKSPACE
    rows = 4 * 3008
    unshared = 2 * ((rows * 4 + 255) // 256 * 256) + (rows * 64 * 4 + 255) // 256 * 256
    assert need > unshared
    ws = torch.empty(need if shared else unshared, dtype=torch.uint8, device="cuda")
    r = ref_of(q, k, v, window, sinks, dout)
    first = fa.fa_bwd_window(q, k, v, o, dout, lse, window, sinks, workspace=ws)
    for got, ref, tol in zip(first, (r.dq, r.dk, r.dv), (r.dq_tol, r.dk_tol, r.dv_tol)):
        close(got, ref, tol, "gradient")
    for _ in range(3):
        again = fa.fa_bwd_window(q, k, v, o, dout, lse, window, sinks, workspace=ws)
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])


# shapes whose plans differ: the units of the sinks' blocks shared, the others, both, neither
SPLITS = [((1, 8, 1, 1500, 1500, 64, 1400, 4), True, True), ((1, 2, 1, 4000, 4000, 64, 130, 4), False, True),
          ((1, 32, 8, 8192, 8192, 64, 4096, 4), True, False), ((2, 8, 8, 1000, 1000, 64, 200, 0), False, False),
          ((1, 8, 1, 2048, 2048, 64, 512, 0), True, False)]


@pytest.mark.parametrize("case", SPLITS, ids=str)
def test_backward_stays_inside_its_workspace(case):
    shape, others, sinks_too = case
    split, sink_split = fa.fa_bwd_window_query_split(*shape)
    assert (split > 1, sink_split > 1) == (others, sinks_too)
    B, Hq, Hkv, Nq, Nk, d, window, sinks = shape
    q, k, v, dout = make(B, Hq, Hkv, Nq, Nk, d, BF16, 550)
    o, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    n, guard = fa.fa_bwd_window_workspace_size(*shape), 1 << 21
    buf = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
    got = fa.fa_bwd_window(q, k, v, o, dout, lse, window, sinks, workspace=buf[guard:guard + n])
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    assert (buf[:guard] == 0x5A).all() and (buf[guard + n:] == 0x5A).all()
    Hn, G = min(Hkv, 2), Hq // Hkv   # the last kv heads against fp64
    r = ref_of(q[:, -Hn * G:], k[:, -Hn:], v[:, -Hn:], window, sinks, dout[:, -Hn * G:])
    for x, ref, tol in zip(got, (r.dq, r.dk, r.dv), (r.dq_tol, r.dk_tol, r.dv_tol)):
        close(x[:, -ref.shape[1] * x.shape[1] // Hkv:].reshape(ref.shape), ref, tol, "gradient")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("Nq,Hq", [(1, 4), (3, 4), (200, 2), (40, 8)])
def test_unseen_keys_may_hold_anything(Nq, Hq, bad):
    """Keys between the sinks and the first query's window: NaN or infinite K and V change nothing."""
    Nk, window, sinks = 1000, 130, 5
    q, k, v, dout = make(1, Hq, 2, Nq, Nk, 128, BF16, 600 + Nq)
    o0, l0 = fa.fa_fwd_window(q, k, v, window, sinks)
    g0 = fa.fa_bwd_window(q, k, v, o0, dout, l0, window, sinks)
    first = Nk - Nq - window + 1
    k[:, :, sinks:first], v[:, :, sinks:first] = bad, bad
    o1, l1 = fa.fa_fwd_window(q, k, v, window, sinks)
    g1 = fa.fa_bwd_window(q, k, v, o1, dout, l1, window, sinks)
    torch.cuda.synchronize()
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    assert torch.equal(g0[1], g1[1]) and torch.equal(g0[2], g1[2])
    assert torch.isfinite(g1[0]).all() and (g1[0].float() - g0[0].float()).abs().max() <= 2.0 ** -7 * g0[0].float().abs().max()
    assert not g1[1][:, :, sinks:first].any() and not g1[2][:, :, sinks:first].any()


def paged(k, v, lens, page, seed, spare=3):
    """k, v [B, Hkv, Nk, d] as pools of pages in random order; what no sequence holds is NaN."""
    B, Hkv, Nk, d = k.shape
    per = -(-Nk // page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = torch.randperm(B * per + spare, generator=g, device="cuda")
    table = order[: B * per].view(B, per)
    pools = []
    for t in (k, v):
        t = t.clone()
        for b, n in enumerate(lens):
            t[b, :, n:] = math.nan
        pool = torch.full((B * per + spare, page, Hkv, d), math.nan, dtype=t.dtype, device="cuda")
        full = torch.full((B, per * page, Hkv, d), math.nan, dtype=t.dtype, device="cuda")
        full[:, :Nk] = t.transpose(1, 2)
        pool[table.reshape(-1)] = full.view(B * per, page, Hkv, d)
        pools.append(pool)
    return pools[0], pools[1], table.to(torch.int32).contiguous()


PAGED = [
    # Hq, Hkv, Nq, d, page, lens, window, sinks
    (8, 2, 1, 128, 64, [1, 700, 300, 0], 128, 4), (8, 8, 1, 64, 128, [1000, 65], 64, 0),
    (4, 1, 4, 128, 64, [3, 200, 129], 33, 70), (16, 1, 1, 96, 256, [5000], 2000, 1),
    (8, 2, 2, 128, 64, [640, 64, 1], 100000, 0), (8, 2, 1, 32, 64, [640, 641], 1, 1),
    # lists longer than the GPU's CTAs, cut anywhere; more sequences than threads; empty ones between
    (16, 4, 1, 128, 64, [9000, 0, 64, 8000, 1], 5000, 130), (4, 2, 1, 64, 64, [(37 * i) % 200 for i in range(300)], 70, 3),
    (32, 8, 1, 128, 64, [2000 + i for i in range(64)], 1024, 4), (2, 1, 8, 128, 64, [0, 0, 5], 100, 0), (2, 2, 1, 64, 64, [0, 0], 3, 3),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", PAGED, ids=str)
def test_paged(case, dtype):
    Hq, Hkv, Nq, d, page, lens, window, sinks = case
    B, Nk = len(lens), max(max(lens), 1)
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, dtype, 700 + PAGED.index(case))
    kp, vp, table = paged(k, v, lens, page, 800)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):   # pages behind the sinks and before the window: given to others
        for t in range(-(-sinks // page), max(0, n - Nq - window + 1) // page):
            table[b, t] = 10 ** 6 if t % 2 else -1
    o, lse = fa.fa_fwd_paged_window(q, kp, vp, table, ln, window, sinks)
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    for b, n in enumerate(lens):
        if n == 0:
            assert not o[b].any() and torch.isneginf(lse[b]).all()
            continue
        r = ref_of(q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n], window, sinks)
        close(o[b:b + 1], r.o, r.o_tol, f"o of sequence {b}")
        close(lse[b:b + 1], r.lse, r.lse_tol, f"lse of sequence {b}")


def test_paged_workspace_and_outputs_given():
    q, k, v, _ = make(2, 8, 2, 1, 900, 128, BF16, 900)
    kp, vp, table = paged(k, v, [900, 800], 64, 901)
    ln = torch.tensor([900, 800], dtype=torch.int32, device="cuda")
    need = fa.fa_fwd_paged_window_workspace_size(2, 8, 2, 1, 64, table.shape[1], 128, 300, 4)
    o, lse = torch.empty_like(q), torch.empty(2, 8, 1, device="cuda")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    fa.fa_fwd_paged_window(q, kp, vp, table, ln, 300, 4, o, lse, workspace=ws)
    o2, l2 = fa.fa_fwd_paged_window(q, kp, vp, table, ln, 300, 4)
    assert need > 0 and torch.equal(o, o2) and torch.equal(lse, l2)
    with pytest.raises(fa.FaError) as e:
        fa.fa_fwd_paged_window(q, kp, vp, table, ln, 300, 4, workspace=ws[:-256].contiguous())
    assert e.value.status == fa.FA_ERR_WORKSPACE


def test_whole_window_is_causal_attention():
    """A window, or sinks, over the whole history is the causal forward: both within the bounds of the same
    reference (which blocks take the software exponential, and how keys are split, may differ)."""
    q, k, v, dout = make(1, 4, 2, 640, 640, 128, BF16, 1000)
    o1, l1 = fa.fa_fwd(q, k, v, causal=True)
    r = ref_of(q, k, v, 640, 640)
    close(o1, r.o, r.o_tol, "o of the causal forward")
    for window, sinks in ((640, 0), (2 ** 31 - 1, 0), (2 ** 40, 0), (1, 2 ** 32 + 640)):   # larger than an int: no remainder
        o2, l2 = fa.fa_fwd_window(q, k, v, window, sinks)
        close(o2, r.o, r.o_tol, "o")
        close(l2, r.lse, r.lse_tol, "lse")


def test_other_stream_and_given_outputs():
    """On a stream that is not current, into outputs of the caller, with a scale of its own."""
    q, k, v, dout = make(2, 4, 2, 150, 400, 96, FP16, 1050)
    s = torch.cuda.Stream()
    o, lse = torch.full_like(q, 9), torch.full(q.shape[:3], 9.0, device="cuda")
    grads = [torch.full_like(t, 9) for t in (q, k, v)]
    s.wait_stream(torch.cuda.current_stream())
    assert fa.fa_fwd_window(q, k, v, 70, 6, o, lse, scale=0.2, stream=s)[0] is o
    fa.fa_bwd_window(q, k, v, o, dout, lse, 70, 6, *grads, scale=0.2, stream=s)
    s.synchronize()
    seen = window_seen(150, 400, 70, 6, q.device).repeat(2, 1)
    r = Ref(grouped(q, 2), k, v, seen, scale=0.2, dout=grouped(dout, 2))
    close(o, r.o, r.o_tol, "o")
    close(lse, r.lse, r.lse_tol, "lse")
    for got, ref, tol in zip(grads, (r.dq, r.dk, r.dv), (r.dq_tol, r.dk_tol, r.dv_tol)):
        close(got, ref, tol, "gradient")
    with pytest.raises(ValueError):
        fa.fa_fwd_window(q, k.transpose(2, 3).contiguous().transpose(2, 3), v, 70)   # not contiguous
    with pytest.raises(ValueError):
        fa.fa_fwd_window(q, k, v, 70, o=o.bfloat16())


def test_graph_and_streams():
    """Captured into a graph and replayed on new inputs, and two windows in flight on two streams."""
    q, k, v, dout = make(1, 4, 2, 700, 700, 64, BF16, 1100)
    q2, k2, v2, dout2 = make(1, 4, 2, 700, 700, 64, BF16, 1101)

    def step(q, k, v, dout, window):
        o, lse = fa.fa_fwd_window(q, k, v, window, 4)
        return (o, lse) + fa.fa_bwd_window(q, k, v, o, dout, lse, window, 4)

    want = {w: step(q2, k2, v2, dout2, w) for w in (100, 333)}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(q, k, v, dout, 100)
    for a, b in ((q, q2), (k, k2), (v, v2), (dout, dout2)):
        a.copy_(b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()

    def same(got, want):
        assert all(torch.equal(got[i], want[i]) for i in (0, 1, 3, 4))
        assert (got[2].float() - want[2].float()).abs().max() <= 2.0 ** -7 * want[2].float().abs().max()

    same(got, want[100])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i, s in enumerate(streams):
        w = (100, 333)[i]
        o, lse = fa.fa_fwd_window(q2, k2, v2, w, 4, stream=s)
        outs.append((o, lse) + fa.fa_bwd_window(q2, k2, v2, o, dout2, lse, w, 4, stream=s))
    torch.cuda.synchronize()
    same(outs[0], want[100])
    same(outs[1], want[333])
    fa.fa_check_device_status()


def test_more_keys_than_two_pow_31_elements():
    """A cache whose K passes 2^31 elements: offsets past 32 bits."""
    B, Hkv, Nk, d, window, sinks = 5, 4, 1 << 20, 128, 1000, 4
    q = torch.randn(B, 8, 1, d, device="cuda", dtype=BF16)
    k = torch.zeros(B, Hkv, Nk, d, device="cuda", dtype=BF16)
    v = torch.zeros_like(k)
    for t in (k, v):
        t[:, :, :sinks].normal_()
        t[:, :, -window:].normal_()
    o, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    keep = list(range(sinks)) + list(range(Nk - window, Nk))
    kk, vv = k[:, :, keep], v[:, :, keep]
    del k, v
    r = Ref(grouped(q, Hkv), kk, vv, torch.ones(1, len(keep), dtype=torch.bool, device="cuda"))
    close(o, r.o, r.o_tol, "o")
    close(lse, r.lse, r.lse_tol, "lse")
