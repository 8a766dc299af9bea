"""Attention of a batch whose sequences share a prefix (fa_fwd_prefix) against fp64."""
import math

import pytest
import torch

import exact_attention_114_b200 as fa
from tests.masked_ref import Ref, close
from tests.test_gpu_window import BF16, FP16, grouped, make

pytestmark = pytest.mark.gpu


def make_prefix(B, Hq, Hkv, Nq, Np, Ns, d, dtype, seed):
    q, k, v, _ = make(B, Hq, Hkv, Nq, Ns, d, dtype, seed)
    _, kp, vp, _ = make(1, 1, Hkv, 1, Np, d, dtype, seed + 1)
    return q, kp[0].contiguous(), vp[0].contiguous(), k, v


def check(q, kp, vp, k, v, lens, causal, o, lse):
    B, Hq, Nq, d = q.shape
    Hkv, Np, Ns = k.shape[1], kp.shape[1], k.shape[2]
    for b in range(B):
        n = Ns if lens is None else min(lens[b], Ns)
        kk, vv = (torch.cat([p, x[b, :, :n]], 1) for p, x in ((kp, k), (vp, v)))
        m = Np + n
        x = (torch.arange(Nq, device="cuda") + m - Nq).unsqueeze(1) if causal else torch.full((Nq, 1), m, device="cuda")
        seen = (torch.arange(m, device="cuda") <= x).repeat(Hq // Hkv, 1)
        r = Ref(grouped(q[b:b + 1], Hkv)[0], kk, vv, seen)
        # partials and their merge: each in fp32
        close(o[b].reshape(Hkv, -1, d), r.o, r.o_tol, f"o of sequence {b}")
        close(lse[b].reshape(Hkv, -1), r.lse, r.lse_tol, f"lse of sequence {b}")


CASES = [
    # B, Hq, Hkv, Nq, Np, Ns, d, lens
    (3, 8, 2, 1, 500, 70, 128, [70, 1, 33]),             # packed tiles, split-KV for the own keys
    (40, 8, 2, 1, 1000, 130, 64, None),                  # several packed tiles, the last one ragged
    (5, 4, 4, 1, 128, 64, 96, [0, 64, 1, 63, 40]),       # a sequence without keys of its own
    (2, 16, 1, 1, 1, 1, 32, [1, 0]),
    (9, 6, 2, 4, 333, 50, 128, [50, 4, 3, 1, 0, 7, 20, 49, 50]),   # fewer own keys than rows
    (4, 8, 2, 9, 700, 129, 128, [129, 128, 9, 60]),      # 36 rows: the tiled kernel for the own keys
    (3, 2, 1, 32, 300, 300, 64, [300, 200, 32]),
    (7, 8, 1, 1, 900, 77, 256, [77, 1, 2, 30, 50, 0, 60]),
    (3, 4, 2, 5, 260, 40, 160, [40, 5, 2]),
    (1, 8, 2, 1, 700, 30, 128, [30]),                    # one sequence: one launch
    (2, 8, 2, 64, 500, 200, 128, [200, 64]),             # rows fill a tile: one launch
    (3, 4, 2, 33, 400, 100, 64, [100, 33, 10]),
    (2, 2, 2, 300, 200, 333, 128, [333, 300]),
    (1, 2, 1, 200, 100, 150, 256, [150]),
    (2, 4, 1, 100, 3, 7, 64, [7, 0]),                    # rows far longer than all keys: some see nothing
    (2, 4, 1, 3, 1, 2, 128, [2, 0]),
    (64, 4, 2, 1, 5000, 40, 128, None),                  # key shares of the prefix
    # packed tiles with the split-KV pass for the own keys (prefixes too long to be read per sequence)
    (70, 16, 8, 1, 520, 140, 64, [(31 * i) % 141 for i in range(70)]),
    (67, 8, 8, 2, 513, 300, 128, [300] * 3 + [1, 0, 2] * 20 + [299] * 4),
    (33, 32, 2, 1, 4100, 5, 96, [i % 6 for i in range(33)]),
    (130, 4, 4, 1, 520, 64, 32, [0] * 129 + [64]),
    (130, 4, 4, 1, 520, 64, 32, [0] * 130),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_prefix(case, causal, dtype):
    *shape, lens = case
    q, kp, vp, k, v = make_prefix(*shape, dtype, 3000 + CASES.index(case))
    if lens is not None:   # the batch's padding holds anything
        for b, n in enumerate(lens):
            k[b, :, n:], v[b, :, n:] = math.nan, math.inf
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_prefix(q, kp, vp, k, v, ln, causal=causal)
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    check(q, kp, vp, k, v, lens, causal, o, lse)


def test_workspace_outputs_and_clamped_lengths():
    shape = (6, 8, 2, 2, 900, 64, 128)
    q, kp, vp, k, v = make_prefix(*shape, BF16, 3100)
    ln = torch.tensor([64, 1000, -5, 0, 1, 30], dtype=torch.int32, device="cuda")
    need = fa.fa_fwd_prefix_workspace_size(*shape)
    guard = 512
    buf = torch.full((need + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    fa.fa_fwd_prefix(q, kp, vp, k, v, ln, o, lse, causal=True, workspace=buf[guard:guard + need])
    o2, l2 = fa.fa_fwd_prefix(q, kp, vp, k, v, ln, causal=True)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert (buf[:guard] == 0x5A).all() and (buf[guard + need:] == 0x5A).all()
    check(q, kp, vp, k, v, [64, 64, 0, 0, 1, 30], True, o, lse)
    with pytest.raises(fa.FaError) as e:
        fa.fa_fwd_prefix(q, kp, vp, k, v, ln, causal=True, workspace=buf[:need - 256].clone())
    assert e.value.status == fa.FA_ERR_WORKSPACE
    # no lse wanted
    p = fa._ptr
    o3 = torch.empty_like(q)
    assert fa.lib().fa_fwd_prefix(0, p(q), p(kp), p(vp), p(k), p(v), p(ln), p(o3), None, *shape, 1 / math.sqrt(128), 1,
                                  None, 0, fa._stream(None)) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, o3)


def test_matches_the_concatenated_cache():
    """The plain forward on prefix and own keys laid out per sequence: equal to rounding."""
    B, Hq, Hkv, Np, Ns, d = 4, 32, 8, 1024, 128, 128
    q, kp, vp, k, v = make_prefix(B, Hq, Hkv, 1, Np, Ns, d, BF16, 3200)
    o, lse = fa.fa_fwd_prefix(q, kp, vp, k, v)
    cat = [torch.cat([p.expand(B, -1, -1, -1), x], 2).contiguous() for p, x in ((kp, k), (vp, v))]
    o1, l1 = fa.fa_fwd(q, *cat)
    torch.cuda.synchronize()
    assert (o.float() - o1.float()).abs().max() <= 2.0 ** -7 * o1.float().abs().max()
    assert (lse - l1).abs().max() <= 1e-5


@pytest.mark.parametrize("Nq,Np", [(1, 900), (1, 33000), (9, 900), (64, 900)])
def test_graph_streams_and_repeats(Nq, Np):
    shape = (6, 8, 2, Nq, Np, 100, 128)
    q, kp, vp, k, v = make_prefix(*shape, BF16, 3300)
    q2, kp2, vp2, k2, v2 = make_prefix(*shape, BF16, 3400)
    ln = torch.tensor([100, 64, 70, 80, 90, 99], dtype=torch.int32, device="cuda")
    want = fa.fa_fwd_prefix(q2, kp2, vp2, k2, v2, ln, causal=True)
    other = fa.fa_fwd_prefix(q, kp, vp, k, v, ln, causal=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = fa.fa_fwd_prefix(q, kp, vp, k, v, ln, causal=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], other[0]) and torch.equal(got[1], other[1])
    for a, b in ((q, q2), (kp, kp2), (vp, vp2), (k, k2), (v, v2)):
        a.copy_(b)
    graph.replay()
    s = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [fa.fa_fwd_prefix(q2, kp2, vp2, k2, v2, ln, causal=True, stream=x) for x in s for _ in range(3)]
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in outs)


PACKED = [
    # rows of several sequences in a tile and the tiled pass for the own keys: prefixes too long to be read per sequence
    (40, 8, 4, 9, 900, 129, 128, [(17 * i) % 130 for i in range(40)]), (90, 2, 1, 32, 1600, 100, 64, [100 - i for i in range(90)]),
    (75, 8, 2, 1, 1100, 77, 256, [i % 78 for i in range(75)]), (70, 4, 2, 5, 1090, 40, 160, [i % 41 for i in range(70)]),
    (3, 6, 1, 3, 33000, 70, 96, [70, 0, 33]), (2, 32, 1, 2, 33000, 100, 128, None), (129, 2, 2, 64, 520, 65, 32, [0] * 128 + [65]),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", PACKED, ids=lambda c: str(c[:7]))
def test_packed_tiled_prefix(case, causal, dtype):
    *shape, lens = case
    assert fa.fa_fwd_prefix_workspace_size(*shape) > 0   # partials of the prefix pass
    q, kp, vp, k, v = make_prefix(*shape, dtype, 3500 + PACKED.index(case))
    if lens is not None:
        for b, n in enumerate(lens):
            k[b, :, n:], v[b, :, n:] = math.nan, math.inf
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_prefix(q, kp, vp, k, v, ln, causal=causal)
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    check(q, kp, vp, k, v, lens, causal, o, lse)
