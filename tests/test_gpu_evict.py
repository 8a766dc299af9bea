"""The weights that keys receive (fa_key_weights, fa_fwd_weights) against fp64, and eviction by them
(fa_kv_evict) against a selection by sorting."""
import math

import numpy as np
import pytest
import torch

import exact_attention_114_b200 as fa
from tests.masked_ref import Ref, close
from tests.test_gpu_window import BF16, FP16, grouped, make

pytestmark = pytest.mark.gpu


def ref_of(q, k, v, causal):
    Hkv, G, Nq, Nk = k.shape[1], q.shape[1] // k.shape[1], q.shape[2], k.shape[2]
    x = (torch.arange(Nq, device="cuda") + Nk - Nq).unsqueeze(1) if causal else torch.full((Nq, 1), Nk, device="cuda")
    return Ref(grouped(q, Hkv), k, v, (torch.arange(Nk, device="cuda") <= x).repeat(G, 1))


SHAPES = [
    # B, Hq, Hkv, Nq, Nk, d
    (1, 4, 1, 1, 1, 128), (2, 8, 2, 1, 700, 64), (3, 16, 4, 2, 1000, 128), (1, 16, 1, 1, 5000, 96), (2, 4, 4, 4, 64, 32),
    (1, 2, 1, 300, 300, 128), (2, 4, 2, 333, 333, 64), (1, 2, 2, 500, 200, 128), (1, 4, 2, 200, 1000, 96),
    (1, 8, 2, 17, 900, 128), (1, 2, 1, 129, 257, 256), (1, 32, 2, 1, 513, 256), (1, 16, 1, 1100, 1100, 64),
    (1, 2, 2, 127, 128, 160),
]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", SHAPES, ids=str)
def test_weights(case, causal, dtype):
    q, k, v, _ = make(*case, dtype, 2000 + SHAPES.index(case))
    start = torch.rand(k.shape[:3], device="cuda")
    o, lse, w = fa.fa_fwd_weights(q, k, v, start, causal=causal)
    again = fa.fa_key_weights(q, k, lse, start, causal=causal)
    fresh = fa.fa_key_weights(q, k, lse, causal=causal)
    place = start.clone()
    fa.fa_fwd_weights(q, k, v, place, place, causal=causal)
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    r = ref_of(q, k, v, causal)
    close(o, r.o, r.o_tol, "o")
    close(lse, r.lse, r.lse_tol, "lse")
    close(fresh, r.w, r.w_tol, "fresh weights")
    tol = r.w_tol + 2.0 ** -24 * (r.w + start)
    close(w, r.w + start, tol, "weights")
    close(again, r.w + start, tol, "weights from lse")
    assert torch.equal(place, w)
    # every row that sees a key gives one weight in all
    rows = torch.isfinite(lse).sum().item()
    assert abs(fresh.double().sum().item() - rows) <= float(r.w_tol.sum())


def test_weights_without_lse_and_long_rows():
    """lse may be left out in C; many rows of one key block are shared between CTAs."""
    q, k, v, _ = make(1, 8, 1, 4096, 4096, 64, BF16, 2100)
    o, lse, w = fa.fa_fwd_weights(q, k, v, causal=True)
    w2, o2 = torch.empty_like(w), torch.empty_like(o)
    p = fa._ptr
    assert fa.lib().fa_fwd_weights(0, p(q), p(k), p(v), p(o2), None, None, p(w2), 1, 8, 1, 4096, 4096, 64, 0.125, 1,
                                   fa._stream(None)) == 0
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    assert torch.equal(w, w2) and torch.equal(o, o2)
    r = ref_of(q, k, v, True)
    close(w, r.w, r.w_tol, "weights")


def select(w, keep, recent):
    """The kept keys of one cache: the newest, then the heaviest (NaN above all), the lower index first."""
    w = np.asarray(w, np.float64) + 0.0
    n = len(w)
    order = np.where(np.isnan(w), np.inf, w)
    newest = np.arange(n) >= n - recent
    return np.sort(np.lexsort((np.arange(n), -order, ~np.isnan(w), ~newest))[:keep])


WEIGHTS = ["random", "ties", "equal", "wild"]


def weights_of(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(shape, generator=g)
    if kind == "ties":
        w = (w * 5).floor() / 4
    elif kind == "equal":
        w = torch.full(shape, 0.25)
    elif kind == "wild":
        w = torch.randn(shape, generator=g) * torch.exp(20 * torch.randn(shape, generator=g))
        pick = torch.rand(shape, generator=g)
        for lo, x in ((0.0, math.nan), (0.1, math.inf), (0.2, -math.inf), (0.3, 0.0), (0.4, -0.0)):
            w[(pick >= lo) & (pick < lo + 0.05)] = x
    return w


EVICT = [
    # B, Hkv, Nk, d, keep, recent
    (1, 1, 1, 64, 1, 0), (2, 3, 300, 64, 77, 5), (1, 2, 1000, 128, 1, 1), (1, 2, 1000, 96, 1, 0), (2, 2, 4097, 32, 1024, 1024),
    (1, 4, 5000, 256, 4999, 100), (3, 1, 64, 160, 100, 10), (1, 1, 100000, 64, 3000, 7), (1, 2, 33, 128, 32, 0),
]


@pytest.mark.parametrize("kind", WEIGHTS)
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict(case, kind):
    B, Hkv, Nk, d, keep, recent = case
    dtype = BF16 if EVICT.index(case) % 2 else FP16
    _, k, v, _ = make(B, 1, Hkv, 1, Nk, d, dtype, 2200)
    w = weights_of(kind, (B, Hkv, Nk), 2300 + EVICT.index(case))
    ko, vo, wo, index = fa.fa_kv_evict(k, v, w.cuda(), keep, recent)
    torch.cuda.synchronize()
    n = min(keep, Nk)
    for b in range(B):
        for h in range(Hkv):
            want = torch.from_numpy(select(w[b, h].numpy(), n, recent))
            assert torch.equal(index[b, h, :n].cpu().long(), want)
            assert torch.equal(ko[b, h, :n], k[b, h, want.cuda()]) and torch.equal(vo[b, h, :n], v[b, h, want.cuda()])
            assert torch.equal(wo[b, h, :n].cpu().nan_to_num(7.0), w[b, h, want].nan_to_num(7.0))
    assert (index[:, :, n:] == -1).all() and not ko[:, :, n:].any() and not wo[:, :, n:].any()


MANY = {
    # weights of 20000 keys of which more than 8192 share sign, exponent and two bits of the mantissa
    "equal": lambda w: torch.full_like(w, 0.25), "zeros": torch.zeros_like, "two": lambda w: torch.where(w < 0.4, 0.25, 0.26),
    "close": lambda w: 1.0 + 0.2 * w, "signs": lambda w: torch.where(w < 0.5, -1.0, -1.1),
}


@pytest.mark.parametrize("kind", MANY)
@pytest.mark.parametrize("keep,recent", [(6000, 100), (19999, 0)])
def test_evict_many_alike(kind, keep, recent):
    """More keys alike in the first digit than the list holds, while all are held in shared memory; a block per
    (batch, kv head) on many SMs at once, repeated: every run selects the same."""
    B, Hkv, Nk, d = 4, 40, 20000, 32
    _, k, v, _ = make(B, 1, Hkv, 1, Nk, d, BF16, 2250)
    w = MANY[kind](torch.rand((B, Hkv, Nk), generator=torch.Generator().manual_seed(2251)))
    wg = w.cuda()
    runs = [fa.fa_kv_evict(k, v, wg, keep, recent) for _ in range(8)]
    torch.cuda.synchronize()
    order = w.double()
    order[..., Nk - recent:] = math.inf
    want = torch.sort(order, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    rows = want.cuda().unsqueeze(-1).expand(-1, -1, -1, d)
    for ko, vo, wo, index in runs:
        assert torch.equal(index.cpu().long(), want)
        assert torch.equal(ko, torch.gather(k, 2, rows)) and torch.equal(vo, torch.gather(v, 2, rows))
        assert torch.equal(wo.cpu(), torch.gather(w, 2, want))


@pytest.mark.parametrize("keep,recent", [(50, 10), (1, 1), (200, 0)])
def test_evict_lengths_and_rows_left_alone(keep, recent):
    """Sequences of their own lengths (none, one, the budget, one more, all): rows behind the last kept key stay."""
    lens = [0, 1, keep, keep + 1, 300, 1000]   # the last is past the cache: clamped to 300
    B, Hkv, Nk, d = len(lens), 2, 300, 64
    _, k, v, _ = make(B, 1, Hkv, 1, Nk, d, BF16, 2400)
    w = weights_of("ties", (B, Hkv, Nk), 2401)
    outs = [torch.full((B, Hkv, keep, d), 3.0, dtype=BF16, device="cuda") for _ in range(2)]
    wo, io = torch.full((B, Hkv, keep), 4.0, device="cuda"), torch.full((B, Hkv, keep), 5, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):   # what lies behind a sequence's end is no candidate
        w[b, :, n:] = math.inf
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fa.fa_kv_evict(k, v, w.cuda(), keep, recent, ln, outs[0], outs[1], wo, io)
    torch.cuda.synchronize()
    for b, n in enumerate(min(x, Nk) for x in lens):
        c = min(n, keep)
        for h in range(Hkv):
            want = torch.from_numpy(select(w[b, h, :n].numpy(), c, min(recent, n)))
            assert torch.equal(io[b, h, :c].cpu().long(), want)
            assert torch.equal(outs[0][b, h, :c], k[b, h, want.cuda()]) and torch.equal(outs[1][b, h, :c], v[b, h, want.cuda()])
        assert (outs[0][b, :, c:] == 3).all() and (outs[1][b, :, c:] == 3).all()
        assert (wo[b, :, c:] == 4).all() and (io[b, :, c:] == 5).all()


def test_evict_without_index_and_weights():
    _, k, v, _ = make(1, 1, 2, 1, 500, 128, BF16, 2500)
    w = torch.rand(1, 2, 500, device="cuda")
    ko, vo, _, _ = fa.fa_kv_evict(k, v, w, 100, 20)
    k2, v2 = torch.empty_like(ko), torch.empty_like(vo)
    p = fa._ptr
    assert fa.lib().fa_kv_evict(0, p(k), p(v), p(w), None, p(k2), p(v2), None, None, 1, 2, 500, 128, 100, 20, fa._stream(None)) == 0
    torch.cuda.synchronize()
    assert torch.equal(ko, k2) and torch.equal(vo, v2)
    with pytest.raises(fa.FaError, match="overlap"):
        fa.fa_kv_evict(k, v, w, 500, 0, None, k, v2.new_empty(1, 2, 500, 128))


def test_a_cache_in_use():
    """Prompt with weights, eviction, decode steps that go on adding, a second eviction; and the eager
    run and a captured one replayed give the same."""
    B, Hq, Hkv, d, N, keep = 2, 8, 2, 128, 700, 256
    q, k, v, _ = make(B, Hq, Hkv, N, N, d, BF16, 2600)
    steps = [make(B, Hq, Hkv, 1, 1, d, BF16, 2601 + i)[:3] for i in range(3)]

    def run():
        _, _, w = fa.fa_fwd_weights(q, k, v, causal=True)
        kc, vc, wc, index = fa.fa_kv_evict(k, v, w, keep, 32)
        outs = [w, index]
        for qs, ks, vs in steps:
            kc, vc = torch.cat([kc, ks], 2), torch.cat([vc, vs], 2)
            wc = torch.cat([wc, wc.new_zeros(B, Hkv, 1)], 2)
            o, lse, wc = fa.fa_fwd_weights(qs, kc, vc, wc)
            outs += [o, lse, wc]
        return outs + list(fa.fa_kv_evict(kc, vc, wc, keep, 32))

    want = run()
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    # the second step against fp64 on the cache as it was kept
    idx = want[1].long().unsqueeze(-1).expand(-1, -1, -1, d)
    kk = torch.cat([torch.gather(k, 2, idx), steps[0][1]], 2)
    vv = torch.cat([torch.gather(v, 2, idx), steps[0][2]], 2)
    r = ref_of(steps[0][0], kk, vv, False)
    close(want[2], r.o, r.o_tol, "o behind an eviction")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
