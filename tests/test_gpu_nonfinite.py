"""A NaN, or a score that overflows, shows in every row that reads it and in no other, wherever a row's keys are
cut between CTAs: O and LSE are NaN then, and LSE = -inf stays what a row without keys gets."""
import math

import pytest
import torch

import exact_attention_114_b200 as fa
from tests.masked_ref import Ref, close, window_seen
from tests.test_gpu_prefix import make_prefix
from tests.test_gpu_window import BF16, FP16, grouped, make, paged

pytestmark = pytest.mark.gpu


def check_rows(got, base, bad):
    """o and lse are NaN in the rows `bad` [B, Hq, Nq] and bitwise as before in the others."""
    torch.cuda.synchronize()
    fa.fa_check_device_status()
    (o, lse), (o0, l0) = got, base
    assert torch.isnan(lse[bad]).all() and torch.isnan(o[bad]).all()
    assert torch.equal(o[~bad], o0[~bad]) and torch.equal(lse[~bad], l0[~bad])


def rows_of(seen, j, B, Hq, Hkv, b, hk):
    """[B, Hq, Nq]: rows of kv head hk of sequence b that see key j, seen [Nq, Nk]."""
    bad = torch.zeros(B, Hq, seen.shape[0], dtype=torch.bool, device="cuda")
    bad[b, hk * (Hq // Hkv):(hk + 1) * (Hq // Hkv)] = seen[:, j]
    return bad


def poison(call, q, k, seen, keys, b=0, hk=0):
    """NaN in a query row, then in one visible key after another (eight in a row, so that every column of a group
    of eight is met): K alone, so that a row that does not see the key has nothing to do with it."""
    B, Hq, Nq, _ = q.shape
    Hkv = k.shape[1]
    base = call(q, k)
    torch.cuda.synchronize()
    for h, i in ((0, 0), (Hq - 1, Nq - 1), (Hq // 2, Nq // 2)):
        q2, bad = q.clone(), torch.zeros(B, Hq, Nq, dtype=torch.bool, device="cuda")
        q2[B - 1, h, i, 3], bad[B - 1, h, i] = math.nan, bool(seen[i].any())
        check_rows(call(q2, k), base, bad)
    for j in keys:
        k2 = k.clone()
        k2[b, hk, j, 5] = math.nan
        check_rows(call(q, k2), base, rows_of(seen, j, B, Hq, Hkv, b, hk))


def eights(*starts):
    return [s + i for s in starts for i in range(8)]


WINDOW = [
    # B, Hq, Hkv, Nq, Nk, d, window, sinks, keys
    (1, 2, 1, 700, 700, 128, 700, 0, eights(0, 400)),        # tiled
    (1, 2, 2, 600, 600, 128, 100, 5, eights(0, 300)),
    (1, 2, 1, 400, 400, 64, 400, 0, eights(130)),
    (1, 8, 1, 40, 5000, 128, 5000, 0, eights(8, 2600)),      # shares merged by a kernel
    (1, 1, 1, 256, 20000, 256, 20000, 0, eights(9000)),
    (1, 4, 2, 512, 4000, 128, 3000, 64, eights(16, 2000)),   # two shares as a cluster
    (1, 8, 2, 1, 60, 128, 60, 0, eights(30)),                # single token, whole
    (2, 8, 2, 1, 9000, 128, 9000, 0, eights(4100)),          # cut between CTAs
    (1, 4, 1, 4, 5000, 64, 3000, 4, [0, 3, 2100, 4998]),
]


@pytest.mark.parametrize("case", WINDOW, ids=str)
def test_window(case):
    B, Hq, Hkv, Nq, Nk, d, window, sinks, keys = case
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, BF16, 4000)
    poison(lambda q, k: fa.fa_fwd_window(q, k, v, window, sinks), q, k, window_seen(Nq, Nk, window, sinks, "cuda"), keys)


@pytest.mark.parametrize("lens,window", [([700], 700), ([9000, 8000], 8000), ([640, 300, 5000], 5000)])
def test_paged_window(lens, window):
    B, Hq, Hkv, d, n = len(lens), 8, 2, 128, lens[0]
    q, k, v, _ = make(B, Hq, Hkv, 1, max(lens), d, FP16, 4100)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call(q, k):
        kp, vp, table = paged(k, v, lens, 64, 4101)
        return fa.fa_fwd_paged_window(q, kp, vp, table, ln, window)

    poison(call, q, k, window_seen(1, n, window, 0, "cuda"), [n - 1, n // 2, n // 2 + 1])


PREFIX = [
    # B, Hq, Hkv, Nq, Np, Ns, d: per sequence, packed with the split-KV or the tiled pass for the own keys, one
    # launch (whole, cut, cluster)
    (3, 8, 2, 1, 500, 70, 128), (2, 8, 2, 1, 9000, 200, 128), (70, 16, 8, 1, 1030, 140, 64), (4, 8, 2, 9, 1500, 300, 128),
    (4, 4, 2, 64, 500, 200, 128), (1, 2, 1, 200, 5000, 300, 256), (2, 4, 2, 128, 2000, 500, 128), (40, 8, 2, 40, 300, 200, 96),
    (40, 8, 4, 9, 900, 129, 128), (75, 8, 2, 1, 1100, 77, 256),
]


@pytest.mark.parametrize("case", PREFIX, ids=str)
def test_prefix(case):
    B, Hq, Hkv, Nq, Np, Ns, d = case
    q, kp, vp, k, v = make_prefix(*case, BF16, 4200)
    seen = (torch.arange(Np + Ns, device="cuda") <= (torch.arange(Nq, device="cuda") + Np + Ns - Nq).unsqueeze(1))
    call = lambda q, k: fa.fa_fwd_prefix(q, kp, vp, k, v, causal=True)  # noqa: E731
    poison(call, q, k, seen[:, Np:], [0, 1, 6, 7, Ns - 1])
    base = call(q, k)
    for j in (0, 6, Np // 2 + 7, Np - 1):   # a prefix key: every row of its kv head in every sequence
        kp2, bad = kp.clone(), torch.zeros(B, Hq, Nq, dtype=torch.bool, device="cuda")
        kp2[1 % Hkv, j, 0] = math.nan
        bad[:, (1 % Hkv) * (Hq // Hkv):(1 % Hkv + 1) * (Hq // Hkv)] = True
        check_rows(fa.fa_fwd_prefix(q, kp2, vp, k, v, causal=True), base, bad)


TILED = [
    # B, Hq, Hkv, Nq, Nk, d, causal, keys: the plain forward that fa_fwd_weights runs for prompts
    (1, 2, 1, 700, 700, 128, True, eights(400)), (1, 4, 2, 300, 900, 64, False, eights(100)), (1, 1, 1, 256, 9000, 128, False, eights(4000)),
    (1, 8, 2, 40, 5000, 64, True, eights(2000)), (1, 2, 2, 100, 9000, 160, False, eights(128)), (2, 2, 1, 300, 300, 256, True, eights(3)),
    (1, 4, 4, 200, 6000, 96, False, eights(5992)),
]


@pytest.mark.parametrize("case", TILED, ids=str)
def test_tiled(case):
    B, Hq, Hkv, Nq, Nk, d, causal, keys = case
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, BF16, 4300)
    seen = window_seen(Nq, Nk, Nk, 0, "cuda") if causal else torch.ones(Nq, Nk, dtype=torch.bool, device="cuda")
    poison(lambda q, k: fa.fa_fwd(q, k, v, causal=causal), q, k, seen, keys)


@pytest.mark.parametrize("shape", [(1, 2, 1, 400, 400, 128), (1, 1, 1, 256, 20000, 256), (1, 4, 2, 512, 4000, 128), (2, 8, 2, 1, 9000, 128),
                                   (1, 4, 4, 2, 200, 64)], ids=str)
def test_infinite_scores(shape):
    """A key with +inf in one column: +inf scores make a row NaN (inf - inf), -inf scores take no weight."""
    B, Hq, Hkv, Nq, Nk, d = shape
    q, k, v, _ = make(*shape, BF16, 4400)
    sign = torch.where(torch.arange(Nq * Hq, device="cuda") % 2 == 0, 1.0, -1.0).to(BF16).view(Hq, Nq)
    q[..., 0] = sign
    seen = window_seen(Nq, Nk, Nk, 0, "cuda")
    for j in eights(Nk // 2) + [0, Nk - 1]:
        k2 = k.clone()
        k2[0, 0, j, 0] = math.inf
        o, lse = fa.fa_fwd_window(q, k2, v, Nk)
        torch.cuda.synchronize()
        at = rows_of(seen, j, B, Hq, Hkv, 0, 0)
        bad = at & (sign > 0)
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
        less = seen.clone()
        less[:, j] = False
        G = Hq // Hkv
        r, r0 = (Ref(grouped(q, Hkv), k, v, s.repeat(G, 1)) for s in (less, seen))
        pick = lambda a, b: torch.where(grouped(at, Hkv).unsqueeze(-1) if a.dim() == 4 else grouped(at, Hkv), a, b)  # noqa: E731
        good = ~grouped(bad, Hkv)
        close(grouped(o, Hkv)[good], pick(r.o, r0.o)[good], pick(r.o_tol, r0.o_tol)[good], "o")
        close(grouped(lse, Hkv)[good], pick(r.lse, r0.lse)[good], pick(r.lse_tol, r0.lse_tol)[good], "lse")


def test_all_scores_minus_infinity():
    """Every visible score -inf: no key has any weight, O = 0 and LSE = -inf, in blocks with and without a mask."""
    for d, Nq, Nk in ((128, 300, 1000), (64, 300, 1000), (128, 1, 1000)):
        q, k, v, _ = make(1, 1, 1, Nq, Nk, d, BF16, 4500)
        q[:, :, ::2, 0], q[:, :, 1::2, 0], k[..., 0] = -1.0, 0.5, math.inf
        o, lse = fa.fa_fwd_window(q, k, v, Nk)
        torch.cuda.synchronize()
        assert not o[:, :, ::2].any() and torch.isneginf(lse[:, :, ::2]).all()
        assert torch.isnan(o[:, :, 1::2]).all() and torch.isnan(lse[:, :, 1::2]).all()


@pytest.mark.parametrize("shape,causal", [((2, 8, 2, 1, 700, 64), False), ((2, 8, 2, 1, 9000, 128), False), ((1, 4, 1, 4, 9000, 128), True)], ids=str)
def test_weights_of_single_tokens(shape, causal):
    """The keys' weights are NaN where a NaN row sees the key, and as before elsewhere: also where units are cut."""
    B, Hq, Hkv, Nq, Nk, d = shape
    q, k, v, _ = make(*shape, BF16, 4600)
    seen = window_seen(Nq, Nk, Nk, 0, "cuda") if causal else torch.ones(Nq, Nk, dtype=torch.bool, device="cuda")
    w0 = fa.fa_fwd_weights(q, k, v, causal=causal)[2]
    for i in {0, Nq - 1}:
        q2 = q.clone()
        q2[0, Hq - 1, i, 1] = math.nan
        w = fa.fa_fwd_weights(q2, k, v, causal=causal)[2]
        bad = torch.zeros_like(w, dtype=torch.bool)
        bad[0, Hkv - 1] = seen[i]
        assert torch.isnan(w[bad]).all() and torch.equal(w[~bad], w0[~bad])
    k2 = k.clone()
    k2[0, 0, Nk // 2, 1] = math.nan
    w = fa.fa_fwd_weights(q, k2, v, causal=causal)[2]
    bad = torch.zeros_like(w, dtype=torch.bool)
    bad[0, 0] = True   # every row sees that key, and some row every key
    assert torch.isnan(w[bad]).all() and torch.equal(w[~bad], w0[~bad])


PROMPTS = [
    # B, Hq, Hkv, Nq, Nk, d, causal: many rows, the last step of a head full or not, a group's rows as one run
    (1, 2, 1, 300, 300, 128, True), (1, 2, 1, 300, 700, 64, False), (1, 2, 2, 256, 513, 128, False), (2, 8, 2, 20, 300, 64, True),
    (1, 2, 1, 200, 300, 256, False), (1, 16, 1, 1100, 1100, 64, True),
]


@pytest.mark.parametrize("case", PROMPTS, ids=str)
def test_weights_of_prompts(case):
    """A NaN query row shows in the weights of every key it sees, whatever its index, and in no other."""
    B, Hq, Hkv, Nq, Nk, d, causal = case
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, BF16, 4650)
    seen = window_seen(Nq, Nk, Nk, 0, "cuda") if causal else torch.ones(Nq, Nk, dtype=torch.bool, device="cuda")
    w0 = fa.fa_fwd_weights(q, k, v, causal=causal)[2]
    assert torch.isfinite(w0).all()
    for i in eights(0, Nq - 8):
        q2 = q.clone()
        q2[0, Hq - 1, i, 1] = math.nan
        w = fa.fa_fwd_weights(q2, k, v, causal=causal)[2]
        bad = torch.zeros_like(w, dtype=torch.bool)
        bad[0, Hkv - 1] = seen[i]
        assert torch.isnan(w[bad]).all() and torch.equal(w[~bad], w0[~bad])


@pytest.mark.parametrize("Nq", [256, 300, 100, 1])
def test_weights_that_vanish_are_zero(Nq):
    """Keys whose scores lie 100 below the others': exp underflows, the weight is 0 and not a small number; and a
    key with an infinite column, whose scores are all -inf, gets 0 too (rows past the last have no say)."""
    q, k, v, _ = make(1, 2, 1, Nq, 700, 64, BF16, 4660)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[:, :, 100:140] = 0.0
    k[:, :, 100:140, 0] = -130.0
    k[:, :, 300, 0] = -math.inf
    o, lse, w = fa.fa_fwd_weights(q, k, v)
    again = fa.fa_key_weights(q, k, lse)
    torch.cuda.synchronize()
    for x in (w, again):
        assert not x[:, :, 100:140].any() and not x[:, :, 300].any() and torch.isfinite(x).all()
        assert abs(float(x.double().sum()) - 2 * Nq) <= 2 * Nq * 1e-4


def test_gradients():
    """A NaN query row: its own gradient, and those of the keys it sees, are NaN, not numbers."""
    q, k, v, dout = make(1, 2, 1, 400, 400, 128, BF16, 4700)
    q[0, 1, 399, 0] = math.nan
    o, lse = fa.fa_fwd_window(q, k, v, 100, 4)
    dq, dk, dv = fa.fa_bwd_window(q, k, v, o, dout, lse, 100, 4)
    torch.cuda.synchronize()
    assert torch.isnan(dq[0, 1, 399]).all()
    for g in (dk, dv):
        assert torch.isnan(g[0, 0, :4]).all() and torch.isnan(g[0, 0, 300:]).all()
    assert torch.isfinite(dv[0, 0, 4:128]).all() and torch.isfinite(dq[0, 0]).all()


@pytest.mark.parametrize("case", [(2, 8, 2, 1, 60, 128, False), (2, 8, 2, 1, 9000, 128, False), (1, 4, 1, 4, 5000, 64, True), (1, 2, 2, 2, 33000, 96, True)],
                         ids=str)
def test_dense_decode(case):
    """The split-KV decode of the plain forward: one split, and several merged."""
    B, Hq, Hkv, Nq, Nk, d, causal = case
    q, k, v, _ = make(B, Hq, Hkv, Nq, Nk, d, BF16, 4800)
    seen = window_seen(Nq, Nk, Nk, 0, "cuda") if causal else torch.ones(Nq, Nk, dtype=torch.bool, device="cuda")
    poison(lambda q, k: fa.fa_fwd(q, k, v, causal=causal), q, k, seen, [0, Nk // 2, Nk // 2 + 1, Nk - 1])


@pytest.mark.parametrize("lens", [[60], [9000, 8000], [640, 300, 5000]])
def test_dense_paged_decode(lens):
    B, Hq, Hkv, d, n = len(lens), 8, 2, 128, lens[0]
    q, k, v, _ = make(B, Hq, Hkv, 1, -(-max(lens) // 64) * 64, d, FP16, 4900)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call(q, k):
        table = torch.arange(B * k.shape[2] // 64, dtype=torch.int32, device="cuda").view(B, -1)
        pool = lambda t: t.transpose(1, 2).reshape(-1, 64, Hkv, d).contiguous()  # noqa: E731
        return fa.fa_fwd_paged(q, pool(k), pool(v), table, ln)

    poison(call, q, k, torch.ones(1, n, dtype=torch.bool, device="cuda"), [0, n // 2, n - 1])


@pytest.mark.parametrize("Nq,Nk", [(300, 300), (128, 20000)])
def test_e4m3(Nq, Nk):
    """The e4m3 forward, whole tiles and key shares: the type's NaN in a query row and in visible keys."""
    g = torch.Generator(device="cuda").manual_seed(5000)
    q, k, v = (torch.randn(1, 2, n, 128, generator=g, device="cuda").to(torch.float8_e4m3fn) for n in (Nq, Nk, Nk))

    def call(q, k):
        return fa.fa_fwd_fp8(q.view(torch.float8_e4m3fn), k.view(torch.float8_e4m3fn), v, 1.0, 1.0, 1.0, causal=True)

    seen = window_seen(Nq, Nk, Nk, 0, "cuda")
    base = call(q, k)
    for i in (0, Nq - 1):
        q2, bad = q.view(torch.uint8).clone(), torch.zeros(1, 2, Nq, dtype=torch.bool, device="cuda")
        q2[0, 1, i, 3], bad[0, 1, i] = 0x7F, True
        check_rows(call(q2, k), base, bad)
    for j in eights(Nk // 2):
        k2 = k.view(torch.uint8).clone()
        k2[0, 0, j, 5] = 0x7F
        check_rows(call(q, k2), base, rows_of(seen, j, 1, 2, 2, 0, 0))
