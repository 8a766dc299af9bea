"""Cases of the long-context operators: attention with a sliding window and sinks (training step, prompt
chunk, decode over a paged and a dense cache), attention of a batch whose sequences share a prefix, and
eviction from a KV cache by accumulated attention weight (the attention that accumulates the weights, and
the selection with its compaction).

``run`` computes them in a plain form (elementary torch operations in fp32, rounded once at the end), or,
where ``own`` is true, through the framework's calls.  Layouts are those of ``include/fa.h``: q, o
[B, Hq, Nq, d]; k, v [B, Hkv, Nk, d]; lse [B, Hq, Nq]; query head h reads kv head h // (Hq // Hkv).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HEADS = [(32, 8), (16, 16), (16, 4), (8, 1), (8, 8), (6, 2), (4, 4)]
DIMS = [64, 128, 128, 96, 256]


def listed():
    return [
        # one layer's attention in training: the repository's GQA shape at 8K, a 1K window and 4 sinks
        dict(name="window step 8K", op="step", type="bf16", B=1, Hq=32, Hkv=8, Nq=8192, Nk=8192, d=128, window=1024, sinks=4),
        # a small model's batch with an odd length and window
        dict(name="window step small", op="step", type="fp16", B=2, Hq=8, Hkv=8, Nq=1000, Nk=1000, d=64, window=200, sinks=1),
        # a chunk of a long prompt appended to 16K tokens (chunked prefill)
        dict(name="window chunk on 16K", op="window", type="bf16", B=1, Hq=32, Hkv=8, Nq=512, Nk=16384, d=128, window=4096, sinks=64),
        # single tokens of a large batch on a paged cache
        dict(name="window decode paged", op="paged", type="bf16", B=64, Hq=32, Hkv=8, Nq=1, Nk=8192, d=128, window=1024, sinks=4, page=64),
        # one user's single token: latency
        dict(name="window decode one", op="window", type="fp16", B=1, Hq=8, Hkv=1, Nq=1, Nk=700, d=64, window=128, sinks=4),
        # single tokens of a batch behind one long system prompt, own parts of different lengths
        dict(name="prefix decode", op="prefix", type="bf16", B=64, Hq=32, Hkv=8, Nq=1, Np=8192, Nk=512, d=128, causal=True),
        # a few users behind a short common prompt: latency
        dict(name="prefix decode few", op="prefix", type="fp16", B=4, Hq=8, Hkv=2, Nq=1, Np=500, Nk=33, d=64, causal=True),
        # several questions on one document: their tokens together, behind the document
        dict(name="prefix questions", op="prefix", type="bf16", B=8, Hq=32, Hkv=8, Nq=64, Np=4096, Nk=200, d=128, causal=True),
        # a decode step that keeps the weight each cached key has received
        dict(name="weights decode", op="weights", type="bf16", B=16, Hq=32, Hkv=8, Nq=1, Nk=8192, d=128, causal=False),
        # a prompt whose keys' weights are summed for a first eviction
        dict(name="weights prompt", op="weights", type="bf16", B=1, Hq=32, Hkv=8, Nq=4096, Nk=4096, d=128, causal=True),
        # caches cut to a quarter, the newest keys kept
        dict(name="evict 8K to 2K", op="evict", type="bf16", B=16, Hkv=8, Nk=8192, d=128, keep=2048, recent=256),
        # one small cache, odd sizes
        dict(name="evict small", op="evict", type="fp16", B=1, Hkv=2, Nk=300, d=64, keep=77, recent=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["step", "step", "window", "window", "paged", "prefix", "prefix", "weights", "weights", "evict"])
        hq, hkv = rng.choice(HEADS)
        d, kind = rng.choice(DIMS), rng.choice(["bf16", "bf16", "fp16"])
        c = dict(op=op, type=kind, B=_log(rng, 1, 64), Hq=hq, Hkv=hkv, d=d)
        if op == "step":
            c["Nq"] = c["Nk"] = _log(rng, 100, 8192)
            c["B"] = _log(rng, 1, 4)
        elif op == "window":
            c["Nq"] = rng.choice([1, 1, _log(rng, 2, 1024)])
            c["Nk"] = c["Nq"] + _log(rng, 64, 16384)
        elif op == "paged":
            c["d"] = min(d, 128)
            c["Nq"], c["page"] = 1, rng.choice([64, 128, 256])
            c["Nk"] = c["page"] * _log(rng, 2, 8192 // c["page"])
        elif op == "prefix":
            c["Nq"] = rng.choice([1, 1, 4, _log(rng, 2, 128)])
            c["Np"], c["Nk"] = _log(rng, 64, 16384), c["Nq"] + _log(rng, 1, 512)
            c["causal"] = True
        elif op == "weights":
            c["Nq"] = rng.choice([1, 1, 1, _log(rng, 32, 4096)])
            c["Nk"] = max(c["Nq"], _log(rng, 100, 16384)) if c["Nq"] == 1 else c["Nq"]
            c["causal"] = c["Nq"] > 1
        else:
            del c["Hq"]
            c["Nk"] = _log(rng, 100, 16384)
            c["keep"] = max(1, int(c["Nk"] * rng.uniform(0.05, 0.9)))
            c["recent"] = int(c["keep"] * rng.choice([0.0, 0.1, 0.5]))
        if op in ("step", "window", "paged"):
            c["window"] = _log(rng, 16, max(32, c["Nk"]))
            c["sinks"] = rng.choice([0, 1, 4, 4, 16, 100])
        # within the largest listed cases: the plain form's scores, the caches, the work
        scores = c["B"] * c.get("Hq", 0) * c.get("Nq", 0) * (c["Nk"] + c.get("Np", 0))
        cache = c["B"] * c["Hkv"] * c["Nk"] * c["d"]
        w = work(c)
        if (scores <= 2 ** (31 if op == "step" else 29) and cache <= 2 ** (29 if op == "paged" else 27)
                and w["bytes"] <= 5.4e8 and w["flops"] <= 4.5e11):
            return c


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _lens(gen, B, most, least):
    """B lengths spread evenly over [least, most], in an order that the seed gives."""
    x = torch.linspace(float(most), float(least), B, dtype=torch.float64).round().to(torch.int32).cuda()
    return x[torch.randperm(B, generator=gen, device="cuda")].contiguous()


def prepare(case, seed):
    c, gen = dict(case), torch.Generator(device="cuda").manual_seed(int(seed))
    dt, B, hkv, d, nk = TYPES[c["type"]], c["B"], c["Hkv"], c["d"], c["Nk"]
    s = dict(case=c)
    if c["op"] == "paged":
        per_seq = nk // c["page"]
        pages = B * per_seq + 3   # a few pages of other sequences among them
        s["k"] = _normal(gen, (pages, c["page"], hkv, d), dt)
        s["v"] = _normal(gen, (pages, c["page"], hkv, d), dt)
        s["table"] = torch.randperm(pages, generator=gen, device="cuda")[: B * per_seq].view(B, per_seq).to(torch.int32).contiguous()
        s["lens"] = _lens(gen, B, nk, max(1, nk // 2))
    else:
        s["k"], s["v"] = _normal(gen, (B, hkv, nk, d), dt), _normal(gen, (B, hkv, nk, d), dt)
    if "Hq" in c:
        s["q"] = _normal(gen, (B, c["Hq"], c["Nq"], d), dt)
    if c["op"] == "step":
        s["dout"] = _normal(gen, s["q"].shape, dt)
    elif c["op"] == "prefix":
        s["kp"], s["vp"] = _normal(gen, (hkv, c["Np"], d), dt), _normal(gen, (hkv, c["Np"], d), dt)
        s["lens"] = _lens(gen, B, nk, c["Nq"])
    elif c["op"] in ("weights", "evict"):
        # weights of a cache in use, a few steps' worth: a few keys hold most of them; a prompt starts from none
        u = torch.rand((B, hkv, nk), generator=gen, device="cuda")
        s["w"] = None if c.get("Nq", 1) > 1 else u.pow(8).mul(50.0 * c.get("Hq", hkv) / hkv / nk).contiguous()
    return s


# ------------------------------------------------------------------ plain forms
def _softmax(s, v):
    """Rows of scores (-inf where masked) times v, and the log-sum-exp; rows without a key give 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    return p, torch.matmul(p, v), (m + torch.log(l)).squeeze(-1)


def _positions(rows, nq, first):
    """Positions of a kv head's rows (query heads one after another, nq rows each), the first row's at `first`."""
    return torch.arange(rows, device="cuda") % nq + first


def _window_mask(pos, nk, window, sinks):
    key = torch.arange(nk, device="cuda")
    p = pos.unsqueeze(-1)
    return (key <= p) & ((key > p - window) | (key < sinks))


def _plain_window(s, k, v, first):
    c = s["case"]
    B, hkv, nq, d = c["B"], c["Hkv"], c["Nq"], c["d"]
    rows = c["Hq"] // hkv * nq
    q = s["q"].float().reshape(B, hkv, rows, d)
    k, v = k.float(), v.float()
    seen = _window_mask(_positions(rows, nq, first), k.shape[2], c["window"], c["sinks"])
    seen = seen if seen.dim() == 2 else seen.unsqueeze(1)
    sc = (torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))).masked_fill_(~seen, -math.inf)
    return (q, k, v) + _softmax(sc, v)


def _plain_step(s):
    c, shape = s["case"], s["q"].shape
    scale = 1.0 / math.sqrt(c["d"])
    q, k, v, p, o, lse = _plain_window(s, s["k"], s["v"], c["Nk"] - c["Nq"])
    do = s["dout"].float().reshape(q.shape)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    dq, dk = torch.matmul(ds, k) * scale, torch.matmul(ds.transpose(-1, -2), q) * scale
    dt = s["q"].dtype
    return dict(o=o.reshape(shape).to(dt), lse=lse.reshape(shape[:3]), dq=dq.reshape(shape).to(dt), dk=dk.to(dt), dv=dv.to(dt))


def _plain_paged(s):
    c, shape = s["case"], s["q"].shape
    t = s["table"].long()
    k = s["k"][t].reshape(c["B"], c["Nk"], c["Hkv"], c["d"]).transpose(1, 2)
    v = s["v"][t].reshape(c["B"], c["Nk"], c["Hkv"], c["d"]).transpose(1, 2)
    o, lse = _plain_window(s, k, v, s["lens"].long().unsqueeze(-1) - c["Nq"])[4:]
    return dict(o=o.reshape(shape).to(s["q"].dtype), lse=lse.reshape(shape[:3]))


def _plain_prefix(s):
    c, shape = s["case"], s["q"].shape
    B, hkv, nq, d = c["B"], c["Hkv"], c["Nq"], c["d"]
    rows = c["Hq"] // hkv * nq
    q = s["q"].float().reshape(B, hkv, rows, d)
    k, v, kp, vp = s["k"].float(), s["v"].float(), s["kp"].float(), s["vp"].float()
    scale = 1.0 / math.sqrt(d)
    sp = torch.einsum("bhrd,hnd->bhrn", q, kp) * scale
    so = torch.matmul(q, k.transpose(-1, -2)) * scale
    lens = s["lens"].long().unsqueeze(-1)
    key = torch.arange(c["Nk"], device="cuda")
    seen = (key < lens).unsqueeze(1)
    pos = _positions(rows, nq, lens - nq).unsqueeze(-1) if c["causal"] else torch.full((1, 1, 1), c["Nk"], device="cuda")
    seen = (seen & (key <= pos)).unsqueeze(1)
    seen_p = (torch.arange(c["Np"], device="cuda") <= pos + c["Np"]).unsqueeze(1)
    sp, so = sp.masked_fill_(~seen_p, -math.inf), so.masked_fill_(~seen, -math.inf)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    base = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    sp, so = torch.exp(sp - base), torch.exp(so - base)
    l = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    o = (torch.einsum("bhrn,hnd->bhrd", sp, vp) + torch.matmul(so, v)) / torch.where(l > 0, l, torch.ones_like(l))
    return dict(o=o.reshape(shape).to(s["q"].dtype), lse=(m + torch.log(l)).reshape(shape[:3]))


def _plain_weights(s):
    c, shape = s["case"], s["q"].shape
    q = s["q"].float().reshape(c["B"], c["Hkv"], -1, c["d"])
    sc = torch.matmul(q, s["k"].float().transpose(-1, -2)) * (1.0 / math.sqrt(c["d"]))
    if c["causal"]:
        pos = _positions(q.shape[2], c["Nq"], c["Nk"] - c["Nq"]).unsqueeze(-1)
        sc = sc.masked_fill_(torch.arange(c["Nk"], device="cuda") > pos, -math.inf)
    p, o, lse = _softmax(sc, s["v"].float())
    return dict(o=o.reshape(shape).to(s["q"].dtype), lse=lse.reshape(shape[:3]), weights=p.sum(-2) if s["w"] is None else s["w"] + p.sum(-2))


def _plain_evict(s):
    c, w = s["case"], s["w"]
    # the newest keys first, then the heaviest; of equal ones the first
    rank = w.clone()
    if c["recent"]:
        rank[..., c["Nk"] - c["recent"]:] = math.inf
    index = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., : c["keep"]].sort(-1).values
    rows = index.unsqueeze(-1).expand(-1, -1, -1, c["d"])
    return dict(k=torch.gather(s["k"], 2, rows), v=torch.gather(s["v"], 2, rows), weights=torch.gather(w, 2, index), index=index.to(torch.int32))


PLAIN = {
    "step": _plain_step, "paged": _plain_paged, "prefix": _plain_prefix, "weights": _plain_weights, "evict": _plain_evict,
}


def _own(s):
    import exact_attention_114_b200 as fa
    c, op = s["case"], s["case"]["op"]
    if op == "step":
        o, lse = fa.fa_fwd_window(s["q"], s["k"], s["v"], c["window"], c["sinks"])
        dq, dk, dv = fa.fa_bwd_window(s["q"], s["k"], s["v"], o, s["dout"], lse, c["window"], c["sinks"])
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    if op == "evict":
        k, v, w, index = fa.fa_kv_evict(s["k"], s["v"], s["w"], c["keep"], c["recent"])
        return dict(k=k, v=v, weights=w, index=index)
    if op == "weights":
        o, lse, w = fa.fa_fwd_weights(s["q"], s["k"], s["v"], s["w"], causal=c["causal"])
        return dict(o=o, lse=lse, weights=w)
    if op == "paged":
        o, lse = fa.fa_fwd_paged_window(s["q"], s["k"], s["v"], s["table"], s["lens"], c["window"], c["sinks"])
    elif op == "prefix":
        o, lse = fa.fa_fwd_prefix(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"], causal=c["causal"])
    else:
        o, lse = fa.fa_fwd_window(s["q"], s["k"], s["v"], c["window"], c["sinks"])
    return dict(o=o, lse=lse)


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "window":
        o, lse = _plain_window(state, state["k"], state["v"], c["Nk"] - c["Nq"])[4:]
        shape = state["q"].shape
        return dict(o=o.reshape(shape).to(state["q"].dtype), lse=lse.reshape(shape[:3]))
    return PLAIN[c["op"]](state)


# ------------------------------------------------------------------ the least work
def _window_pairs(nq, nk, window, sinks):
    """(query, key) pairs that a head's rows see, and keys that any of them sees."""
    pos = torch.arange(nq, dtype=torch.int64) + nk - nq
    lo = torch.clamp(pos - window + 1, min=0)
    own_keys = torch.clamp(pos - lo + 1, min=0)
    sink_keys = torch.clamp(torch.minimum(lo, torch.full_like(lo, sinks)), min=0) * (pos >= 0)
    first = max(0, nk - nq - window + 1)
    return int((own_keys + sink_keys).sum()), (nk - first) + min(first, sinks)


def work(case):
    c = case
    B, hq, hkv, nq, nk, d = c["B"], c.get("Hq", 0), c["Hkv"], c.get("Nq", 0), c["Nk"], c["d"]
    q_bytes, lse_bytes, row = 2 * B * hq * nq * d, 4 * B * hq * nq, 2 * d
    if c["op"] in ("step", "window"):
        pairs, keys = _window_pairs(nq, nk, c["window"], c["sinks"])
        kv = 2 * B * hkv * keys * row
        if c["op"] == "step":
            return dict(bytes=4 * q_bytes + 2 * kv + lse_bytes, flops=14 * B * hq * pairs * d)
        return dict(bytes=2 * q_bytes + kv + lse_bytes, flops=4 * B * hq * pairs * d)
    if c["op"] == "paged":
        lens = torch.linspace(float(nk), float(max(1, nk // 2)), B, dtype=torch.float64).round().to(torch.int64).tolist()
        keys = sum(_window_pairs(1, n, c["window"], c["sinks"])[1] for n in lens)
        return dict(bytes=2 * q_bytes + 2 * hkv * keys * row + lse_bytes + 4 * B * (1 + nk // c["page"]), flops=4 * hq * keys * d)
    if c["op"] == "prefix":
        lens = torch.linspace(float(nk), float(nq), B, dtype=torch.float64).round().to(torch.int64).tolist()
        pairs = sum(_window_pairs(nq, c["Np"] + n, c["Np"] + n, 0)[0] for n in lens)
        return dict(bytes=2 * q_bytes + 2 * hkv * row * (c["Np"] + sum(lens)) + lse_bytes + 4 * B, flops=4 * hq * pairs * d)
    if c["op"] == "weights":
        pairs = _window_pairs(nq, nk, nk, 0)[0] if c["causal"] else nq * nk
        return dict(bytes=2 * q_bytes + 2 * B * hkv * nk * row + lse_bytes + (4 if nq > 1 else 8) * B * hkv * nk, flops=4 * B * hq * pairs * d)
    kept = min(c["keep"], nk)
    return dict(bytes=B * hkv * (4 * nk + kept * (4 * row + 8)), flops=0)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_head(q, k, v, seen):
    """One kv head in fp64: q [rows, d], k, v [n, d], seen [rows, n]; o, lse (and p through them)."""
    sc = torch.where(seen, (q @ k.T) / math.sqrt(q.shape[-1]), -math.inf)
    lse = torch.logsumexp(sc, -1)
    p = torch.where(seen, torch.exp(sc - torch.where(torch.isinf(lse), 0.0, lse).unsqueeze(-1)), 0.0)
    return p, p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, hkv, nk, d = c["B"], c["Hkv"], c["Nk"], c["d"]
    if c["op"] == "evict":
        w = s["w"].cpu().numpy().astype(np.float64)
        newest = np.arange(nk) >= nk - c["recent"]
        at = np.empty((B, hkv, c["keep"]), np.int64)
        for b in range(B):
            for h in range(hkv):
                at[b, h] = np.sort(np.lexsort((np.arange(nk), -w[b, h], ~newest))[: c["keep"]])
        at = torch.from_numpy(at).cuda()
        pick = tuple(torch.meshgrid(torch.arange(B), torch.arange(hkv), indexing="ij"))
        pick = tuple(x.unsqueeze(-1).cuda() for x in pick) + (at,)
        return dict(k=s["k"][pick].double(), v=s["v"][pick].double(), weights=s["w"][pick].double(), index=at)
    nq = c["Nq"]
    g = c["Hq"] // hkv
    q = s["q"].double().view(B, hkv, g * nq, d)
    i = torch.arange(nq, device="cuda").repeat(g)
    out = {}
    for b in range(B):
        for h in range(hkv):
            if c["op"] == "paged":
                n = int(s["lens"][b])
                at = torch.arange(n, device="cuda")
                page = s["table"][b].long()[at // c["page"]]
                k, v = (s[x][page, at % c["page"], h].double() for x in "kv")
            elif c["op"] == "prefix":
                n = int(s["lens"][b])
                k, v = (torch.cat([s[x + "p"][h], s[x][b, h, :n]]).double() for x in "kv")
            else:
                k, v = s["k"][b, h].double(), s["v"][b, h].double()
            n = k.shape[0]
            j, pos = torch.arange(n, device="cuda")[None, :], (i + n - nq)[:, None]
            seen = j <= pos if c["op"] != "weights" or c["causal"] else j < n
            if "window" in c:
                seen = seen & ((pos - j < c["window"]) | (j < c["sinks"]))
            x = q[b, h]
            grad = c["op"] == "step"
            if grad:
                x, k, v = (t.clone().requires_grad_() for t in (x, k, v))
            p, o, lse = _exact_head(x, k, v, seen.expand(g * nq, n))
            got = dict(o=o.detach().view(g, nq, d), lse=lse.detach().view(g, nq))
            if grad:
                do = s["dout"][b].view(hkv, g * nq, d)[h].double()
                dq, got["dk"], got["dv"] = torch.autograd.grad((o * do).sum(), (x, k, v))
                got["dq"] = dq.view(g, nq, d)
            if c["op"] == "weights":
                got["weights"] = p.sum(0) + (0.0 if s["w"] is None else s["w"][b, h].double())
            for name, t in got.items():
                if name not in out:
                    lead = (B, hkv) if name in ("dk", "dv", "weights") else (B, hkv, g)
                    out[name] = torch.empty(lead + tuple(t.shape[-1:] if name == "weights" else t.shape[-2:] if name in ("dk", "dv") else t.shape[1:]), dtype=torch.float64, device="cuda")
                out[name][b, h] = t
    return {n: t if n in ("dk", "dv", "weights") else t.view((B, c["Hq"]) + tuple(t.shape[3:])) for n, t in out.items()}
