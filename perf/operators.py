"""The operators of a decode step around the weight products, as measurable cases.

A decode step with Q4_K weights alternates weight products with five other operators: `norm` closes one block and
opens the next, `append` rotates the new queries and keys and writes keys and values into a paged cache, `attn` lets
the new tokens attend to that cache (and adds up the weight that each cached token received), `evict` shrinks a cache
to a budget by that weight, and `sample` draws the next tokens from the logits.

Where `own` is false, run() computes them with elementary torch operations in 32 bits; where it is true it calls the
library.  exact() is the definition in 64 bits.  Sizes are those of the library's own decode and mixture-of-experts
workloads (hidden sizes 5120 and 2048) with generic head layouts, page sizes and vocabularies.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
ROPE_BASE = 1e6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user, a short conversation: every call is latency
        dict(name="attn_one_short", op="attn", B=1, n_q=1, Hq=40, Hkv=8, D=128, kv="bf16", page=16, lo=1000, hi=1000,
             window=0, scores=False),
        # speculative verification of 3 drafts (the library's M = 4 workload) for 16 ragged sequences, small pages
        dict(name="attn_verify_ragged", op="attn", B=16, n_q=4, Hq=32, Hkv=4, D=128, kv="bf16", page=16, lo=33,
             hi=6001, window=0, scores=False),
        # one very long document in an 8-bit cache: the whole GPU has to share one sequence
        dict(name="attn_long_e4m3", op="attn", B=1, n_q=1, Hq=40, Hkv=8, D=128, kv="e4m3", page=64, lo=200001,
             hi=200001, window=0, scores=False),
        # a full serving batch that keeps the accumulated weights for a later eviction: the largest call
        dict(name="attn_batch_weights", op="attn", B=64, n_q=1, Hq=40, Hkv=8, D=128, kv="bf16", page=32, lo=2000,
             hi=8192, window=0, scores=True),
        # steady state of a cache at its budget: one token more per step, one token less
        dict(name="evict_one", op="evict", B=32, Hkv=8, D=128, kv="bf16", page=16, lo=2049, hi=2049, budget=2048,
             sinks=4, recent=256),
        # a batch of long prompts cut to half, ragged
        dict(name="evict_half", op="evict", B=16, Hkv=8, D=128, kv="bf16", page=64, lo=9001, hi=16384, budget=8192,
             sinks=4, recent=1024),
        # one new token for each of 16 sequences
        dict(name="append_decode", op="append", B=16, T=16, Hq=40, Hkv=8, D=128, kv="bf16", page=16, rot=128,
             half=True, meta=True),
        # the prompts of 5 sequences (8191 tokens together) going into an 8-bit cache, rotary pairs interleaved
        dict(name="append_prompt_e4m3", op="append", B=5, T=8191, Hq=32, Hkv=4, D=128, kv="e4m3", page=64, rot=64,
             half=False, meta=False),
        # one token between two blocks, norms on both sides of the residual
        dict(name="norm_one", op="norm", M=1, D=5120, post="rms", pre="rms", gate="none", res="fp32"),
        # a prefill chunk with a per-channel gate and a 16-bit residual stream
        dict(name="norm_prompt", op="norm", M=4096, D=5120, post="rms", pre="rms", gate="channel", res="bf16"),
        # one user with the usual chat settings
        dict(name="sample_one", op="sample", M=1, V=128001, t=0.7, k=50, p=0.9, m=0.0),
        # a serving batch, every row with its own settings around these, no top-k
        dict(name="sample_batch", op="sample", M=256, V=151936, t=1.0, k=0, p=0.95, m=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "evict", "append", "norm", "sample"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128, 256])
    kv = rng.choice(["bf16", "e4m3"])
    page = rng.choice([1, 16, 24, 32, 64, 128])
    group = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "attn":
        n_q = rng.choice([1, 1, 1, 2, 4, 7])
        hi = _log(rng, 1, 200001)
        lo = max(1, int(hi * rng.choice([1.0, 0.5, 0.03])))
        most = max(1, int(64 * 5000 * 8 * 128 / (hi * Hkv * D)))  # cached values of the largest listed case
        most = max(1, min(most, int(64 * 5000 * 40 * 128 / (hi * Hkv * group * n_q * D))))  # and its products
        return dict(op=op, B=_log(rng, 1, min(128, most)), n_q=n_q, Hq=Hkv * group, Hkv=Hkv, D=D, kv=kv, page=page,
                    lo=lo, hi=hi, window=rng.choice([0, 0, 0, 1000]), scores=rng.random() < 0.3)
    if op == "evict":
        hi = _log(rng, 20, 32768)
        most = max(1, int(16 * 12000 * 8 * 128 / (hi * Hkv * D)))
        budget = max(8, min(hi - 1, int(hi * rng.uniform(0.3, 1.0))))
        return dict(op=op, B=_log(rng, 1, min(64, most)), Hkv=Hkv, D=D, kv=kv, page=page, lo=max(1, hi // 2), hi=hi,
                    budget=budget, sinks=rng.choice([0, 4]), recent=budget // 8)
    if op == "append":
        T = min(_log(rng, 1, 8191), max(1, int(8191 * 40 * 128 / ((group + 2) * Hkv * D))))
        return dict(op=op, B=_log(rng, 1, min(64, T)), T=T, Hq=Hkv * group, Hkv=Hkv, D=D, kv=kv, page=page,
                    rot=rng.choice([D, D // 2, 0]), half=rng.random() < 0.7, meta=rng.random() < 0.5)
    if op == "norm":
        width = rng.choice([2048, 5120, 768, _log(rng, 64, 16384)])
        width = width if width != 3072 else 3073
        return dict(op=op, M=_log(rng, 1, max(1, min(8192, 4096 * 5120 // width))), D=width,
                    post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "channel", "token"]), res=rng.choice(["fp32", "bf16"]))
    V = _log(rng, 1000, 200000)
    return dict(op=op, M=_log(rng, 1, max(1, min(256, 256 * 151936 // V))), V=V,
                t=round(rng.uniform(0.3, 1.3), 3), k=rng.choice([0, 1, 20, 50, 400]),
                p=rng.choice([1.0, 0.95, 0.9, 0.5]), m=rng.choice([0.0, 0.0, 0.02, 0.1]))


def _lens(c):
    """The batch's lengths, spread evenly over [lo, hi]."""
    if c["B"] == 1:
        return [c["hi"]]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // (c["B"] - 1) for i in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "norm":
        r = 4 if c["res"] == "fp32" else 2
        gate = {"none": 0, "channel": 4 * c["D"], "token": 4 * c["M"] * c["D"]}[c["gate"]]
        return {"bytes": c["M"] * c["D"] * (4 + 2 * r + 2) + gate, "flops": 10 * c["M"] * c["D"]}
    if c["op"] == "sample":
        return {"bytes": 4 * c["M"] * c["V"] + 28 * c["M"], "flops": 20 * c["M"] * c["V"]}
    e = 2 if c["kv"] == "bf16" else 1
    row = c["Hkv"] * c["D"]
    if c["op"] == "append":
        q = c["Hq"] * c["D"]
        return {"bytes": c["T"] * (4 * (q + 2 * row) + 2 * q + 2 * row * e + 4 * c["rot"]),
                "flops": 3 * c["T"] * (q + row)}
    lens = _lens(c)
    if c["op"] == "evict":
        # every score and position is read and the kept ones written; a mover's key and value are read and written
        moved = sum(max(0, min(c["budget"], n - c["budget"])) * (c["budget"] / n) for n in lens)
        kept = sum(min(n, c["budget"]) for n in lens)
        return {"bytes": int(8 * c["Hkv"] * (sum(lens) + kept) + moved * row * e * 4), "flops": 0}
    seen = [min(n, c["window"] + c["n_q"] - 1) if c["window"] else n for n in lens]
    b = sum(seen) * row * 2 * e + c["B"] * c["n_q"] * c["Hq"] * c["D"] * 4
    if c["scores"]:
        b += 8 * c["Hkv"] * sum(seen)
    return {"bytes": b, "flops": 4 * sum(seen) * c["Hq"] * c["n_q"] * c["D"]}


# ---------------------------------------------------------------- what a program has in hand

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pool(c, g, pages):
    """A pool of pages, [page][head][slot][D], filled with keys or values."""
    shape = (pages, c["Hkv"], c["page"], c["D"])
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    return x.to(torch.float8_e4m3fn) if c["kv"] == "e4m3" else x


def _cache(c, g, longest):
    """Page pools and a page table whose pages lie scattered in the pools."""
    per = -(-longest // c["page"])
    pages = c["B"] * per + 3
    table = torch.randperm(pages, generator=g, device=DEV)[:c["B"] * per].to(torch.int32).view(c["B"], per)
    return dict(k=_pool(c, g, pages), v=_pool(c, g, pages), table=table, k_scale=0.5 if c["kv"] == "e4m3" else 1.0,
                v_scale=0.25 if c["kv"] == "e4m3" else 1.0)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c=c)
    randn = lambda *n: torch.randn(n, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "norm":
        M, D = c["M"], c["D"]
        s["y"] = randn(M, D) * 3
        s["r"] = (randn(M, D) * 2).to(torch.float32 if c["res"] == "fp32" else torch.bfloat16)
        s["post_w"], s["pre_w"] = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
        s["post_b"] = 0.1 * randn(D) if c["post"] == "layer" else None
        s["pre_b"] = 0.1 * randn(D) if c["pre"] == "layer" else None
        s["gate"] = {"none": None, "channel": 0.5 + 0.3 * randn(1, D),
                     "token": 0.5 + 0.3 * randn(M, D) if c["gate"] == "token" else None}[c["gate"]]
        s["scale"], s["eps"] = 0.7, 1e-6
        s["r_out"] = torch.zeros_like(s["r"])
        s["x"] = torch.zeros(M, D, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "sample":
        M, V = c["M"], c["V"]
        # logits of a language model: a broad bulk and, in each row, a few dozen candidates that stand out
        z = randn(M, V) * 2.2
        z.scatter_add_(1, torch.randint(0, V, (M, 24), generator=g, device=DEV), 4 + 3 * randn(M, 24).abs())
        s["logits"] = z
        one = torch.ones(M, device=DEV)
        vary = torch.rand(M, generator=g, device=DEV) if M > 1 else 0.5 * one
        s["t"] = c["t"] * (0.8 + 0.4 * vary)
        s["k"] = (c["k"] * one).to(torch.int32)
        s["p"] = torch.where(one * c["p"] < 1, c["p"] - 0.05 * vary, one)
        s["m"] = c["m"] * one
        s["u"] = torch.rand(M, generator=g, device=DEV)
        s["token"] = torch.zeros(M, dtype=torch.int32, device=DEV)
        s["prob"] = torch.zeros(M, device=DEV)
    elif c["op"] == "append":
        T, B, Hq, Hkv, D = c["T"], c["B"], c["Hq"], c["Hkv"], c["D"]
        per = [T // B + (i < T % B) for i in range(B)]
        before = 100 if T > B else 777  # what each sequence holds already
        s["cache"] = _cache(c, g, before + max(per))
        # one product made q, k and v of every token side by side
        s["qkv"] = randn(T, (Hq + 2 * Hkv) * D)
        s["seq"] = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(per, device=DEV)).to(torch.int32)
        s["slot"] = torch.cat([torch.arange(before, before + n, device=DEV) for n in per]).to(torch.int32)
        s["pos"] = s["slot"] + 1000  # some of the sequence was evicted before
        half = c["rot"] // 2
        s["rope"] = None
        if half:
            f = ROPE_BASE ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
            a = torch.arange(int(s["pos"].max()) + 1, device=DEV, dtype=torch.float64)[:, None] * f
            s["rope"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        s["q"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["weight"] = s["where"] = None
        if c["meta"]:
            n = s["cache"]["table"].shape[1] * c["page"]
            s["weight"] = randn(B, Hkv, n).abs()
            s["where"] = torch.arange(n, device=DEV, dtype=torch.int32).expand(B, Hkv, n).contiguous()
    elif c["op"] == "evict":
        B, Hkv = c["B"], c["Hkv"]
        s["cache"] = _cache(c, g, c["hi"])
        n = s["cache"]["table"].shape[1] * c["page"]
        perm = torch.randperm(B, generator=g, device=DEV)
        s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)[perm]
        # accumulated weights are heavy-tailed; equal ones (tokens that nothing looked at) are common
        w = torch.exp(2 * randn(B, Hkv, n))
        s["weight"] = torch.where(torch.rand(B, Hkv, n, generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
        # an earlier eviction left the slots of each head out of order
        gap = torch.randint(1, 3, (B, Hkv, n), generator=g, device=DEV)
        where = torch.cumsum(gap, -1) - 1
        swap = torch.arange(n, device=DEV)
        m = min(n, c["lo"]) // 2
        swap[:m] = torch.randperm(m, generator=g, device=DEV)
        s["where"] = where[:, :, swap].to(torch.int32).contiguous()
        s["new_lens"] = torch.zeros_like(s["lens"])
        s["weight_out"], s["where_out"] = torch.zeros_like(s["weight"]), torch.zeros_like(s["where"])
    else:
        B, n_q, Hq, D = c["B"], c["n_q"], c["Hq"], c["D"]
        s["cache"] = _cache(c, g, c["hi"])
        perm = torch.randperm(B, generator=g, device=DEV)
        s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)[perm]
        # logits of a few units: some tokens stand out, none takes all
        s["q"] = (randn(B, n_q, Hq, D) * (2.0 / s["cache"]["k_scale"])).to(torch.bfloat16)
        s["scale"], s["decay"] = D ** -0.5, 0.98
        s["o"] = torch.zeros(B, n_q, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["weight"] = randn(B, c["Hkv"], s["cache"]["table"].shape[1] * c["page"]).abs() if c["scores"] else None
    return s


def run(state):
    op = state["c"]["op"]
    return (_own if own else _plain)[op](state)


# ---------------------------------------------------------------- plain forms

def _norm(x, kind, w, b, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return x if b is None else x + b


def _plain_norm(s):
    c = s["c"]
    y = _norm(s["y"], c["post"], s["post_w"], s["post_b"], s["eps"])
    if s["gate"] is not None:
        y = y * s["gate"]
    h = s["r"].float() + s["scale"] * y
    s["r_out"].copy_(h)
    s["x"].copy_(_norm(h, c["pre"], s["pre_w"], s["pre_b"], s["eps"]))
    return {"r": s["r_out"], "x": s["x"]}


# 2^-f = 2^-1/2 2^-(f - 1/2): the series of the exponential around the middle of [0, 1)
_POLY = [float(np.float32(2 ** -0.5 * (-math.log(2)) ** i / math.factorial(i))) for i in range(8)]
_LOG2E = float(np.float32(1 / math.log(2)))
ONE = 1 << 24


def _weights(z, top, t):
    """Integer weights of the logits, 2^40 for the largest: floor(2^(40 - (top - z) / (t ln 2))) to 24 bits."""
    d = torch.where(z == top, torch.zeros_like(z), top - z) * ((1.0 / t) * _LOG2E)
    fine = d < 41
    d = torch.where(fine, d, torch.zeros_like(d))
    n = torch.floor(d)
    f = d - n - 0.5
    p = torch.full_like(f, _POLY[7])
    p = p * f + _POLY[6]
    p = p * f + _POLY[5]
    p = p * f + _POLY[4]
    p = p * f + _POLY[3]
    p = p * f + _POLY[2]
    p = p * f + _POLY[1]
    p = p * f + _POLY[0]
    w = ((p * 16777216.0).to(torch.int64) << 16) >> n.to(torch.int64)
    return torch.where(fine, w, torch.zeros_like(w))


def _part(total, share):
    """floor(total * share / 2^24) in 64 bits."""
    return (total >> 24) * share + (((total & (ONE - 1)) * share) >> 24)


def _plain_sample(s):
    z = torch.where(torch.isnan(s["logits"]), torch.full_like(s["logits"], -math.inf), s["logits"])
    V = z.shape[1]
    z, index = torch.sort(z, dim=1, descending=True, stable=True)
    top = z[:, :1]
    t = s["t"][:, None]
    greedy = ~(t > 0)
    w = _weights(z, top, torch.where(greedy, torch.ones_like(t), t))
    rank = torch.arange(V, device=z.device)
    k = s["k"].to(torch.int64)[:, None]
    w = torch.where((k <= 0) | (rank < k), w, torch.zeros_like(w))
    before = torch.cumsum(w, 1) - w
    share = (s["p"].clamp(0, 1) * 16777216.0).to(torch.int64)[:, None]
    least = (s["m"].clamp(0, 1) * 16777216.0).to(torch.int64)[:, None]
    nucleus = (share >= ONE) | (rank == 0) | (before < _part(w.sum(1, keepdim=True), share))
    keep = nucleus & (w >= _part(w[:, :1], least))
    keep = torch.where(greedy, rank == 0, keep)
    w = torch.where(keep, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, index, w)
    total = w.sum(1, keepdim=True)
    u = (s["u"].clamp(0, 1) * 16777216.0).to(torch.int64).clamp(max=ONE - 1)[:, None]
    token = (torch.cumsum(w, 1) <= _part(total, u)).sum(1)
    none = torch.isneginf(top[:, 0])
    at = token.clamp(max=V - 1)[:, None]
    s["prob"].copy_(torch.where(none, torch.zeros_like(top[:, 0]), (torch.gather(w, 1, at).float() / total.float())[:, 0]))
    s["token"].copy_(torch.where(none, torch.full_like(token, -1), token))
    return {"token": s["token"], "prob": s["prob"]}


def _rotate(x, table, half):
    """x [T][H][D] with its first 2 * (table width / 2) values rotated."""
    if table is None:
        return x
    n = table.shape[1] // 2
    cos, sin = table[:, None, :n], table[:, None, n:]
    if half:
        a, b = x[..., :n], x[..., n:2 * n]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, x[..., 2 * n:]], -1)


def _bytes(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def _stored(x, scale, pool):
    x = x * (1.0 / scale)
    return x.clamp(-448, 448).to(pool.dtype).view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else x.to(pool.dtype)


def _plain_append(s):
    c, a = s["c"], s["cache"]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    q, k, v = (x.view(T, -1, D) for x in s["qkv"].split([Hq * D, Hkv * D, Hkv * D], 1))
    pos = s["pos"].long()
    table = None if s["rope"] is None else s["rope"][pos]
    s["q"].copy_(_rotate(q, table, c["half"]))
    seq, slot = s["seq"].long(), s["slot"].long()
    page = a["table"][seq, slot // c["page"]].long()
    _bytes(a["k"])[page, :, slot % c["page"]] = _stored(_rotate(k, table, c["half"]), a["k_scale"], a["k"])
    _bytes(a["v"])[page, :, slot % c["page"]] = _stored(v, a["v_scale"], a["v"])
    out = {"q": s["q"], "k": a["k"], "v": a["v"]}
    if c["meta"]:
        s["weight"][seq, :, slot] = 0.0
        s["where"][seq, :, slot] = s["pos"][:, None].expand(T, Hkv)
        out |= {"weight": s["weight"], "where": s["where"]}
    return out


def _plain_evict(s):
    c, a = s["c"], s["cache"]
    n = s["weight"].shape[2]
    at = torch.arange(n, device=DEV)
    lens = s["lens"][:, None, None]
    new = lens.clamp(max=c["budget"])
    there = at < lens
    newest = torch.where(there, s["where"], torch.full_like(s["where"], -1)).amax(2, keepdim=True)
    held = (s["where"] < c["sinks"]) | (s["where"] > newest - c["recent"])
    # the lightest first, equal ones by slot; then what is not protected, what is, and what is not there
    order = torch.sort(s["weight"], dim=2, stable=True).indices
    kind = torch.gather(torch.where(there, held.to(torch.int8), torch.full_like(held, 2, dtype=torch.int8)), 2, order)
    order = torch.gather(order, 2, torch.sort(kind, dim=2, stable=True).indices)
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order))
    gone = there & (rank < lens - new)
    hole, mover = (gone & (at < new)).nonzero(), (there & ~gone & (at >= new)).nonzero()
    b, h, to = hole.unbind(1)
    src = mover[:, 2]
    page_to, page_src = a["table"][b, to // c["page"]].long(), a["table"][b, src // c["page"]].long()
    for pool in (_bytes(a["k"]), _bytes(a["v"])):
        pool[page_to, h, to % c["page"]] = pool[page_src, h, src % c["page"]]
    for x, y in ((s["weight"], s["weight_out"]), (s["where"], s["where_out"])):
        torch.where(at < new, x, y, out=y)
        y[b, h, to] = x[b, h, src]
    s["new_lens"].copy_(new[:, 0, 0])
    return {"k": a["k"], "v": a["v"], "weight": s["weight_out"], "where": s["where_out"], "lens": s["new_lens"]}


def _plain_attn(s):
    c, a = s["c"], s["cache"]
    B, n_q, Hq, Hkv, D = c["B"], c["n_q"], c["Hq"], c["Hkv"], c["D"]
    k = a["k"][a["table"].long()] if c["kv"] == "bf16" else _bytes(a["k"])[a["table"].long()].view(a["k"].dtype)
    v = a["v"][a["table"].long()] if c["kv"] == "bf16" else _bytes(a["v"])[a["table"].long()].view(a["v"].dtype)
    k, v = (x.float().transpose(1, 2).reshape(B, Hkv, -1, D) for x in (k, v))
    q = s["q"].float().view(B, n_q, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    z = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, n_q, Hq // Hkv, -1) * (s["scale"] * a["k_scale"])
    at = torch.arange(k.shape[2], device=DEV)
    end = s["lens"][:, None] - n_q + 1 + torch.arange(n_q, device=DEV)
    seen = at < end[:, :, None]
    if c["window"]:
        seen = seen & (at >= end[:, :, None] - c["window"])
    seen = seen[:, None, :, None]
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    top = z.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(z - top), torch.zeros_like(z))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    o = torch.matmul(p.view(B, Hkv, -1, k.shape[2]), v) * a["v_scale"]
    s["o"].copy_(o.view(B, Hkv, n_q, -1, D).permute(0, 2, 1, 3, 4).reshape(B, n_q, Hq, D))
    if not c["scores"]:
        return {"o": s["o"]}
    there = at < s["lens"][:, None, None]
    s["weight"].copy_(torch.where(there, s["weight"] * s["decay"] + p.sum((2, 3)), s["weight"]))
    return {"o": s["o"], "weight": s["weight"]}


_plain = {"norm": _plain_norm, "sample": _plain_sample, "append": _plain_append, "evict": _plain_evict,
          "attn": _plain_attn}


# ---------------------------------------------------------------- the library's calls

def _handle(s):
    """The cache's descriptor: a program makes it once, beside the pools."""
    import q4_weight_quantized_gb300 as q4k
    if "handle" not in s:
        a = s["cache"]
        s["handle"] = q4k.kv_cache(a["k"], a["v"], a["table"], k_scale=a["k_scale"], v_scale=a["v_scale"])
    return s["handle"]


def _workspace(s, size):
    if "ws" not in s:
        s["ws_bytes"] = size()
        s["ws"] = torch.empty(max(1, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return s["ws"], s["ws_bytes"]


def _own_norm(s):
    import q4_weight_quantized_gb300 as q4k
    c = s["c"]
    kind = {"none": q4k.Q4K_NORM_NONE, "rms": q4k.Q4K_NORM_RMS, "layer": q4k.Q4K_NORM_LAYER}
    M, D = c["M"], c["D"]
    q4k.q4k_norm_residual(M, D, s["y"], D, kind[c["post"]], s["post_w"], s["post_b"], s["eps"], s["gate"],
                          D if c["gate"] == "token" else 0, s["scale"], s["r"], s["r_out"], D,
                          q4k.Q4K_RES_FP32 if c["res"] == "fp32" else q4k.Q4K_RES_BF16, kind[c["pre"]], s["pre_w"],
                          s["pre_b"], s["eps"], s["x"], D)
    return {"r": s["r_out"], "x": s["x"]}


def _own_sample(s):
    import q4_weight_quantized_gb300 as q4k
    c = s["c"]
    q4k.q4k_sample(s["logits"], c["M"], c["V"], c["V"], s["t"], s["k"], s["p"], s["m"], s["u"], s["token"], s["prob"])
    return {"token": s["token"], "prob": s["prob"]}


def _own_append(s):
    import q4_weight_quantized_gb300 as q4k
    c, a = s["c"], s["cache"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    ld, base = (Hq + 2 * Hkv) * D, s["qkv"].data_ptr()
    q4k.q4k_kv_append(_handle(s), c["T"], Hq, base, ld, base + 4 * Hq * D, ld, base + 4 * (Hq + Hkv) * D, ld, s["seq"],
                      s["slot"], s["pos"], s["rope"], 0 if s["rope"] is None else s["rope"].shape[0], c["rot"],
                      q4k.Q4K_ROPE_HALF if c["half"] else q4k.Q4K_ROPE_PAIRS, s["q"], Hq * D, s["weight"], s["where"],
                      s["weight"].shape[2] if c["meta"] else 0)
    out = {"q": s["q"], "k": a["k"], "v": a["v"]}
    return out | {"weight": s["weight"], "where": s["where"]} if c["meta"] else out


def _own_evict(s):
    import q4_weight_quantized_gb300 as q4k
    c, a, n = s["c"], s["cache"], s["weight"].shape[2]
    cache = _handle(s)
    ws, size = _workspace(s, lambda: q4k.q4k_kv_evict_workspace_size(cache, n))
    q4k.q4k_kv_evict(cache, s["lens"], s["new_lens"], c["budget"], c["sinks"], c["recent"], s["weight"], s["where"],
                     s["weight_out"], s["where_out"], n, ws, size)
    return {"k": a["k"], "v": a["v"], "weight": s["weight_out"], "where": s["where_out"], "lens": s["new_lens"]}


def _own_attn(s):
    import q4_weight_quantized_gb300 as q4k
    c = s["c"]
    cache, ld = _handle(s), c["Hq"] * c["D"]
    n = s["weight"].shape[2] if c["scores"] else 0
    ws, size = _workspace(s, lambda: q4k.q4k_attn_decode_workspace_size(cache, c["Hq"], c["n_q"], n))
    q4k.q4k_attn_decode(cache, s["lens"], s["q"], ld, c["Hq"], c["n_q"], s["scale"], 0.0, c["window"], s["o"], ld,
                        s["weight"], n, s["decay"], ws, size)
    return {"o": s["o"], "weight": s["weight"]} if c["scores"] else {"o": s["o"]}


_own = {"norm": _own_norm, "sample": _own_sample, "append": _own_append, "evict": _own_evict, "attn": _own_attn}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "sample": _exact_sample, "append": _exact_append, "evict": _exact_evict,
                "attn": _exact_attn}[case["op"]](case, s)


def _exact_norm(c, s):
    def norm(x, kind, w, b):
        if kind == "none":
            return x
        m = x.mean(1, keepdim=True) if kind == "layer" else 0.0
        out = (x - m) * ((x - m).pow(2).mean(1, keepdim=True) + s["eps"]).rsqrt() * w.double()
        return out + b.double() if b is not None else out
    h = norm(s["y"].double(), c["post"], s["post_w"], s["post_b"])
    h = s["r"].double() + s["scale"] * h * (1.0 if s["gate"] is None else s["gate"].double())
    return {"r": h, "x": norm(h, c["pre"], s["pre_w"], s["pre_b"])}


def _exact_sample(c, s):
    """Row by row on the host: 32-bit weights as the definition has them, sums in whole numbers."""
    logits, f = s["logits"].cpu().numpy(), np.float32
    t, p, m, u = (s[n].cpu().numpy() for n in "tpmu")
    k = s["k"].cpu().numpy()
    token, prob = np.zeros(c["M"], np.int32), np.zeros(c["M"])
    for i in range(c["M"]):
        z = logits[i]
        top = z.max()
        d = (top - z) * (f(1) / f(t[i]) * f(_LOG2E))
        near = np.flatnonzero(d < 41)
        n = np.floor(d[near])
        x = d[near] - n - f(0.5)
        y = np.full_like(x, f(_POLY[7]))
        for a in reversed(_POLY[:7]):
            y = y * x + f(a)
        w = (np.rint(y.astype(np.float64) * 2 ** 24).astype(np.int64) << 16) >> n.astype(np.int64)
        order = np.lexsort((near, -z[near]))
        if k[i] > 0:
            order = order[:k[i]]
        ws = w[order]
        cut = lambda total, share: int(total) * int(np.floor(float(share) * 2 ** 24)) >> 24  # noqa: E731
        keep = ws >= cut(ws[0], m[i])
        if p[i] < 1:
            before = np.concatenate([[0], np.cumsum(ws)[:-1]])
            keep &= (before < cut(ws.sum(), p[i])) | (np.arange(len(ws)) == 0)
        ids = np.sort(near[order[keep]])
        wi = w[np.searchsorted(near, ids)]
        j = int(np.searchsorted(np.cumsum(wi), cut(wi.sum(), u[i]), side="right"))
        token[i], prob[i] = ids[j], wi[j] / wi.sum()
    return {"token": token, "prob": prob}


def _exact_append(c, s):
    a, T, D = s["cache"], c["T"], c["D"]
    x = s["qkv"].double().view(T, c["Hq"] + 2 * c["Hkv"], D)
    n, turn = c["rot"] // 2, c["Hq"] + c["Hkv"]
    if n:
        i = torch.arange(n, device=DEV)
        first, second = (i, i + n) if c["half"] else (2 * i, 2 * i + 1)
        e = torch.complex(x[:, :turn, first], x[:, :turn, second])
        r = s["rope"].double()[s["pos"].long()]
        e = e * torch.complex(r[:, :n], r[:, n:])[:, None]
        x[:, :turn, first], x[:, :turn, second] = e.real, e.imag
    pools = {}
    for name, part in (("k", x[:, c["Hq"]:turn]), ("v", x[:, turn:])):
        pool = a[name].double()
        part = part / a[name + "_scale"]
        for b in range(c["B"]):
            mine = (s["seq"] == b).nonzero()[:, 0]
            slot = s["slot"][mine].long()
            pool[a["table"][b][slot // c["page"]].long(), :, slot % c["page"]] = part[mine]
        pools[name] = pool
    out = {"q": x[:, :c["Hq"]], **pools}
    if c["meta"]:
        out |= {"weight": s["weight"].double(), "where": None}
        for b in range(c["B"]):
            out["weight"][b][:, s["slot"][s["seq"] == b].long()] = 0.0
    return out


def _exact_evict(c, s):
    """Sequence by sequence and head by head on the host."""
    a, size = s["cache"], c["page"]
    weight, where, lens = (s[n].cpu().numpy() for n in ("weight", "where", "lens"))
    out_w, out_p = np.zeros(weight.shape), np.zeros(where.shape, np.int32)
    moves = []
    for b in range(c["B"]):
        n, new = int(lens[b]), min(int(lens[b]), c["budget"])
        for h in range(c["Hkv"]):
            w, p = weight[b, h, :n], where[b, h, :n]
            safe = (p < c["sinks"]) | (p > p.max() - c["recent"])
            gone = np.zeros(n, bool)
            gone[np.lexsort((np.arange(n), w, safe))[:n - new]] = True
            src = np.flatnonzero(~gone[new:]) + new
            to = np.flatnonzero(gone[:new])
            take = np.arange(new)
            take[to] = src
            out_w[b, h, :new], out_p[b, h, :new] = w[take], p[take]
            moves.append(np.stack([np.full_like(to, b), np.full_like(to, h), to, src], 1))
    b, h, to, src = torch.from_numpy(np.concatenate(moves)).to(DEV).unbind(1)
    pools = {}
    for name in "kv":
        pool = a[name].double() if c["kv"] == "e4m3" else a[name].clone()
        pool[a["table"][b, to // size].long(), h, to % size] = pool[a["table"][b, src // size].long(), h, src % size]
        pools[name] = pool.double()
    return {**pools, "weight": out_w, "where": out_p, "lens": np.minimum(lens, c["budget"])}


def _exact_attn(c, s):
    a, G = s["cache"], c["Hq"] // c["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    weight = s["weight"].double() if c["scores"] else None
    for b in range(c["B"]):
        n = int(s["lens"][b])
        if weight is not None:
            weight[b, :, :n] *= s["decay"]
        pages = a["table"][b].long()
        for h in range(c["Hkv"]):
            k, v = (a[x][:, h][pages] if c["kv"] == "bf16" else _bytes(a[x])[:, h][pages].view(a[x].dtype) for x in "kv")
            k, v = k.double().flatten(0, 1) * a["k_scale"], v.double().flatten(0, 1) * a["v_scale"]
            for j in range(c["n_q"]):
                end = n - c["n_q"] + 1 + j
                begin = max(0, end - c["window"]) if c["window"] else 0
                if end <= begin:
                    continue
                x = s["q"][b, j, h * G:(h + 1) * G].double()
                p = torch.softmax(x @ k[begin:end].T * s["scale"], -1)
                o[b, j, h * G:(h + 1) * G] = p @ v[begin:end]
                if weight is not None:
                    weight[b, h, begin:end] += p.sum(0)
    return {"o": o, "weight": weight} if c["scores"] else {"o": o}
