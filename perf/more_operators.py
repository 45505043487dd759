"""The operators of a step that mixes prompts and decode tokens of many requests, as measurable cases.

Such a step needs, beside the weight products and the operators of a decode step: `plan`, which gives every request its
pages and every new token its slot; `norm8`, the norm between two blocks with its output in 8 bits for the next product;
`lora`, the low-rank adapters of the requests beside a shared projection; and `attn`, the attention of ragged chunks of
new tokens over the paged cache.

Where `own` is false, run() computes them with elementary torch operations in 32 bits (whole numbers in 64); where it is
true it calls the library.  exact() is the definition in 64 bits.  Sizes are those of the library's own decode and
mixture-of-experts workloads (hidden sizes 5120 and 2048, 17408 between them) with generic head layouts, page sizes,
ranks and batches.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 requests: a token each, every sixteenth opens a page, two requests have ended
        dict(name="plan_decode", op="plan", B=64, lo=1, hi=1, page=16, old=4000, over=2, surplus=0, short=False),
        # prompts arrive for 256 slots of a server, others give pages back after an eviction
        dict(name="plan_prompts", op="plan", B=256, lo=0, hi=509, page=16, old=2000, over=20, surplus=9, short=False),
        # one token between two blocks, the next product taking 8-bit activations
        dict(name="norm8_one", op="norm8", M=1, D=5120, post="none", pre="rms", gate="none", res="fp32"),
        # a prefill chunk with norms on both sides of a 16-bit residual stream
        dict(name="norm8_prompt", op="norm8", M=4096, D=5120, post="rms", pre="rms", gate="none", res="bf16"),
        # a decode batch in which most requests bring their own small adapter
        dict(name="lora_decode", op="lora", T=32, K=5120, N=5120, R=16, nA=24, ragged=False, none=0.2, runs=1),
        # speculative verification, 4 tokens a request, adapters of different ranks
        dict(name="lora_verify", op="lora", T=64, K=5120, N=17408, R=64, nA=16, ragged=True, none=0.1, runs=4),
        # prompts of a few tenants going through the up projection
        dict(name="lora_prompt", op="lora", T=4096, K=5120, N=17408, R=16, nA=4, ragged=False, none=0.0, runs=512),
        # a short question into an empty cache: latency
        dict(name="attn_short", op="attn", ones=0, B=1, n_lo=33, n_hi=33, c_lo=0, c_hi=0, Hq=40, Hkv=8, D=128, kv="bf16",
             page=16, window=0, cap=0.0),
        # a whole prompt at once
        dict(name="attn_prompt", op="attn", ones=0, B=1, n_lo=8192, n_hi=8192, c_lo=0, c_hi=0, Hq=40, Hkv=8, D=128,
             kv="bf16", page=16, window=0, cap=0.0),
        # a chunk of a very long prompt, most of it in an 8-bit cache already
        dict(name="attn_chunk_e4m3", op="attn", ones=0, B=1, n_lo=512, n_hi=512, c_lo=65536, c_hi=65536, Hq=40, Hkv=8,
             D=128, kv="e4m3", page=64, window=0, cap=0.0),
        # a mixed step: 20 requests decode a token each while chunks of 4 prompts run beside them
        dict(name="attn_mixed", op="attn", ones=20, B=24, n_lo=301, n_hi=512, c_lo=100, c_hi=3001, Hq=32, Hkv=4, D=128,
             kv="bf16", page=32, window=0, cap=0.0),
        # ragged prompts of a model with small heads and a sliding window
        dict(name="attn_window", op="attn", ones=0, B=6, n_lo=999, n_hi=4001, c_lo=0, c_hi=500, Hq=32, Hkv=8, D=64,
             kv="bf16", page=24, window=1024, cap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["plan", "norm8", "lora", "lora", "attn", "attn", "attn"])
    if op == "plan":
        B = _log(rng, 1, 4096)
        hi = _log(rng, 1, max(1, min(8192, 131072 // B)))
        return dict(op=op, B=B, lo=rng.choice([0, 1, hi]), hi=hi, page=rng.choice([1, 16, 24, 32, 64, 128]),
                    old=_log(rng, 1, max(1, min(65536, 512000 // B))), over=int(B * rng.choice([0.0, 0.1])),
                    surplus=rng.choice([0, 0, 5]), short=rng.random() < 0.3)
    if op == "norm8":
        D = rng.choice([2048, 5120, 768, 32 * _log(rng, 2, 512)])
        return dict(op=op, M=_log(rng, 1, max(1, min(8192, 4096 * 5120 // D))), D=D,
                    post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "channel", "token"]), res=rng.choice(["fp32", "bf16"]))
    if op == "lora":
        K, N = rng.choice([2048, 5120, 768, 17408, 8 * _log(rng, 8, 2000)]), rng.choice([2048, 5120, 17408, _log(rng, 50, 17408)])
        R, nA = rng.choice([8, 16, 16, 32, 64, 128]), _log(rng, 1, 48)
        most = min(4096 * 17408 // max(K, N), 4096 * 512 * 22528 // (nA * R * (K + N)))
        T = _log(rng, 1, max(1, min(8192, most)))
        return dict(op=op, T=T, K=K, N=N, R=R, nA=nA, ragged=rng.random() < 0.5, none=rng.choice([0.0, 0.2]),
                    runs=rng.choice([1, 1, 4, 300]))
    Hkv, group, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128, 128, 256])
    n = _log(rng, 1, 8192)
    c = rng.choice([0, _log(rng, 1, 65536), _log(rng, 1, 65536)])
    while n > 1 and n * (n + c) * Hkv * group * D > 8192 * 8192 * 20 * 128:
        n = (n + 1) // 2
    most = min(8192 * 8192 * 20 * 128 // (n * (n + c) * Hkv * group * D), 10 ** 8 // ((n + c) * Hkv * D))
    B = _log(rng, 1, max(1, min(64, most)))
    ones = rng.choice([0, 0, B // 2, B])
    return dict(op=op, ones=ones, B=B, n_lo=int(n * rng.choice([0.0, 0.5, 1.0])), n_hi=n, c_lo=int(c * rng.choice([0.1, 1.0])),
                c_hi=c, Hq=Hkv * group, Hkv=Hkv, D=D, kv=rng.choice(["bf16", "e4m3"]), page=rng.choice([1, 16, 24, 32, 64, 128]),
                window=rng.choice([0, 0, 0, 1000]), cap=rng.choice([0.0, 0.0, 0.0, 30.0]))


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _tokens(c):
    """New tokens and cached ones of every sequence: `ones` of them have a single new token and lie among the others."""
    long = c["B"] - c["ones"]
    new = _spread(c["n_lo"], c["n_hi"], long) if long else []
    step = max(1, c["B"] // max(1, long))
    mix, left = [], list(new)
    for i in range(c["B"]):
        mix.append(left.pop(0) if left and (i % step == step - 1 or c["B"] - i <= len(left)) else 1)
    if sum(mix) == 0:
        mix[0] = 1
    return mix, _spread(c["c_lo"], c["c_hi"], c["B"])[::-1]


def _ids(c, g):
    """Adapter of every token: `runs` consecutive tokens belong to a request."""
    n = -(-c["T"] // c["runs"])
    one = torch.randint(0, c["nA"], (n,), generator=g, device=DEV)
    bare = torch.rand(n, generator=g, device=DEV) < c["none"]
    bare[0] = False
    one = torch.where(bare, torch.full_like(one, -1), one)
    return one.repeat_interleave(c["runs"])[:c["T"]].to(torch.int32).contiguous()


def work(case):
    c = case
    if c["op"] == "plan":
        T = sum(_spread(c["lo"], c["hi"], c["B"]))
        return {"bytes": c["B"] * 28 + T * 12 + (T // c["page"]) * 8, "flops": 0}
    if c["op"] == "norm8":
        r = 4 if c["res"] == "fp32" else 2
        gate = {"none": 0, "channel": 4 * c["D"], "token": 4 * c["M"] * c["D"]}[c["gate"]]
        return {"bytes": c["M"] * c["D"] * (4 + 2 * r + 1) + c["M"] * c["D"] // 8 + gate, "flops": 14 * c["M"] * c["D"]}
    if c["op"] == "lora":
        rank = c["R"] * (0.55 if c["ragged"] else 1.0)
        T = c["T"] * (1 - c["none"])
        used = min(c["nA"], max(1, -(-c["T"] // c["runs"])))
        return {"bytes": int(T * (2 * c["K"] + 8 * c["N"]) + used * rank * 2 * (c["K"] + c["N"])),
                "flops": int(2 * T * rank * (c["K"] + c["N"]))}
    e, pairs, seen = (2 if c["kv"] == "bf16" else 1), 0, 0
    for n, old in zip(*_tokens(c)):
        w = c["window"] or (old + n)
        first = max(0, old + 1 - w)
        seen += (old + n - first) if n else 0
        full = max(0, min(n, old + n - w))  # rows whose window is full
        rest = n - full
        pairs += full * w + rest * old + rest * (rest + 1) // 2
    rows = sum(_tokens(c)[0])
    return {"bytes": seen * c["Hkv"] * c["D"] * 2 * e + rows * c["Hq"] * c["D"] * 4, "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------- what a program has in hand

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pool(c, g, pages):
    """A pool of pages, [page][head][slot][D], filled with keys or values."""
    x = torch.empty((pages, c["Hkv"], c["page"], c["D"]), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    return x.to(torch.float8_e4m3fn) if c["kv"] == "e4m3" else x


def _int(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c=c)
    randn = lambda *n: torch.randn(n, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "plan":
        B, page = c["B"], c["page"]
        perm = torch.randperm(B, generator=g, device=DEV)
        new = _int(_spread(c["lo"], c["hi"], B))[perm]
        over = torch.randperm(B, generator=g, device=DEV)[:c["over"]]
        s["T"] = max(1, int(new.sum()))
        new[over] = -1
        s["new"] = new
        s["lens"] = torch.randint(0, c["old"] + 1, (B,), generator=g, device=DEV).to(torch.int32)
        s["pos"] = s["lens"] + 100 * (torch.arange(B, device=DEV) % 3).to(torch.int32)  # some were evicted from before
        extra = torch.randint(0, c["surplus"] + 1, (B,), generator=g, device=DEV)
        s["held"] = ((s["lens"] + page - 1) // page + extra).to(torch.int32)
        s["per"] = -(-(c["old"] + c["hi"]) // page) + c["surplus"] + 1
        need = int(torch.clamp((s["lens"] + new.clamp(min=0) + page - 1) // page - s["held"], min=0).sum())
        held = int(s["held"].sum())
        free = int(need * 0.6) if c["short"] else need + 50
        pages = B * s["per"] + 51
        free = min(free, pages - held)
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((B, s["per"]), -1, dtype=torch.int32, device=DEV)
        mine = torch.arange(s["per"], device=DEV) < s["held"][:, None]
        s["table"][mine] = ids[:held]
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        s["free"][:free] = ids[held:held + free]
        s["count"], s["pages"] = _int([free]), pages
        s["count_out"], s["held_out"], s["after"] = _int([0]), torch.zeros_like(s["held"]), torch.zeros_like(s["lens"])
        s["starts"] = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        s["seq"], s["slot"], s["where"] = (torch.zeros(s["T"], dtype=torch.int32, device=DEV) for _ in range(3))
        # the pools that the table is for (their sizes are all that matters here)
        s["k"], s["v"] = (torch.zeros(pages, 1, page, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    elif c["op"] == "norm8":
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
        s["q"] = torch.zeros(M, D, dtype=torch.int8, device=DEV)
        s["s"] = torch.zeros(M, D // 32, device=DEV)
        s["value"] = torch.zeros(M, D // 32, 32, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "lora":
        T, K, N, R, nA = c["T"], c["K"], c["N"], c["R"], c["nA"]
        s["x"] = randn(T, K).to(torch.bfloat16)
        s["y"] = randn(T, N) * 1.5
        s["a"] = (randn(nA, R, K) * K ** -0.5).to(torch.bfloat16)
        s["b"] = (randn(nA, N, R) * 0.05).to(torch.bfloat16)
        rank = torch.randint(1, R + 1, (nA,), generator=g, device=DEV).to(torch.int32)
        s["rank"] = rank if c["ragged"] else torch.full_like(rank, R)
        s["scale"] = 2.0 * torch.rand(nA, generator=g, device=DEV) + 0.1
        s["ids"] = _ids(c, g)
    else:
        new, old = _tokens(c)
        B, Hq, D, page = c["B"], c["Hq"], c["D"], c["page"]
        lens = [n + m for n, m in zip(new, old)]
        per = max(1, -(-max(lens) // page))
        pages = B * per + 3
        s["table"] = torch.randperm(pages, generator=g, device=DEV)[:B * per].to(torch.int32).view(B, per)
        s["k"], s["v"] = _pool(c, g, pages), _pool(c, g, pages)
        s["k_scale"], s["v_scale"] = (0.5, 0.25) if c["kv"] == "e4m3" else (1.0, 1.0)
        s["lens"], s["new"], s["n_max"] = _int(lens), new, max(new)
        s["starts"] = _int([sum(new[:i]) for i in range(B + 1)])
        T = sum(new)
        # logits of a few units: some tokens stand out, none takes all
        s["q"] = (randn(T, Hq, D) * (2.0 / s["k_scale"])).to(torch.bfloat16)
        s["o"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["scale"] = D ** -0.5
    return s


def run(state):
    op = state["c"]["op"]
    return (_own if own else _plain)[op](state)


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    c, page, T = s["c"], s["c"]["page"], s["T"]
    lens, held, count = s["lens"].long(), s["held"].long(), s["count"].long()
    over = s["new"] < 0
    n = s["new"].long().clamp(min=0)
    n = torch.where(lens + n <= s["per"] * page, n, torch.zeros_like(n))
    n = torch.where(torch.cumsum(n, 0) <= T, n, torch.zeros_like(n))
    want = torch.where(over, torch.zeros_like(n), (lens + n + page - 1) // page)
    back, need = (held - want).clamp(min=0), (want - held).clamp(min=0)
    there = count + back.sum()
    grant = (need == 0) | (torch.cumsum(need, 0) <= there)
    n, take = torch.where(grant, n, torch.zeros_like(n)), torch.where(grant, need, torch.zeros_like(need))
    s["held_out"].copy_(torch.where(grant, want, held))
    s["after"].copy_(torch.where(over, torch.zeros_like(n), lens + n))
    s["count_out"].copy_(there - take.sum())
    at = torch.arange(s["per"], device=DEV)
    back_at = count + (torch.cumsum(back, 0) - back)[:, None] + at - want[:, None]
    give = (at >= want[:, None]) & (at < held[:, None])
    s["free"][back_at[give]] = s["table"][give]
    take_at = there - 1 - (torch.cumsum(take, 0) - take)[:, None] - (at - held[:, None])
    get = (at >= held[:, None]) & (at < (held + take)[:, None])
    s["table"][get] = s["free"][take_at[get]]
    ends = torch.cumsum(n, 0)
    s["starts"][1:] = ends
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(ends, t, right=True)
    live = seq < c["B"]
    seq = torch.where(live, seq, torch.zeros_like(seq))
    i = t - (ends - n)[seq]
    s["seq"].copy_(torch.where(live, seq, torch.full_like(seq, -1)))
    s["slot"].copy_(torch.where(live, lens[seq] + i, torch.zeros_like(i)))
    s["where"].copy_(torch.where(live, s["pos"].long()[seq] + i, torch.zeros_like(i)))
    return {x: s[x] for x in ("table", "held_out", "free", "count_out", "after", "starts", "seq", "slot", "where")}


def _norm(x, kind, w, b, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return x if b is None else x + b


def _value(s):
    """What the 8-bit values stand for, in the 16 bits in which a product takes them."""
    torch.mul(s["q"].view(s["value"].shape), s["s"][:, :, None], out=s["value"])
    return {"r": s["r_out"], "s": s["s"], "x": s["value"]}


def _plain_norm8(s):
    c = s["c"]
    y = _norm(s["y"], c["post"], s["post_w"], s["post_b"], s["eps"])
    if s["gate"] is not None:
        y = y * s["gate"]
    h = s["r"].float() + s["scale"] * y
    s["r_out"].copy_(h)
    x = _norm(h, c["pre"], s["pre_w"], s["pre_b"], s["eps"]).view(c["M"], -1, 32)
    s["s"].copy_(x.abs().amax(-1) / 127.0)
    step = s["s"][:, :, None]
    q = torch.where(step > 0, x / step, torch.zeros_like(x))
    s["q"].view(x.shape).copy_(torch.round(q).clamp(-127, 127))
    return _value(s)


def _plain_lora(s):
    c = s["c"]
    T, K, N, R, nA = c["T"], c["K"], c["N"], c["R"], c["nA"]
    # every token through all adapters side by side, those that are not its own taken out between the products
    v = torch.matmul(s["x"].float(), s["a"].float().view(nA * R, K).t()).view(T, nA, R)
    mine = s["ids"][:, None] == torch.arange(nA, device=DEV)
    part = mine[:, :, None] & (torch.arange(R, device=DEV) < s["rank"][:, None])
    v = torch.where(part, v * s["scale"][:, None], torch.zeros_like(v))
    s["y"].add_(torch.matmul(v.view(T, nA * R), s["b"].float().transpose(1, 2).reshape(nA * R, N)))
    return s["y"]


def _bytes(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def _plain_attn(s):
    c = s["c"]
    B, n, Hq, Hkv, D = c["B"], s["n_max"], c["Hq"], c["Hkv"], c["D"]
    k, v = (_bytes(s[x])[s["table"].long()].view(s[x].dtype).float().transpose(1, 2).reshape(B, Hkv, -1, D) for x in "kv")
    starts, lens = s["starts"].long(), s["lens"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=DEV)
    # the sequences side by side, padded to the longest chunk
    q = s["q"][(starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    z = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"] * s["k_scale"])
    if c["cap"]:
        z = torch.tanh(z.div_(c["cap"])).mul_(c["cap"])
    z = z.view(B, Hkv, n, Hq // Hkv, -1)
    at = torch.arange(k.shape[2], device=DEV)
    end = (lens - count + 1)[:, None] + i
    seen = at < end[:, :, None]
    if c["window"]:
        seen = seen & (at >= end[:, :, None] - c["window"])
    seen = seen & (i < count[:, None])[:, :, None]
    z.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, k.shape[2]), v).view(B, Hkv, n, Hq // Hkv, D) * s["v_scale"]
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(starts[1:], t, right=True)
    s["o"].copy_(o[seq, t - starts[seq]])
    return s["o"]


_plain = {"plan": _plain_plan, "norm8": _plain_norm8, "lora": _plain_lora, "attn": _plain_attn}


# ---------------------------------------------------------------- the library's calls

def _handle(s):
    """The cache's descriptor: a program makes it once, beside the pools."""
    import q4_weight_quantized_gb300 as q4k
    if "handle" not in s:
        s["handle"] = q4k.kv_cache(s["k"], s["v"], s["table"], k_scale=s.get("k_scale", 1.0), v_scale=s.get("v_scale", 1.0))
    return s["handle"]


def _workspace(s, size):
    if "ws" not in s:
        s["ws_bytes"] = size()
        s["ws"] = torch.empty(max(1, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return s["ws"], s["ws_bytes"]


def _own_plan(s):
    import q4_weight_quantized_gb300 as q4k
    cache = _handle(s)
    ws, size = _workspace(s, lambda: q4k.q4k_batch_plan_workspace_size(cache))
    q4k.q4k_batch_plan(cache, s["lens"], s["new"], s["pos"], s["held"], s["held_out"], s["free"], s["count"], s["count_out"],
                       s["T"], s["after"], s["starts"], s["seq"], s["slot"], s["where"], ws, size)
    return {x: s[x] for x in ("table", "held_out", "free", "count_out", "after", "starts", "seq", "slot", "where")}


def _own_norm8(s):
    import q4_weight_quantized_gb300 as q4k
    c = s["c"]
    kind = {"none": q4k.Q4K_NORM_NONE, "rms": q4k.Q4K_NORM_RMS, "layer": q4k.Q4K_NORM_LAYER}
    M, D = c["M"], c["D"]
    q4k.q4k_norm_residual_x8(M, D, s["y"], D, kind[c["post"]], s["post_w"], s["post_b"], s["eps"], s["gate"],
                             D if c["gate"] == "token" else 0, s["scale"], s["r"], s["r_out"], D,
                             q4k.Q4K_RES_FP32 if c["res"] == "fp32" else q4k.Q4K_RES_BF16, kind[c["pre"]], s["pre_w"],
                             s["pre_b"], s["eps"], None, 0, s["q"], s["s"])
    return _value(s)


def _own_lora(s):
    import q4_weight_quantized_gb300 as q4k
    c = s["c"]
    T, K, N, R, nA = c["T"], c["K"], c["N"], c["R"], c["nA"]
    ws, size = _workspace(s, lambda: q4k.q4k_lora_add_workspace_size(nA, N, K, R, T))
    q4k.q4k_lora_add(nA, N, K, R, s["a"], s["b"], s["rank"], s["scale"], s["ids"], s["x"], T, K, s["y"], N, ws, size)
    return s["y"]


def _own_attn(s):
    import q4_weight_quantized_gb300 as q4k
    c = s["c"]
    cache, ld, T = _handle(s), c["Hq"] * c["D"], s["q"].shape[0]
    ws, size = _workspace(s, lambda: q4k.q4k_attn_chunk_workspace_size(cache, T, c["Hq"]))
    q4k.q4k_attn_chunk(cache, s["starts"], s["lens"], s["q"], T, ld, c["Hq"], s["scale"], c["cap"], c["window"], s["o"], ld,
                       ws, size)
    return s["o"]


_own = {"plan": _own_plan, "norm8": _own_norm8, "lora": _own_lora, "attn": _own_attn}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"plan": _exact_plan, "norm8": _exact_norm8, "lora": _exact_lora, "attn": _exact_attn}[case["op"]](case, s)


def _exact_plan(c, s):
    """Request by request on the host, with the free list as a list."""
    lens, new, pos, held = (s[x].tolist() for x in ("lens", "new", "pos", "held"))
    table, pool = s["table"].tolist(), s["free"].tolist()
    size, free = c["page"], pool[:int(s["count"][0])]
    ask, want, asked = [], [], 0
    for b in range(c["B"]):
        n = max(0, new[b])
        n = n if lens[b] + n <= s["per"] * size else 0
        asked += n
        ask.append(n if asked <= s["T"] else 0)
        want.append(0 if new[b] < 0 else -(-(lens[b] + ask[b]) // size))
    for b in range(c["B"]):
        free += table[b][want[b]:held[b]]
    pool[:len(free)] = free
    there, needed, starts, seq, slot, where = len(free), 0, [0], [], [], []
    for b in range(c["B"]):
        needed += max(0, want[b] - held[b])
        if want[b] > held[b] and needed > there:
            ask[b], want[b] = 0, held[b]
        for j in range(held[b], want[b]):
            table[b][j] = free.pop()
        for i in range(ask[b]):
            seq.append(b), slot.append(lens[b] + i), where.append(pos[b] + i)
        starts.append(len(seq))
    pad = s["T"] - len(seq)
    out = {"table": table, "held_out": want, "free": pool, "count_out": [len(free)],
           "after": [0 if n < 0 else m + k for n, m, k in zip(new, lens, ask)], "starts": starts, "seq": seq + [-1] * pad,
           "slot": slot + [0] * pad, "where": where + [0] * pad}
    return {x: _int(y) for x, y in out.items()}


def _exact_norm8(c, s):
    def norm(x, kind, w, b):
        if kind == "none":
            return x
        m = x.mean(1, keepdim=True) if kind == "layer" else 0.0
        out = (x - m) * ((x - m).pow(2).mean(1, keepdim=True) + s["eps"]).rsqrt() * w.double()
        return out + b.double() if b is not None else out
    h = norm(s["y"].double(), c["post"], s["post_w"], s["post_b"])
    h = s["r"].double() + s["scale"] * h * (1.0 if s["gate"] is None else s["gate"].double())
    x = norm(h, c["pre"], s["pre_w"], s["pre_b"]).view(s["value"].shape)
    step = x.abs().max(-1).values / 127
    return {"r": h, "s": step, "x": torch.round(x / step[..., None]) * step[..., None]}


def _exact_lora(c, s):
    """Adapter by adapter over the tokens that are its own."""
    y = s["y"].double()
    for a in range(c["nA"]):
        mine, r = (s["ids"] == a).nonzero()[:, 0], int(s["rank"][a])
        if len(mine):
            inner = s["x"][mine].double() @ s["a"][a, :r].double().T
            y[mine] += float(s["scale"][a]) * (inner @ s["b"][a, :, :r].double().T)
    return y


def _exact_attn(c, s):
    """Head by head, a block of query rows at a time."""
    G = c["Hq"] // c["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    begin = 0
    for b, n in enumerate(s["new"]):
        length, pages = int(s["lens"][b]), s["table"][b].long()
        for h in range(c["Hkv"]):
            k, v = (_bytes(s[x])[:, h][pages].view(s[x].dtype).double().flatten(0, 1)[:length] for x in "kv")
            for first in range(0, n, 1024):
                rows = torch.arange(first, min(n, first + 1024), device=DEV)
                x = s["q"][begin + rows, h * G:(h + 1) * G].double()
                z = torch.einsum("rgd,jd->rgj", x, k) * (s["scale"] * s["k_scale"])
                z = c["cap"] * torch.tanh(z / c["cap"]) if c["cap"] else z
                age = (length - n + rows)[:, None] - torch.arange(length, device=DEV)  # 0: the token itself
                dead = (age < 0) | (age >= c["window"]) if c["window"] else age < 0
                p = torch.softmax(z.masked_fill(dead[:, None], -math.inf), -1)
                o[begin + rows, h * G:(h + 1) * G] = torch.einsum("rgj,jd->rgd", p, v) * s["v_scale"]
        begin += n
    return o
