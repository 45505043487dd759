"""The example's decode loop against the same steps in plain 64-bit arithmetic, and with a cache at its budget."""
import numpy as np
import pytest
import torch

import oracle
import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    oracle.build()
    build_library()
    return q4k.load()


def bits(a):
    """64-bit values as bf16 bit patterns, and the values they stand for."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.float32).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16), t.double().numpy()


def test_steps_match_the_plain_model(ref):
    from examples.decode_loop import Decoder
    d = Decoder(batch=3, budget=10 ** 6, max_len=32, seed=3)
    rng = np.random.default_rng(0)
    H, D, heads, kvh = d.hidden, d.dim, d.heads, d.kv_heads
    keys = [np.zeros((3, kvh, 16, D)) for _ in range(d.layers)]
    vals = [np.zeros((3, kvh, 16, D)) for _ in range(d.layers)]
    table = np.arange(3)[:, None]                       # the plain cache: a page of 16 slots a sequence
    norm = lambda r, w: R.norm_residual(None, 0, None, None, 0, None, 1, r, 1, w, None, d.eps)[1]  # noqa: E731
    f = lambda t: t.double().cpu().numpy()              # noqa: E731
    for step in range(6):
        tokens = torch.from_numpy(rng.integers(0, d.vocab, 3).astype(np.int32)).cuda()
        u = torch.rand(3, device="cuda")
        logits, token = d.step(tokens, u)
        got, drawn = f(logits), token.tolist()
        r = f(d.embed[tokens.long()])
        xb, _ = bits(norm(r, f(d.layer[0]["norm1"])))
        for i, w in enumerate(d.layer):
            qkv = oracle.gemm(w["qkv"][0], d.qkv_width, H, xb).astype(np.float32).reshape(3, -1, D)
            turn = np.repeat(d.rope[step:step + 1].cpu().numpy(), 3, 0)
            q = bits(R.rope(qkv[:, :heads], turn, D, False))[1]
            keys[i][:, :, step] = bits(R.rope(qkv[:, heads:heads + kvh], turn, D, False))[1]
            vals[i][:, :, step] = bits(qkv[:, heads + kvh:])[1]
            o = R.attn_decode(keys[i], vals[i], table, [step + 1] * 3, q[:, None], 1, D ** -0.5)[0].reshape(3, -1)
            r = r + oracle.gemm(w["out"][0], H, heads * D, bits(o)[0])
            xb, _ = bits(norm(r, f(w["norm2"])))
            route = oracle.gemm(w["router"][0], d.experts, H, xb)
            ids = np.argsort(-route, 1)[:, :d.topk].astype(np.int32)
            g = np.exp(np.take_along_axis(route, ids, 1))
            g = (g / g.sum(1, keepdims=True)).astype(np.float32)
            r = r + oracle.moe_ffn(w["gate"][0], w["up"][0], w["down"][0], d.experts, d.width, H, xb, ids, g)
            xb, _ = bits(norm(r, f(d.layer[i + 1]["norm1"] if i + 1 < d.layers else d.norm_last)))
        want = oracle.gemm(d.head[0], d.vocab, H, xb)
        # some thirty roundings to bf16 (2^-9 each at most) lie between the token and a logit, and add like noise
        assert np.linalg.norm(got - want) <= np.linalg.norm(want) * 30 ** 0.5 * 2.0 ** -9, step
        for b in range(3):
            assert drawn[b] == R.sample(got[b].astype(np.float32), 0.8, 50, 0.95, 0.0, float(u[b]))[0]
    q4k.q4k_check_device()


def test_a_cache_at_its_budget():
    from examples.decode_loop import Decoder

    def run():
        d = Decoder(batch=2, budget=12, max_len=16, seed=5)
        g = torch.Generator(device="cuda").manual_seed(1)
        token, out = torch.tensor([5, 6], dtype=torch.int32, device="cuda"), []
        for _ in range(30):
            logits, token = d.step(token, torch.rand(2, generator=g, device="cuda"))
            token = token.clone()
            assert torch.isfinite(logits).all()
            out.append(token)
        q4k.q4k_check_device()
        return d, torch.stack(out)

    d, first = run()
    assert torch.equal(first, run()[1])                 # the same numbers, the same tokens
    assert d.lens.tolist() == [12, 12]
    for c in d.caches:
        held = c["positions"][:, :, :12]
        for b in range(2):
            for h in range(d.kv_heads):
                p = set(held[b, h].tolist())
                assert len(p) == 12 and {0, 26, 27, 28, 29} <= p   # the sink, and the recent ones
