"""The example's steps of prompts' chunks and decode tokens together, against the same steps in plain 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import oracle
import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R
from oracle import step_ref
from tests.test_decode_loop import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    oracle.build()
    build_library()
    return q4k.load()


class Plain:
    """The server's model, a token's history as a list of keys and values.  Which experts a token goes to is a discrete choice that a
    rounding decides where two are about equal: there it takes the server's (`chosen`, one entry a layer), if they are."""

    def __init__(self, s):
        self.s = s
        self.keys = [[[] for _ in range(s.batch)] for _ in range(s.layers)]
        self.vals = [[[] for _ in range(s.batch)] for _ in range(s.layers)]

    def step(self, n_new, tokens, chosen):
        s, f = self.s, lambda t: t.double().cpu().numpy()
        H, D, heads, kvh = s.hidden, s.dim, s.heads, s.kv_heads
        norm = lambda r, w: R.norm_residual(None, 0, None, None, 0, None, 1, r, 1, w, None, s.eps)[1]  # noqa: E731
        adapter, ranks, scales = s.adapter.tolist(), s.ranks.tolist(), s.scales.tolist()
        owner = np.repeat(np.arange(s.batch), np.maximum(n_new, 0))
        ids = [adapter[b] for b in owner]
        add = lambda lora, x, y: step_ref.lora_add(f(lora[0]), f(lora[1]), ranks, scales, ids, x, y)[0]  # noqa: E731
        pos = np.concatenate([len(self.keys[0][b]) + np.arange(max(0, n)) for b, n in enumerate(n_new)]).astype(int)
        turn = s.rope[torch.from_numpy(pos).cuda()].cpu().numpy()
        r = f(s.embed[tokens.long()])
        x = norm(r, f(s.layer[0]["norm1"]))
        for i, w in enumerate(s.layer):
            q8, s8 = step_ref.in_eight(x.astype(np.float32))
            qkv = add(w["qkv_lora"], bits(x)[1], oracle.gemm_x8(w["qkv"][0], s.qkv_width, H, q8, s8)).astype(np.float32).reshape(len(r), -1, D)
            q = bits(R.rope(qkv[:, :heads], turn, D, False))[1]
            k, v = bits(R.rope(qkv[:, heads:heads + kvh], turn, D, False))[1], bits(qkv[:, heads + kvh:])[1]
            o = np.zeros((len(r), heads, D))
            for t, b in enumerate(owner):
                self.keys[i][b].append(k[t])
                self.vals[i][b].append(v[t])
                kk, vv = np.stack(self.keys[i][b]), np.stack(self.vals[i][b])
                for h in range(heads):
                    z = kk[:, h // (heads // kvh)] @ q[t, h] * D ** -0.5
                    p = np.exp(z - z.max())
                    o[t, h] = p @ vv[:, h // (heads // kvh)] / p.sum()
            ob, ov = bits(o.reshape(len(r), -1))
            r = r + add(w["out_lora"], ov, oracle.gemm(w["out"][0], H, heads * D, ob).astype(np.float64))
            xb, _ = bits(norm(r, f(w["norm2"])))
            route = oracle.gemm(w["router"][0], s.experts, H, xb)
            best = np.argsort(-route, 1)[:, :s.topk].astype(np.int32)
            for row, mine, theirs in zip(route, best, chosen[i]):
                if set(mine) != set(theirs):
                    # (a logit is off by a few hundredths of its row's norm: see below)
                    assert row[mine].min() - row[theirs].min() <= 0.1 * np.linalg.norm(row)
                    mine[:] = theirs
            g = np.exp(np.take_along_axis(route, best, 1))
            g = (g / g.sum(1, keepdims=True)).astype(np.float32)
            r = r + oracle.moe_ffn(w["gate"][0], w["up"][0], w["down"][0], s.experts, s.width, H, xb, best, g)
            x = norm(r, f(s.layer[i + 1]["norm1"] if i + 1 < s.layers else s.norm_last))
        ends = np.cumsum(np.maximum(n_new, 0)) - 1
        for b, n in enumerate(n_new):
            if n < 0:
                for i in range(s.layers):
                    self.keys[i][b], self.vals[i][b] = [], []
        return oracle.gemm(s.head[0], s.vocab, H, bits(x[np.maximum(ends, 0)])[0])


@pytest.fixture
def chosen(monkeypatch):
    """The experts that each call of the expert layer was given."""
    calls, real = [], q4k.q4k_moe_ffn
    monkeypatch.setattr(q4k, "q4k_moe_ffn", lambda *a: (calls.append(a[7].cpu().numpy()), real(*a)))
    return calls


def run(s, n_new, tokens, u=None):
    t = torch.tensor(tokens, device="cuda")
    return s.step(torch.tensor(n_new, dtype=torch.int32, device="cuda"), t, torch.full((s.batch,), 0.5, device="cuda") if u is None else u)


def test_steps_match_the_plain_model(chosen):
    """Chunks, single tokens, requests without new tokens, one that ends and whose pages go to another."""
    from examples.mixed_step import Server
    s = Server(batch=4, pages=14, max_len=96, tokens=80, seed=3)
    s.adapter.copy_(torch.tensor([1, -1, 0, 2], dtype=torch.int32))
    plain, rng = Plain(s), np.random.default_rng(0)
    for step, n_new in enumerate(([20, 7, 0, 1], [30, 1, 17, 1], [1, 1, 18, 1], [-1, 1, 1, 33], [60, 1, 1, 1], [1, 1, 1, -1])):
        total = sum(max(0, n) for n in n_new)
        tokens = rng.integers(0, s.vocab, total).tolist()
        logits, _ = run(s, n_new, tokens)
        want = plain.step(n_new, torch.tensor(tokens, device="cuda"), chosen[-s.layers:])
        rows = [b for b in range(4) if n_new[b] > 0]
        got = logits.double().cpu().numpy()[rows]
        # between a token and its logits lie some thirty roundings to bf16 and f16-sized weights (2^-8 at most each) and four to 8
        # bits (half of 1/127 of a block's largest value, so at most 2^-7 of its norm), which add like noise
        assert np.linalg.norm(got - want[rows]) <= np.linalg.norm(want[rows]) * (30 * 2.0 ** -16 + 4 * 2.0 ** -14) ** 0.5, step
    assert s.lens.tolist() == [61, 12, 38, 0]
    held = s.held.tolist()
    assert held == [4, 1, 3, 0] and int(s.count) == 14 - sum(held)
    pages = sum((s.table[b, :held[b]].tolist() for b in range(4)), []) + s.free[:int(s.count)].tolist()
    assert sorted(pages) == list(range(14))
    q4k.q4k_check_device()


def test_a_prompt_in_chunks_and_at_once():
    """The same cache contents and logits, to the roundings, however a prompt is cut and whatever runs beside it."""
    from examples.mixed_step import Server
    tokens = np.random.default_rng(1).integers(0, 1000, 70).tolist()

    def logits_of(cuts, beside):
        s = Server(batch=2, pages=12, max_len=96, tokens=80, seed=5)
        s.adapter.copy_(torch.tensor([2, 0], dtype=torch.int32))
        at, out = 0, None
        for n in cuts:
            extra = 1 if beside else 0
            out = run(s, [n, extra], tokens[at:at + n] + [3] * extra)[0][0].clone()
            at += n
        q4k.q4k_check_device()
        return out.double()

    whole = logits_of([70], False)
    for cuts, beside in (([33, 37], False), ([1, 16, 17, 36], True), ([69, 1], True)):
        got = logits_of(cuts, beside)
        assert torch.linalg.norm(got - whole) <= torch.linalg.norm(whole) * (2 * (30 * 2.0 ** -16 + 4 * 2.0 ** -14)) ** 0.5


def test_tokens_without_pages_wait():
    from examples.mixed_step import Server
    s = Server(batch=2, pages=3, max_len=96, tokens=80, seed=5)
    with pytest.raises(RuntimeError):
        run(s, [30, 40], [1] * 70)     # the first has its two pages, the second lacks two
    assert s.lens.tolist() == [30, 0] and s.held.tolist() == [2, 0] and int(s.count) == 1


def test_example_runs(capsys):
    from examples import mixed_step
    mixed_step.main(30)
    assert "ends" in capsys.readouterr().out
