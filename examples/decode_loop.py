"""A decode loop of a small decoder with Q4_K weights: every operator of a step, in the order a server runs them.

Per step and layer: qkv product, rotary append to the paged cache, attention over it (adding up the weight each cached
token received), eviction once a cache is over its budget, output product, residual and norm, routed expert layer,
residual and norm; then the vocabulary's product and sampling.  Weights are random; the point is the calls.

    python examples/decode_loop.py [steps]
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import q4_weight_quantized_gb300 as q4k  # noqa: E402
import synth  # noqa: E402


class Decoder:
    hidden, heads, kv_heads, dim, layers = 512, 8, 2, 64, 2
    experts, topk, width, vocab = 4, 2, 256, 1000
    page, eps, base = 16, 1e-6, 10000.0

    def __init__(self, batch: int, budget: int, max_len: int, seed: int = 1, sinks: int = 1, recent: int = 4):
        self.batch, self.budget, self.sinks, self.recent = batch, budget, sinks, recent
        self.qkv_width = (self.heads + 2 * self.kv_heads) * self.dim
        dev = torch.device("cuda")
        counter = iter(range(10 ** 6))

        def q4(rows, cols, copies=1):
            """Random Q4_K blocks, on the host (for a check) and on the device."""
            w = np.concatenate([synth.weights(synth.seed(seed, next(counter)), rows, cols, cols ** -0.5) for _ in range(copies)])
            return w, torch.from_numpy(w).to(dev)

        g = torch.Generator(device="cpu").manual_seed(seed)
        self.embed = torch.randn(self.vocab, self.hidden, generator=g).to(dev)
        self.layer = []
        for _ in range(self.layers):
            self.layer.append(dict(
                qkv=q4(self.qkv_width, self.hidden), out=q4(self.hidden, self.heads * self.dim), router=q4(self.experts, self.hidden),
                gate=q4(self.width, self.hidden, self.experts), up=q4(self.width, self.hidden, self.experts),
                down=q4(self.hidden, self.width, self.experts), norm1=torch.rand(self.hidden, generator=g).to(dev) + 0.5,
                norm2=torch.rand(self.hidden, generator=g).to(dev) + 0.5))
        self.norm_last, self.head = torch.ones(self.hidden, device=dev), q4(self.vocab, self.hidden)
        half = self.dim // 2
        angle = torch.arange(4096, dtype=torch.float64)[:, None] * self.base ** (-torch.arange(half, dtype=torch.float64) / half)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().to(dev)

        # one paged cache per layer; the pages of a sequence lie scattered in the pool
        per = -(-max_len // self.page)
        self.slots = per * self.page
        self.caches = []
        for i in range(self.layers):
            k = torch.zeros(batch * per, self.kv_heads, self.page, self.dim, dtype=torch.bfloat16, device=dev)
            v = torch.zeros_like(k)
            table = torch.randperm(batch * per, generator=g).to(torch.int32).view(batch, per).to(dev)
            weights = torch.zeros(batch, self.kv_heads, self.slots, device=dev)
            positions = torch.zeros(batch, self.kv_heads, self.slots, dtype=torch.int32, device=dev)
            self.caches.append(dict(k=k, v=v, table=table, weights=weights, positions=positions, c=q4k.kv_cache(k, v, table)))
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.pos = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.seq = torch.arange(batch, dtype=torch.int32, device=dev)

        # buffers and workspaces that every step uses again
        new = lambda *shape, t=torch.float32: torch.empty(*shape, dtype=t, device=dev)  # noqa: E731
        self.x, self.y, self.qkv = new(batch, self.hidden, t=torch.bfloat16), new(batch, self.hidden), new(batch, self.qkv_width)
        self.q = new(batch, self.heads, self.dim, t=torch.bfloat16)
        self.o = new(batch, self.heads * self.dim, t=torch.bfloat16)
        self.route, self.logits = new(batch, self.experts), new(batch, self.vocab)
        self.r, self.new_lens = new(batch, self.hidden), torch.empty_like(self.lens)
        self.token, self.prob = torch.zeros(batch, dtype=torch.int32, device=dev), new(batch)
        c = self.caches[0]["c"]
        size = max(q4k.q4k_attn_decode_workspace_size(c, self.heads, 1, self.slots), q4k.q4k_kv_evict_workspace_size(c, self.slots),
                   q4k.q4k_moe_ffn_workspace_size(self.experts, self.width, self.hidden, batch, self.topk))
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)

    def product(self, w, rows, x, y):
        cols = x.shape[1]
        q4k.q4k_gemm(w[1], rows, cols, x, self.batch, cols, y, rows)

    def add_and_norm(self, y, weight):
        """r += y; x = the next block's input."""
        q4k.q4k_norm_residual(self.batch, self.hidden, y, self.hidden, q4k.Q4K_NORM_NONE, None, None, 0.0, None, 0, 1.0, self.r,
                              self.r, self.hidden, q4k.Q4K_RES_FP32, q4k.Q4K_NORM_RMS, weight, None, self.eps, self.x, self.hidden)

    def step(self, tokens, u, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0):
        """One token for each sequence: the logits and, drawn from them by the numbers u in [0, 1), the next tokens."""
        B, W = self.batch, self.qkv_width
        self.r.copy_(self.embed[tokens.long()])
        self.add_and_norm(None, self.layer[0]["norm1"])
        after = self.lens + 1
        over = bool((after > self.budget).any()) if self.budget < self.slots else False
        for i, (w, c) in enumerate(zip(self.layer, self.caches)):
            self.product(w["qkv"], W, self.x, self.qkv)
            k_at = self.qkv.data_ptr() + 4 * self.heads * self.dim
            v_at = k_at + 4 * self.kv_heads * self.dim
            q4k.q4k_kv_append(c["c"], B, self.heads, self.qkv, W, k_at, W, v_at, W, self.seq, self.lens, self.pos, self.rope,
                              self.rope.shape[0], self.dim, q4k.Q4K_ROPE_HALF, self.q, self.heads * self.dim, c["weights"],
                              c["positions"], self.slots)
            q4k.q4k_attn_decode(c["c"], after, self.q, self.heads * self.dim, self.heads, 1, self.dim ** -0.5, 0.0, 0, self.o,
                                self.heads * self.dim, c["weights"], self.slots, 1.0, self.ws, self.ws.numel())
            if over:
                q4k.q4k_kv_evict(c["c"], after, self.new_lens, self.budget, self.sinks, self.recent, c["weights"], c["positions"],
                                 c["weights"], c["positions"], self.slots, self.ws, self.ws.numel())
            self.product(w["out"], self.hidden, self.o, self.y)
            self.add_and_norm(self.y, w["norm2"])
            self.product(w["router"], self.experts, self.x, self.route)
            gates, ids = torch.softmax(self.route, 1).topk(self.topk, 1)
            gates = (gates / gates.sum(1, keepdim=True)).contiguous()
            q4k.q4k_moe_ffn(w["gate"][1], w["up"][1], w["down"][1], self.experts, self.width, self.hidden, self.x,
                            ids.to(torch.int32).contiguous(), gates, B, self.topk, self.y, self.ws, self.ws.numel())
            self.add_and_norm(self.y, self.layer[i + 1]["norm1"] if i + 1 < self.layers else self.norm_last)
        self.product(self.head, self.vocab, self.x, self.logits)
        full = lambda v, t=torch.float32: torch.full((B,), v, dtype=t, device="cuda")  # noqa: E731
        q4k.q4k_sample(self.logits, B, self.vocab, self.vocab, full(temperature), full(top_k, torch.int32), full(top_p), full(min_p),
                       u, self.token, self.prob)
        self.lens = self.new_lens.clone() if over else after
        self.pos = self.pos + 1
        return self.logits, self.token


def main(steps: int) -> None:
    d = Decoder(batch=4, budget=24, max_len=48)
    g = torch.Generator(device="cuda").manual_seed(0)
    token = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    out = []
    for _ in range(steps):
        _, token = d.step(token, torch.rand(d.batch, generator=g, device="cuda"))
        token = token.clone()
        out.append(token)
    q4k.q4k_check_device()
    for b, row in enumerate(torch.stack(out, 1).tolist()):
        held = sorted(d.caches[0]["positions"][b, 0, :int(d.lens[b])].tolist())
        print(f"sequence {b}: {row}\n  cached positions, first head: {held}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
