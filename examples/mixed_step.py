"""Steps of a small server that runs chunks of prompts and decode tokens of many requests together, some with adapters.

Per step: pages and slots for the new tokens; then per layer the qkv product over 8-bit activations with the requests' adapters
beside it, rotary append to the paged cache, attention of the chunks over it, the output product with its adapters, residual and norm,
the routed expert layer, residual and norm (8 bits for the next product); then the vocabulary's product and sampling for the requests
whose last token this step has.  Requests come and go; their pages return to the free list.  Weights are random; the point is the calls.

    python examples/mixed_step.py [steps]
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


class Server:
    hidden, heads, kv_heads, dim, layers = 512, 8, 2, 64, 2
    experts, topk, width, vocab = 4, 2, 256, 1000
    page, eps, base = 16, 1e-6, 10000.0
    adapters, rank = 3, 16

    def __init__(self, batch: int, pages: int, max_len: int, tokens: int, seed: int = 1):
        """`batch` requests at a time, `pages` pages in each pool, at most `tokens` tokens a step."""
        self.batch, self.tokens = batch, tokens
        self.qkv_width, self.q_width = (self.heads + 2 * self.kv_heads) * self.dim, self.heads * self.dim
        dev = torch.device("cuda")
        counter = iter(range(10 ** 6))

        def q4(rows, cols, copies=1):
            """Random Q4_K blocks, on the host (for a check) and on the device."""
            w = np.concatenate([synth.weights(synth.seed(seed, next(counter)), rows, cols, cols ** -0.5) for _ in range(copies)])
            return w, torch.from_numpy(w).to(dev)

        g = torch.Generator(device="cpu").manual_seed(seed)
        rand = lambda *n: torch.randn(n, generator=g)  # noqa: E731

        def lora(rows, cols):
            """Adapters of a projection: [adapters][rank][cols] and [adapters][rows][rank]."""
            return ((rand(self.adapters, self.rank, cols) * cols ** -0.5).to(torch.bfloat16).to(dev),
                    (rand(self.adapters, rows, self.rank) * 0.1).to(torch.bfloat16).to(dev))

        self.embed = rand(self.vocab, self.hidden).to(dev)
        self.layer = []
        for _ in range(self.layers):
            self.layer.append(dict(
                qkv=q4(self.qkv_width, self.hidden), out=q4(self.hidden, self.q_width), router=q4(self.experts, self.hidden),
                gate=q4(self.width, self.hidden, self.experts), up=q4(self.width, self.hidden, self.experts),
                down=q4(self.hidden, self.width, self.experts), norm1=(rand(self.hidden).abs() + 0.5).to(dev),
                norm2=(rand(self.hidden).abs() + 0.5).to(dev), qkv_lora=lora(self.qkv_width, self.hidden),
                out_lora=lora(self.hidden, self.q_width)))
        self.norm_last, self.head = torch.ones(self.hidden, device=dev), q4(self.vocab, self.hidden)
        self.ranks = torch.tensor([16, 5, 11], dtype=torch.int32, device=dev)
        self.scales = torch.tensor([1.0, 2.0, 0.5], device=dev)
        half = self.dim // 2
        angle = torch.arange(4096, dtype=torch.float64)[:, None] * self.base ** (-torch.arange(half, dtype=torch.float64) / half)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().to(dev)

        # the pools of a layer; one table of pages and one free list for all layers
        int32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=dev)  # noqa: E731
        self.table = int32(batch, -(-max_len // self.page))
        self.caches = []
        for _ in range(self.layers):
            k = torch.zeros(pages, self.kv_heads, self.page, self.dim, dtype=torch.bfloat16, device=dev)
            v = torch.zeros_like(k)
            self.caches.append(dict(k=k, v=v, c=q4k.kv_cache(k, v, self.table)))
        self.free = torch.randperm(pages, generator=g).to(torch.int32).to(dev)
        self.count = torch.tensor([pages], dtype=torch.int32, device=dev)
        self.lens, self.held, self.adapter = int32(batch), int32(batch), torch.full((batch,), -1, dtype=torch.int32, device=dev)
        self.starts, self.seq, self.slot, self.pos = int32(batch + 1), int32(tokens), int32(tokens), int32(tokens)

        # buffers and workspaces that every step uses again
        new = lambda *shape, t=torch.float32: torch.empty(*shape, dtype=t, device=dev)  # noqa: E731
        T, c, n = tokens, self.caches[0]["c"], self.adapters
        self.x, self.y, self.qkv = new(T, self.hidden, t=torch.bfloat16), new(T, self.hidden), new(T, self.qkv_width)
        self.q8, self.s8 = new(T, self.hidden, t=torch.int8), new(T, self.hidden // 32)
        self.q, self.o = new(T, self.q_width, t=torch.bfloat16), new(T, self.q_width, t=torch.bfloat16)
        self.route, self.r, self.logits = new(T, self.experts), new(T, self.hidden), new(batch, self.vocab)
        self.token, self.prob = int32(batch), new(batch)
        size = max(q4k.q4k_batch_plan_workspace_size(c), q4k.q4k_attn_chunk_workspace_size(c, T, self.heads),
                   q4k.q4k_lora_add_workspace_size(n, self.qkv_width, self.hidden, self.rank, T),
                   q4k.q4k_lora_add_workspace_size(n, self.hidden, self.q_width, self.rank, T),
                   q4k.q4k_gemm_x8_workspace_size(T, self.hidden),
                   q4k.q4k_moe_ffn_workspace_size(self.experts, self.width, self.hidden, T, self.topk))
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)

    def product(self, w, rows, x, n, y):
        q4k.q4k_gemm(w[1], rows, x.shape[1], x, n, x.shape[1], y, rows, self.ws, self.ws.numel())

    def adapt(self, lora, rows, x, n, y, ids):
        """y += what the requests' adapters make of x."""
        a, b = lora
        q4k.q4k_lora_add(self.adapters, rows, x.shape[1], self.rank, a, b, self.ranks, self.scales, ids, x, n, x.shape[1], y, rows,
                         self.ws, self.ws.numel())

    def add_and_norm(self, y, weight, n, eight):
        """r += y; x = the next block's input, in 8 bits as well where the next product takes them."""
        args = (n, self.hidden, y, self.hidden, q4k.Q4K_NORM_NONE, None, None, 0.0, None, 0, 1.0, self.r, self.r, self.hidden,
                q4k.Q4K_RES_FP32, q4k.Q4K_NORM_RMS, weight, None, self.eps, self.x, self.hidden)
        if eight:
            q4k.q4k_norm_residual_x8(*args, self.q8, self.s8)
        else:
            q4k.q4k_norm_residual(*args)

    def step(self, n_new, tokens, u, temperature=0.8):
        """n_new[b] new tokens of each request (negative: it is over), side by side in `tokens`; all must be granted.  Returns the
        logits of each request's last token and, drawn from them by the numbers u, the next tokens (no new tokens: of no meaning)."""
        B, T, W = self.batch, self.tokens, self.qkv_width
        q4k.q4k_batch_plan(self.caches[0]["c"], self.lens, n_new, None, self.held, self.held, self.free, self.count, self.count, T,
                           self.lens, self.starts, self.seq, self.slot, self.pos, self.ws, self.ws.numel())
        n = int(self.starts[-1])
        if n != len(tokens):
            raise RuntimeError(f"{n} of {len(tokens)} tokens have pages")
        if n == 0:
            return self.logits, self.token
        ids = self.adapter[self.seq[:n].long()].contiguous()
        self.r[:n] = self.embed[tokens.long()]
        self.add_and_norm(None, self.layer[0]["norm1"], n, True)
        for i, (w, c) in enumerate(zip(self.layer, self.caches)):
            q4k.q4k_gemm_x8(w["qkv"][1], W, self.hidden, self.q8, self.s8, n, self.qkv, W, self.ws, self.ws.numel())
            self.adapt(w["qkv_lora"], W, self.x, n, self.qkv, ids)
            k_at = self.qkv.data_ptr() + 4 * self.q_width
            v_at = k_at + 4 * self.kv_heads * self.dim
            q4k.q4k_kv_append(c["c"], n, self.heads, self.qkv, W, k_at, W, v_at, W, self.seq, self.slot, self.pos, self.rope,
                              self.rope.shape[0], self.dim, q4k.Q4K_ROPE_HALF, self.q, self.q_width)
            q4k.q4k_attn_chunk(c["c"], self.starts, self.lens, self.q, n, self.q_width, self.heads, self.dim ** -0.5, 0.0, 0, self.o,
                               self.q_width, self.ws, self.ws.numel())
            self.product(w["out"], self.hidden, self.o, n, self.y)
            self.adapt(w["out_lora"], self.hidden, self.o, n, self.y, ids)
            self.add_and_norm(self.y, w["norm2"], n, False)
            self.product(w["router"], self.experts, self.x, n, self.route)
            gates, best = torch.softmax(self.route[:n], 1).topk(self.topk, 1)
            gates = (gates / gates.sum(1, keepdim=True)).contiguous()
            q4k.q4k_moe_ffn(w["gate"][1], w["up"][1], w["down"][1], self.experts, self.width, self.hidden, self.x,
                            best.to(torch.int32).contiguous(), gates, n, self.topk, self.y, self.ws, self.ws.numel())
            last = i + 1 == self.layers
            self.add_and_norm(self.y, self.norm_last if last else self.layer[i + 1]["norm1"], n, not last)
        ends = (self.starts[1:].long() - 1).clamp(min=0)
        self.product(self.head, self.vocab, self.x[ends].contiguous(), B, self.logits)
        full = lambda v, t=torch.float32: torch.full((B,), v, dtype=t, device="cuda")  # noqa: E731
        q4k.q4k_sample(self.logits, B, self.vocab, self.vocab, full(temperature), full(50, torch.int32), full(0.95), None, u, self.token,
                       self.prob)
        return self.logits, self.token


def main(steps: int) -> None:
    s = Server(batch=4, pages=40, max_len=160, tokens=80)
    g = torch.Generator().manual_seed(0)
    left = [[], [], [], []]           # of each request's prompt
    made = [[], [], [], []]
    s.adapter.copy_(torch.tensor([0, -1, 2, 1], dtype=torch.int32))
    last = torch.zeros(4, dtype=torch.int32)
    busy = [False] * 4
    for step in range(steps):
        n_new, tokens = [], []
        for b in range(4):
            if not busy[b]:           # a new request takes the place
                left[b] = torch.randint(0, s.vocab, (int(torch.randint(3, 90, (1,), generator=g)),), generator=g).tolist()
                made[b], busy[b] = [], True
            elif len(made[b]) >= 12:  # over
                print(f"step {step}: request {b} ends: {made[b]}")
                n_new.append(-1)
                busy[b] = False
                continue
            take = left[b][:20] or ([int(last[b])] if made[b] else [])
            left[b] = left[b][20:]
            n_new.append(len(take))
            tokens += take
        _, token = s.step(torch.tensor(n_new, dtype=torch.int32, device="cuda"), torch.tensor(tokens, device="cuda"),
                          torch.rand(4, generator=g).cuda())
        last = token.cpu()
        for b in range(4):
            if n_new[b] > 0 and not left[b]:
                made[b].append(int(last[b]))
    q4k.q4k_check_device()
    print(f"{int(s.count)} pages free, lengths {s.lens.tolist()}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
