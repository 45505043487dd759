"""The norm between two blocks with its output in 8 bits."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref, step_ref
from tests.test_decode_ops import BF, gen_of, lib, np64  # noqa: F401

pytestmark = pytest.mark.gpu
KIND = {"none": 0, "rms": 1, "layer": 2}


def make(M, D, res, gate, bias, seed=0, pad=0):
    g = gen_of(D + M + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ld = D + pad
    y, r = (rnd(M, ld) * 4 + 0.5)[:, :D], (rnd(M, ld) * 2).to(res)[:, :D]
    p = dict(y=y, r=r, pw=1 + 0.2 * rnd(D), qw=1 + 0.2 * rnd(D), pb=rnd(D) if bias else None, qb=rnd(D) if bias else None,
             gate=None if gate is None else rnd(1 if gate == "row" else M, D), ld=ld, res=res)
    return p


def call(p, post, pre, x=None, r_out=None, eight=True, q=None, s=None):
    M, D = p["y"].shape
    args = (M, D, p["y"], p["ld"], KIND[post], p["pw"], p["pb"], 1e-5, p["gate"], D if p["gate"] is not None and p["gate"].shape[0] > 1 else 0,
            0.7, p["r"], r_out, p["ld"], q4k.Q4K_RES_FP32 if p["res"] == torch.float32 else q4k.Q4K_RES_BF16, KIND[pre], p["qw"],
            p["qb"], 1e-6, x, 0 if x is None else x.stride(0))
    if not eight:
        return q4k.q4k_norm_residual(*args)
    q = torch.full((M, D), 99, dtype=torch.int8, device="cuda") if q is None else q
    s = torch.full((M, D // 32), -1.0, device="cuda") if s is None else s
    q4k.q4k_norm_residual_x8(*args, q, s)
    return q, s


SIZES = [(1, 32, 0), (3, 64, 0), (2, 5120, 0), (3, 768, 3), (2, 96, 1), (2, 16384, 0), (2, 16416, 0), (1, 40000, 0), (700, 5120, 0),
         (700, 768, 0), (2100, 64, 0), (401, 2048, 0), (300, 5120, 1), (2, 12384, 5)]


@pytest.mark.parametrize("M,D,pad", SIZES)
@pytest.mark.parametrize("gate,res", [(None, torch.float32), ("row", BF), ("all", torch.float32)])
def test_eight_bits_of_what_is_known_exactly(M, D, pad, gate, res):
    """Without a next norm the fp32 residual is what is quantized: q and s equal the rule's bits.  The other outputs are
    q4k_norm_residual's, bit for bit."""
    p = make(M, D, torch.float32, gate, res == BF, pad=pad)
    h, h2 = torch.zeros(M, p["ld"], device="cuda"), torch.zeros(M, p["ld"], device="cuda")
    x, x2 = torch.zeros(M, D, dtype=BF, device="cuda"), torch.zeros(M, D, dtype=BF, device="cuda")
    q, s = call(p, "rms", "none", x, h)
    call(p, "rms", "none", x2, h2, eight=False)
    assert torch.equal(h, h2) and torch.equal(x, x2)
    wq, ws = step_ref.in_eight(h[:, :D].cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    q2, s2 = call(p, "rms", "none")  # neither residual nor bf16
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert (h[:, D:] == 0).all()


@pytest.mark.parametrize("M,D,pad", [(1, 5120, 0), (3, 768, 3), (700, 5120, 0), (1401, 64, 0), (2, 20000, 0), (500, 1024, 0)])
@pytest.mark.parametrize("post,pre,gate,res,bias", [("rms", "rms", None, BF, False), ("none", "layer", "row", torch.float32, True),
                                                    ("layer", "rms", "all", BF, True)])
def test_eight_bits_of_a_norm(M, D, pad, post, pre, gate, res, bias):
    """The values are off by half a step, s / 2, and by what test_norm allows the fp32 values; their bf16 form is
    q4k_norm_residual's."""
    p = make(M, D, res, gate, bias, pad=pad)
    r1, r2 = (torch.zeros(M, p["ld"], dtype=res, device="cuda") for _ in range(2))
    x, x2 = torch.zeros(M, D, dtype=BF, device="cuda"), torch.zeros(M, D, dtype=BF, device="cuda")
    q, s = call(p, post, pre, x, r1)
    call(p, post, pre, x2, r2, eight=False)
    assert torch.equal(r1, r2) and torch.equal(x, x2)
    q2, s2 = call(p, post, pre)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    f = lambda t: None if t is None else np64(t)  # noqa: E731
    h, want = decode_ref.norm_residual(f(p["y"]), KIND[post], f(p["pw"]), f(p["pb"]), 1e-5, f(p["gate"]), 0.7, f(p["r"]), KIND[pre],
                                       f(p["qw"]), f(p["qb"]), 1e-6)
    gt = 1 if p["gate"] is None else np.abs(f(p["gate"]))
    terms = np.abs(h) + np.abs(h - f(p["r"])) + np.abs(f(p["r"])) + (0 if p["pb"] is None else np.abs(f(p["pb"])) * 0.7 * gt)
    base = (h - h.mean(1, keepdims=True)) if pre == "layer" else h
    off = (np.abs(want) + (0 if p["qb"] is None else np.abs(f(p["qb"]))) +
           terms * np.abs(f(p["qw"])) / np.sqrt((base ** 2).mean(1, keepdims=True) + 1e-6)) * 200 * 2.0 ** -24
    step = np64(s).repeat(32, 1)
    assert (np.abs(np64(q) * step - want) <= step * (0.5 + 127 * 3 * 2.0 ** -24) + off).all()
    top = np.abs(want).reshape(M, -1, 32).max(2)
    assert (np.abs(np64(s) * 127 - top) <= off.reshape(M, -1, 32).max(2) + top * 2.0 ** -22).all()
    assert (np.abs(np64(q)).reshape(M, -1, 32).max(2) == 127).all()


@pytest.mark.parametrize("D,pad", [(128, 0), (128, 1), (17024, 0)])
def test_eight_bits_of_zeros_and_of_no_numbers(D, pad):
    M = 6
    h = torch.randn(M, D + pad, generator=gen_of(1), device="cuda")[:, :D]
    h[0] = 0
    h[1, 40] = float("nan")
    h[2, 70], h[2, 71] = float("inf"), -float("inf")
    h[3] *= 1e-38
    h[4, 32:64] = 0.0
    q, s = torch.zeros(M, D, dtype=torch.int8, device="cuda"), torch.zeros(M, D // 32, device="cuda")
    q4k.q4k_norm_residual_x8(M, D, None, 0, 0, None, None, 0.0, None, 0, 1.0, h, None, D + pad, q4k.Q4K_RES_FP32, 0, None, None, 0.0,
                             None, 0, q, s)
    wq, ws = step_ref.in_eight(h.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True) and np.isnan(ws[1, 1]) and np.isinf(ws[2, 2])
    wq[1, 32:64] = 0
    wq[2, 64:96] = 0
    wq[2, 70], wq[2, 71] = 127, -127
    assert np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("M,D,pad", [(4, 128, 0), (4, 128, 1), (2, 17024, 0), (800, 4096, 0), (2100, 64, 0)])
def test_eight_bits_of_the_smallest_values(M, D, pad):
    """Blocks whose largest value is so small that its 127th part is 0: zeros, as blocks of zeros are; a little more, and they are there."""
    k = torch.arange(M * D, device="cuda").view(M, D // 32, 32)
    top = 60 + k[:, :, :1] // 32 % 9               # in steps of 2^-149: 60 .. 68 (64 / 127 is the first above a half)
    h = (k * 37 % (2 * top + 1) - top).to(torch.int32)
    h[:, :, 5], h[:, :, 9] = 0, top[:, :, 0].to(torch.int32)
    flat = torch.zeros(M, D + pad, device="cuda")
    flat[:, :D] = (h.abs() | (h < 0).to(torch.int32) << 31).view(torch.float32).reshape(M, D)
    q, s = torch.full((M, D), 99, dtype=torch.int8, device="cuda"), torch.full((M, D // 32), -1.0, device="cuda")
    q4k.q4k_norm_residual_x8(M, D, None, 0, 0, None, None, 0.0, None, 0, 1.0, flat, None, D + pad, q4k.Q4K_RES_FP32, 0, None, None, 0.0,
                             None, 0, q, s)
    steps = s.view(torch.int32)
    assert torch.equal(steps, (top[:, :, 0] >= 64).to(torch.int32))
    assert torch.equal(q.view(M, D // 32, 32).int(), torch.where((steps > 0)[:, :, None], h.clamp(-127, 127), 0))


@pytest.mark.parametrize("M,pad", [(4, 0), (4, 1), (800, 0)])
def test_eight_bits_near_the_middle_and_over_all_sizes(M, pad):
    """Values at, just below and just above the middle between two whole numbers of steps, at every power of two; scales of any
    mantissa: the rule's bits."""
    D, g = 4096, gen_of(6)
    e = torch.randint(-140, 126, (M, D // 32, 1), generator=g, device="cuda").float()
    top = (1 + torch.rand(M, D // 32, 1, generator=g, device="cuda")) * torch.exp2(e)
    k = torch.randint(-127, 127, (M, D // 32, 32), generator=g, device="cuda").float()
    near = torch.randint(-2, 3, (M, D // 32, 32), generator=g, device="cuda")
    h = ((k + 0.5) * (top / 127.0))
    h = (h.view(torch.int32) + near.to(torch.int32)).view(torch.float32)  # neighbours of the middle
    h = torch.minimum(h.abs(), top) * torch.sign(h)
    h[:, :, 7:8] = top
    h[:, 0] = torch.where(near[:, 0] > 0, torch.full_like(k[:, 0], 127.0), k[:, 0] + 0.5)  # a scale of 1, exact ties
    h[:, 0, 7] = 127.0
    flat = torch.zeros(M, D + pad, device="cuda")
    flat[:, :D] = h.reshape(M, D)
    q, s = torch.zeros(M, D, dtype=torch.int8, device="cuda"), torch.zeros(M, D // 32, device="cuda")
    q4k.q4k_norm_residual_x8(M, D, None, 0, 0, None, None, 0.0, None, 0, 1.0, flat, None, D + pad, q4k.Q4K_RES_FP32, 0, None, None, 0.0,
                             None, 0, q, s)
    wq, ws = step_ref.in_eight(flat[:, :D].cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_eight_bits_go_into_the_product(ref, syn):
    """The output is what q4k_gemm_x8 takes: the same product as with the rule's bits from the host."""
    M, D, N = 5, 1024, 256
    p = make(M, D, torch.float32, None, False)
    h = torch.zeros(M, D, device="cuda")
    q, s = call(p, "rms", "none", None, h)
    w = syn.weights(syn.seed(0, 3), N, D)
    wd = torch.from_numpy(w).cuda()
    y, y2 = torch.zeros(M, N, device="cuda"), torch.zeros(M, N, device="cuda")
    q4k.q4k_gemm_x8(wd, N, D, q, s, M, y, N)
    hq, hs = step_ref.in_eight(h.cpu().numpy())
    q4k.q4k_gemm_x8(wd, N, D, torch.from_numpy(hq).cuda(), torch.from_numpy(hs).cuda(), M, y2, N)
    assert torch.equal(y, y2)
    want = ref.gemm_x8(w, N, D, hq, hs)
    assert np.abs(y.cpu().numpy() - want).max() <= np.abs(want).max() * 2e-4


def test_eight_bits_of_a_row_alone_in_batch_invariant_mode():
    p = make(400, 5120, BF, None, False)
    old = q4k.q4k_set_batch_invariant(True)
    try:
        q, s = call(p, "rms", "rms")
        one = dict(p, y=p["y"][37:38], r=p["r"][37:38])
        q1, s1 = call(one, "rms", "rms")
    finally:
        q4k.q4k_set_batch_invariant(old)
    assert torch.equal(q[37:38], q1) and torch.equal(s[37:38], s1)


def test_eight_bits_in_a_graph_and_in_place():
    p = make(300, 768, BF, None, False)
    r0 = p["r"].clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q, s = torch.zeros(300, 768, dtype=torch.int8, device="cuda"), torch.zeros(300, 24, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(p, "rms", "rms", None, p["r"], q=q, s=s)
    p["y"].normal_(generator=gen_of(4))
    graph.replay()
    torch.cuda.synchronize()
    r1 = torch.zeros_like(r0)
    q1, s1 = call(dict(p, r=r0), "rms", "rms", None, r1)
    assert torch.equal(q, q1) and torch.equal(s, s1) and torch.equal(p["r"], r1)
