"""Low-rank adapters beside a projection, against the plain 64-bit form.

Products are exact; a value is the sum of y, and of R inner values times b, each a sum of K products.  With every fp32 addition
rounded to 2^-24 of a partial sum that is at most the sum of the magnitudes `mag`, and at most (K / 16 + R / 16 + 30) such
additions on the way of a product (MMA steps, and the joins of warps, parts, pieces and y; the order inside an MMA step is
counted as 16), the error is at most mag * (K / 16 + R + 60) * 2^-24."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import step_ref
from tests.test_decode_ops import BF, gen_of, lib, np64  # noqa: F401

pytestmark = pytest.mark.gpu


def make(nA, N, K, R, T, ids, seed=0, pad_x=0, pad_y=0, off_y=0):
    g = gen_of(seed + N + K + R + T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = torch.full((T, K + pad_x), float("nan"), dtype=BF, device="cuda")
    x[:, :K] = rnd(T, K)
    y = torch.full((T * (N + pad_y) + off_y,), 7.0, device="cuda")[off_y:].view(T, N + pad_y)
    y[:, :N] = rnd(T, N)
    if ids == "mixed":
        i = torch.randint(-1, nA, (T,), generator=g, device="cuda")
    elif ids == "runs":
        i = torch.arange(T, device="cuda") * nA // T
    else:
        i = torch.full((T,), ids, device="cuda")
    ranks = torch.randint(0, R + 1, (nA,), generator=g, device="cuda").to(torch.int32)
    a, b = (rnd(nA, R, K) * K ** -0.5).to(BF), rnd(nA, N, R).to(BF)
    # what lies beyond a rank has no part
    for j in range(nA):
        a[j, int(ranks[j]):] = float("nan")
        b[j, :, int(ranks[j]):] = float("inf")
    return dict(a=a, b=b, ranks=ranks, scales=rnd(nA), ids=i.to(torch.int32), x=x, y=y, N=N, K=K, R=R, T=T)


def copy_of(y):
    """A copy that lies as many values off 16 bytes as y does."""
    off = y.data_ptr() // 4 % 4
    return torch.empty(y.numel() + off, device="cuda")[off:].view(y.shape).copy_(y)


def call(p, y, ranks=True, scales=True, stream=None, ws=None):
    nA = p["a"].shape[0]
    size = q4k.q4k_lora_add_workspace_size(nA, p["N"], p["K"], p["R"], p["T"])
    assert size > 0
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    q4k.q4k_lora_add(nA, p["N"], p["K"], p["R"], p["a"], p["b"], p["ranks"] if ranks else None, p["scales"] if scales else None, p["ids"],
                     p["x"], p["T"], p["x"].stride(0), y, y.stride(0), ws, ws.numel(), stream)
    return y


def check(p, got, ranks=None, scales=None):
    N, K, R = p["N"], p["K"], p["R"]
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    want, mag = step_ref.lora_add(f(p["a"]), f(p["b"]), p["ranks"].tolist() if ranks is None else ranks,
                                  p["scales"].tolist() if scales is None else scales, p["ids"].tolist(), f(p["x"])[:, :K], f(p["y"])[:, :N])
    tol = mag * (K / 16 + R + 60) * 2.0 ** -24
    assert (np.abs(np64(got)[:, :N] - want) <= tol).all(), float((np.abs(np64(got)[:, :N] - want) / tol).max())
    bare = ((p["ids"] < 0) | (p["ids"] >= p["a"].shape[0])).cpu().numpy()
    assert np.array_equal(np64(got)[bare], np64(p["y"])[bare])
    assert (got[:, N:] == 7.0).all()


SHAPES = [  # nA, N, K, R, T, ids, pads and offset of y
    (1, 64, 64, 8, 1, 0, 0, 0, 0), (3, 50, 72, 8, 5, "mixed", 8, 3, 1), (4, 257, 1000, 16, 17, "mixed", 0, 0, 0),
    (24, 512, 2048, 16, 32, "mixed", 0, 0, 0), (2, 1000, 520, 24, 33, 1, 16, 4, 0), (5, 300, 768, 32, 64, "runs", 0, 0, 0),
    (7, 129, 136, 48, 100, "mixed", 0, 3, 0), (3, 640, 512, 64, 191, "mixed", 0, 0, 0), (2, 200, 264, 128, 192, "mixed", 0, 0, 0),
    (2, 200, 264, 128, 193, "mixed", 0, 0, 0), (40, 100, 128, 16, 700, "mixed", 0, 0, 2), (3, 333, 256, 72, 1000, "runs", 0, 0, 0),
    (1, 96, 5120, 16, 400, 0, 0, 0, 0), (1024, 64, 64, 8, 3000, "mixed", 0, 0, 0),
    (40, 100, 136, 16, 7, "mixed", 0, 0, 0), (1000, 48, 64, 64, 150, "mixed", 0, 0, 3), (3, 5120, 64, 16, 2, "mixed", 0, 0, 0), (6, 17, 2048, 40, 500, "mixed", 0, 0, 0)]


@pytest.mark.parametrize("nA,N,K,R,T,ids,pad_x,pad_y,off_y", SHAPES)
def test_lora(nA, N, K, R, T, ids, pad_x, pad_y, off_y):
    p = make(nA, N, K, R, T, ids, pad_x=pad_x, pad_y=pad_y, off_y=off_y)
    got = call(p, copy_of(p["y"]))
    assert got.data_ptr() % 16 == 4 * off_y
    q4k.q4k_check_device()
    check(p, got)
    assert torch.equal(call(p, copy_of(p["y"])), got)  # the same call, the same bits


def test_lora_ids_out_of_range_with_more_adapters_than_tokens():
    p = make(50, 64, 64, 8, 6, "mixed")
    p["ids"][:] = torch.tensor([3, 50, 3, -1, 2 ** 31 - 1, 49], device="cuda")
    check(p, call(p, p["y"].clone()))
    with pytest.raises(q4k.Q4KError) as e:
        q4k.q4k_check_device()
    assert e.value.status == q4k.Q4K_ERR_INDEX


@pytest.mark.parametrize("T", [40, 300])
def test_lora_defaults_and_ids_out_of_range(T):
    p = make(3, 128, 256, 16, T, "mixed")
    p["a"], p["b"] = (torch.nan_to_num(p[n], nan=0.5, posinf=0.25) for n in "ab")
    got = call(p, p["y"].clone(), ranks=False, scales=False)
    check(p, got, ranks=[16] * 3, scales=[1.0] * 3)
    q4k.q4k_check_device()
    p["ids"][T // 2], p["ranks"][0], p["ranks"][1] = 3, 99, -2
    p["a"][2, int(p["ranks"][2]):] = float("nan")
    check(p, call(p, p["y"].clone()))
    with pytest.raises(q4k.Q4KError) as e:
        q4k.q4k_check_device()
    assert e.value.status == q4k.Q4K_ERR_INDEX
    p["ids"].fill_(-1)
    assert torch.equal(call(p, p["y"].clone()), p["y"])
    q4k.q4k_check_device()


@pytest.mark.parametrize("T", [30, 400])
def test_lora_what_is_not_a_number_keeps_to_its_token(T):
    p = make(2, 130, 256, 16, T, "mixed")
    p["ids"][:] = torch.arange(T, device="cuda") % 2
    p["ranks"][:] = 16
    p["a"], p["b"] = (torch.nan_to_num(p[n], nan=0.5, posinf=0.25) for n in "ab")
    clean = call(p, p["y"].clone())
    p["x"][5, 3], p["x"][9, 4] = float("nan"), float("inf")
    got = call(p, p["y"].clone())
    rest = [t for t in range(T) if t not in (5, 9)]
    assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[5]).all() and not torch.isfinite(got[9]).any()


def test_lora_large_and_small_values():
    """Inner values near the ends of the fp32 range keep their exact pieces."""
    p = make(1, 64, 64, 8, 3, 0)
    p["ranks"][:], p["scales"][:] = 8, 1.0
    p["a"].fill_(1.0), p["b"].fill_(1.0)
    p["y"].zero_()
    p["x"].zero_()
    p["x"][0, 0], p["x"][0, 1] = 2.0 ** 100, 2.0 ** 80
    p["x"][1, 0], p["x"][1, 1] = 2.0 ** -60, 2.0 ** -80
    p["x"][2, 0] = 3e37
    got = call(p, p["y"].clone())
    assert (got[0] == 8 * (2.0 ** 100 + 2.0 ** 80)).all() and (got[1] == 8 * (2.0 ** -60 + 2.0 ** -80)).all()
    assert (np.abs(np64(got[2]) / (8 * float(p["x"][2, 0])) - 1) <= 2.0 ** -20).all()


def test_lora_offsets_past_32_bits():
    """Rows of x and y more than 2^32 bytes apart."""
    N, K, R, T = 64, 64, 8, 3
    g = gen_of(5)
    x = torch.empty(2 * (1 << 30) + K + 8, dtype=BF, device="cuda").as_strided((T, K), (1 << 30, 1))
    y = torch.empty(2 * (1 << 30) + N, device="cuda").as_strided((T, N), (1 << 30, 1))
    x.copy_(torch.randn(T, K, generator=g, device="cuda"))
    y.copy_(torch.randn(T, N, generator=g, device="cuda"))
    p = make(2, N, K, R, T, "mixed")
    p["ids"][:] = torch.tensor([1, 0, 1], device="cuda")
    p.update(x=x, y=y.clone())
    call(p, y)
    q4k.q4k_check_device()
    check(dict(p, x=x.contiguous()), y.contiguous())


@pytest.mark.parametrize("T", [50, 500])
def test_lora_on_another_stream_in_a_graph_and_after_a_product(T, ref, syn):
    """Beside the projection that it belongs to, on one stream; replayed with other ids and inputs."""
    N, K = 256, 512
    w = syn.weights(syn.seed(0, 1), N, K)
    wd = torch.from_numpy(w).cuda()
    p = make(4, N, K, 16, T, "mixed")
    y = torch.empty(T, N, device="cuda")
    size = q4k.q4k_gemm_workspace_size(T, N, K)
    gws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    ws = torch.empty(q4k.q4k_lora_add_workspace_size(4, N, K, 16, T), dtype=torch.uint8, device="cuda")

    def step(stream):
        q4k.q4k_gemm(wd, N, K, p["x"], T, K, y, N, gws, size, stream)
        call(p, y, stream=stream, ws=ws)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(None)
    for seed in range(3):
        p["ids"].copy_(torch.randint(-1, 4, (T,), generator=gen_of(seed), device="cuda"))
        p["x"].copy_(torch.randn(T, K, generator=gen_of(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        base = torch.empty(T, N, device="cuda")
        q4k.q4k_gemm(wd, N, K, p["x"], T, K, base, N, gws, size)
        check(dict(p, y=base), y)
    q4k.q4k_check_device()


@pytest.mark.parametrize("nA,N,K,R,T,ids,pad_y,off_y", [
    (1024, 300, 64, 16, 192, 1023, 0, 0), (1024, 72, 64, 8, 192, "runs", 0, 0), (40, 6526, 768, 16, 83, 5, 0, 0),
    (10, 11559, 512, 128, 15, 3, 1, 0), (30, 20000, 64, 8, 3, "mixed", 0, 0), (8, 17, 4096, 64, 150, "runs", 0, 0),
    (16, 1024, 264, 128, 100, "runs", 0, 0), (6, 2000, 96, 32, 190, "mixed", 4, 0), (9, 640, 8192, 64, 1, 8, 0, 0),
    (1, 2048, 328, 128, 838, "runs", 0, 0), (3, 515, 4096, 8, 1028, "runs", 0, 1), (20, 333, 336, 64, 700, "mixed", 0, 0),
    (2, 1030, 200, 32, 500, "mixed", 2, 0), (1, 128, 64, 40, 194, 0, 0, 0),
])
def test_few_adapters_share_the_gpu(nA, N, K, R, T, ids, pad_y, off_y):
    """Clusters by groups of tokens and parts of the columns; tiles over several CTAs; pieces split once a CTA."""
    p = make(nA, N, K, R, T, ids, pad_y=pad_y, off_y=off_y)
    got = call(p, copy_of(p["y"]))
    check(p, got)
    assert torch.equal(call(p, copy_of(p["y"])), got)
    q4k.q4k_check_device()


def test_the_first_call_of_a_process_leaves_no_error_behind():
    code = """
import torch, q4_weight_quantized_gb300 as q4k
for R in (128, 64, 32, 16, 8):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    y, ws = torch.ones(4, 64, device="cuda"), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    q4k.q4k_lora_add(2, 64, 64, R, z(2, R, 64), z(2, 64, R), None, None, torch.zeros(4, dtype=torch.int32, device="cuda"), z(4, 64), 4, 64,
                     y, 64, ws, ws.numel(), None)
    assert float((y + 1).sum()) == 512  # (a launch that looks for errors)
q4k.q4k_check_device()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("nA,N,K,R,T", [(2, 130, 64, 8, 5), (3, 300, 136, 16, 40), (2, 257, 64, 32, 100), (2, 96, 72, 64, 190), (1, 640, 64, 128, 33),
                                        (3, 200, 64, 8, 500), (2, 333, 136, 16, 700), (2, 128, 64, 24, 400), (2, 260, 64, 64, 300), (3, 96, 72, 128, 600)])
@pytest.mark.parametrize("whole", [False, True])
def test_lora_infinities_within_the_rank(nA, N, K, R, T, whole):
    """An infinite b times an inner value is infinite whatever the value's bits (so that parts of it may be 0); 0 * infinity is no
    number; other columns are what they are without."""
    p = make(nA, N, K, R, T, "mixed", seed=7)
    p["ranks"][:] = R - 3
    p["a"], p["b"] = (torch.nan_to_num(p[n], nan=0.5, posinf=0.25) for n in "ab")
    p["scales"][:] = torch.tensor([1.0, -0.5, 2.0])[:nA]
    if not whole:  # inner values of 8 bits: one product each
        at = torch.arange(T, device="cuda") % K
        value = torch.where(torch.arange(T, device="cuda") % 3 == 0, -2.0, 0.5)
        p["x"].zero_()
        p["x"][torch.arange(T, device="cuda"), at] = value.to(BF)
        p["x"][T // 2] = 0
    inf = float("inf")
    for i, (n, r, v) in enumerate([(1, 0, inf), (2, R - 4, -inf), (N - 1, R // 2, inf), (N // 2, 1, float("nan")), (N // 2 + 3, 2, inf)]):
        p["b"][i % nA, n, r] = v
    p["b"][0, 17, 3:5] = torch.tensor([inf, -inf])
    got = np64(call(p, p["y"].clone()))
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    with np.errstate(invalid="ignore"):
        want = step_ref.lora_add(f(p["a"]), f(p["b"]), p["ranks"].tolist(), p["scales"].tolist(), p["ids"].tolist(), f(p["x"])[:, :K],
                                 f(p["y"]))[0]
    odd = ~np.isfinite(want)
    assert odd.any() and np.isinf(want).any()
    assert np.array_equal(np.nan_to_num(want[odd], nan=7.0, posinf=8.0, neginf=9.0), np.nan_to_num(got[odd], nan=7.0, posinf=8.0, neginf=9.0))
    p["b"] = torch.nan_to_num(p["b"], nan=0.0, posinf=0.0, neginf=0.0)
    clean = np64(call(p, p["y"].clone()))
    assert np.array_equal(got[~odd], clean[~odd])
    q4k.q4k_check_device()


@pytest.mark.parametrize("R,T", [(8, 5), (16, 60), (64, 100), (128, 30), (8, 400), (16, 500), (32, 300), (128, 250)])
def test_lora_infinite_inner_values_and_infinities(R, T):
    """One infinite x and adapters of rank 1: infinity times each b, an infinite one or 0 included."""
    p = make(2, 100, 64, R, T, "mixed", seed=9)
    p["ranks"][:] = 1
    p["a"][:, 0, 5], p["b"][:, 3, 0], p["b"][:, 4, 0] = 2.0, float("inf"), -float("inf")
    p["b"][:, 5, 0], p["b"][0, 6, 0] = 0.0, float("nan")
    p["x"][::3, 5] = float("inf")
    p["x"][1::3, 5] = -float("inf")
    got = np64(call(p, p["y"].clone()))
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    with np.errstate(invalid="ignore"):
        want = step_ref.lora_add(f(p["a"]), f(p["b"]), [1, 1], p["scales"].tolist(), p["ids"].tolist(), f(p["x"])[:, :64], f(p["y"])[:, :100])[0]
    odd = ~np.isfinite(want)
    assert np.isinf(want[:, 3]).any() and np.isnan(want[:, 5]).any() and (~odd).any()
    assert np.array_equal(np.isfinite(got), ~odd)
    assert np.array_equal(np.nan_to_num(want[odd], nan=7.0, posinf=8.0, neginf=9.0), np.nan_to_num(got[odd], nan=7.0, posinf=8.0, neginf=9.0))
    q4k.q4k_check_device()
