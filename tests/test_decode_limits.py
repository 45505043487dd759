"""The decode-step operators at the largest sizes they take: caches of 2^31 - 2 slots, whose last tile, chunk and step end
beyond 2^31.  The slots share two pages."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from tests.test_decode_ops import F8, gen_of, np64

pytestmark = pytest.mark.gpu

PAGE, PAGES = 49981, 42966     # their product is 2^31 - 2
N = PAGE * PAGES
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    yield q4k.load()
    torch.cuda.empty_cache()


def test_attn_over_the_longest_cache():
    """Two new tokens over every slot; the last slot, which only the second one reads, holds a value without a number in
    the second call.

    Errors: a lane adds up the weights of N / (the shares, 2 at least an SM) / 4 warps / 8 lanes slots, one MMA accumulates
    those of N / shares / 4 warps / 16 slots; each addition rounds by 2^-24 of the sum, an MMA's two by 2^-22."""
    assert N == 2 ** 31 - 2
    g = gen_of(1)
    D, sms = 64, torch.cuda.get_device_properties(0).multi_processor_count
    k = torch.randn(2, 1, PAGE, D, generator=g, device="cuda").to(F8)
    v = (1 + 0.5 * torch.randn(2, 1, PAGE, D, generator=g, device="cuda")).to(F8)
    table = torch.zeros(1, PAGES, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.randn(1, 2, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    cache = q4k.kv_cache(k, v, table)
    size = q4k.q4k_attn_decode_workspace_size(cache, 1, 2, N)
    assert size >= 8 * N
    ws = torch.full((size + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    w = torch.zeros(N + GUARD, device="cuda")
    w[N:] = -1.0

    kk, vv, qq = np64(k).reshape(-1, D), np64(v).reshape(-1, D), np64(q).reshape(2, D)
    many = np.repeat([PAGES - 1.0, 1.0], PAGE)
    p = np.exp(kk @ qq.T * scale).T * many
    p[0, -1] = 0.0                                   # the first token does not see the second one's slot
    p /= p.sum(1, keepdims=True)
    want, mag, each = p @ vv, p @ np.abs(vv), p / many
    near = N / (2 * sms) / 4 * (2.0 ** -24 / 8 + 2.0 ** -22 / 16) + 2.0 ** -11

    def call():
        o = torch.full_like(q, float("nan"))
        q4k.q4k_attn_decode(cache, lens, q, D, 1, 2, scale, 0.0, 0, o, D, w, N, 1.0, ws, size)
        q4k.q4k_check_device()
        assert (ws[size:] == 0x5A).all() and (w[N:] == -1.0).all()
        return np64(o).reshape(2, D)

    got = call()
    assert (np.abs(got - want) <= mag * near + np.abs(want) * 2.0 ** -8).all()
    slots = w[:N].view(PAGES, PAGE)
    sum0, sum1 = (torch.from_numpy(x).cuda() for x in (each[:, :PAGE].sum(0), each[:, PAGE:].sum(0)))
    for at in (0, 1, PAGES // 2, PAGES - 3, PAGES - 2):
        assert ((slots[at].double() - sum0).abs() <= sum0 * near).all(), at
    assert torch.equal(slots[:-2].amin(0), slots[:-2].amax(0))    # every copy of a slot has the same score
    assert ((slots[-1].double() - sum1).abs() <= sum1 * near).all()
    v.view(torch.uint8)[1, 0, -1] = 0x7F             # NaN
    again = call()
    assert np.array_equal(again[0], got[0]) and np.isnan(again[1]).all()


@pytest.mark.parametrize("equal", [False, True])
def test_evict_from_the_longest_cache(equal):
    """Three slots of no weight leave, the last one among them; and of equal weights, all but the last 4096 slots."""
    g = gen_of(2)
    D = 64
    k, v = (torch.randn(2, 1, PAGE, D, generator=g, device="cuda").to(F8) for _ in range(2))
    table = torch.zeros(1, PAGES, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    w = torch.ones(N + GUARD, device="cuda")
    p = torch.full((N + GUARD,), -1, dtype=torch.int32, device="cuda")
    p[:N] = torch.arange(N, dtype=torch.int32, device="cuda")
    lens, new = torch.tensor([N], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    gone = [5, 123456789, N - 1]
    budget = 4096 if equal else N - 3
    if not equal:
        w[torch.tensor(gone, device="cuda")] = 0.0
    cache = q4k.kv_cache(k, v, table)
    size = q4k.q4k_kv_evict_workspace_size(cache, N)
    assert size >= 8 * (N // 2)
    ws = torch.full((size + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    rows = k.view(torch.uint8).clone()
    q4k.q4k_kv_evict(cache, lens, new, budget, 0, 0, w, p, w, p, N, ws, size)
    q4k.q4k_check_device()
    assert new.tolist() == [budget] and (ws[size:] == 0x5A).all()
    del ws
    want = torch.full((N + GUARD,), -1, dtype=torch.int32, device="cuda")
    want[:N] = torch.arange(N, dtype=torch.int32, device="cuda")
    weights = torch.ones(N + GUARD, device="cuda")
    now = k.view(torch.uint8)
    if equal:
        want[:4096] = torch.arange(N - 4096, N, dtype=torch.int32, device="cuda")
        assert torch.equal(now[0, 0, :4096], rows[1, 0, PAGE - 4096:])
    else:
        weights[torch.tensor(gone, device="cuda")] = 0.0
        for at, j in zip(gone[:2], (N - 3, N - 2)):
            want[at], weights[at] = j, 1.0
            assert torch.equal(now[0, 0, at % PAGE], rows[1, 0, j % PAGE])
    assert torch.equal(p, want) and torch.equal(w, weights)
