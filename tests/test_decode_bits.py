"""What the decode-step operators promise of their bits: e4m3 caches and queries of any size, and rows that do not depend
on the rest of a call in batch-invariant mode."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R
from tests.test_decode_ops import BF, F8, gen_of, np64, pool, run_attn, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


@pytest.mark.parametrize("e", [-126, -120, -115, -112, -111, -100, 120])
def test_attn_e4m3_queries_down_to_the_smallest(e):
    """Queries whose largest value is near either end of bf16's range (below 2^-126 with the bits that bf16 has there).
    Errors as in the other attention tests; p enters the second product to 2^-11."""
    g = gen_of(13)
    D, n = 64, 128
    k, v = pool((8, 1, 16, D), F8, "phsd", g)
    table = table_of(1, 8, 8, g)
    q = (torch.randn(1, 1, 3, D, generator=g, device="cuda") * 2.0 ** e).to(BF)
    scale = 2.0 ** min(-1 - e, 125)
    o = run_attn(k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), q, 1, scale)
    want, _, mag, big = R.attn_decode(np64(k), np64(v), table.cpu().numpy(), [n], np64(q), 1, scale)
    assert np.abs(want - np64(v).reshape(-1, D)[:n].mean(0)).max() > 0.1  # (not what equal scores give)
    err = (D * 2.0 ** -24 + 2.0 ** -20) * big[..., None]
    assert (np.abs(np64(o) - want) <= mag * (2.2 * err + 2.0 ** -14 + 2.0 ** -11) + np.abs(want) * 2.0 ** -8 + 2.0 ** -20).all()


@pytest.mark.parametrize("D", [8, 64, 300, 768, 1000, 5120, 10240, 12288])
@pytest.mark.parametrize("post,pre,gate,res,bias", [
    (1, 1, "row", BF, False), (2, 1, None, torch.float32, True), (0, 2, "all", torch.float32, True), (1, 0, "all", BF, True),
    (1, 2, "row", torch.float32, True)])
def test_norm_rows_do_not_depend_on_the_batch(D, post, pre, gate, res, bias):
    """Batch-invariant mode: a row has the same bits alone and among many."""
    g = gen_of(D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    M = 2100 if D <= 1000 else 500
    y, r = rnd(M, D) * 3, (rnd(M, D) * 2).to(res)
    w1, w2 = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
    b1, b2 = (rnd(D), rnd(D)) if bias else (None, None)
    gt = None if gate is None else rnd(1 if gate == "row" else M, D)
    kind = q4k.Q4K_RES_FP32 if res == torch.float32 else q4k.Q4K_RES_BF16

    def call(lo, hi):
        out, x = torch.zeros(hi - lo, D, dtype=res, device="cuda"), torch.zeros(hi - lo, D, dtype=BF, device="cuda")
        q4k.q4k_norm_residual(hi - lo, D, y[lo:hi], D, post, w1, b1, 1e-5, gt[lo:hi] if gate == "all" else gt,
                              D if gate == "all" else 0, 0.7, r[lo:hi], out, D, kind, pre, w2, b2, 1e-6, x, D)
        return out, x

    was = q4k.q4k_set_batch_invariant(True)
    try:
        out, x = call(0, M)
        for lo, hi in [(0, 1), (1, 2), (M - 1, M), (7, 24), (100, 251), (100, 252), (100, 253), (150, 453)]:
            some, xs = call(lo, hi)
            assert torch.equal(some, out[lo:hi]) and torch.equal(xs, x[lo:hi]), (lo, hi)
    finally:
        q4k.q4k_set_batch_invariant(was)
    q4k.q4k_check_device()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("D,G,n", [(64, 4, 2), (64, 12, 6), (64, 32, 40), (128, 5, 4), (128, 9, 18), (128, 24, 2), (256, 8, 10), (256, 16, 64)])
def test_attn_weights_keep_their_bits_in_the_second_product(dtype, D, G, n):
    """Values of +1 and -1: what is left of a sum of weights that nearly cancel shows how far each is off.

    Errors: a score by e (D additions of products that sum to big at most, the exponential), a weight then by e^(2 e), and by
    2^-15 at most for its two 16-bit halves and the sums; o's own rounding is 2^-8 of what is left."""
    g = gen_of(D + n)
    B, Hkv, page = 24, 2, 16
    per = -(-n // page)
    k, v = pool((B * per, Hkv, page, D), dtype, "phsd", g)
    v.copy_(torch.where(torch.rand(v.shape, generator=g, device="cuda") < 0.5, 1.0, -1.0))
    table = table_of(B, per, B * per, g)
    q = torch.randn(B, 1, Hkv * G, D, generator=g, device="cuda").to(BF)
    o = run_attn(k, v, table, torch.full((B,), n, dtype=torch.int32, device="cuda"), q, 1, D ** -0.5)
    want, _, mag, big = R.attn_decode(np64(k), np64(v), table.cpu().numpy(), [n] * B, np64(q), 1, D ** -0.5)
    e = (D * 2.0 ** -24 + 2.0 ** -20) * big[..., None]
    assert (np.abs(np64(o) - want) <= mag * (2.2 * e + 2.0 ** -15) + np.abs(want) * 2.0 ** -8 + 1e-30).all()
