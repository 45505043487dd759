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


