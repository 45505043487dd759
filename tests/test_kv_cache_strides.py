"""kv_cache() takes tensors whose dimensions of one element have any stride: torch counts such tensors as contiguous, so
a caller has no call that would change them."""
import pytest
import torch

import q4_weight_quantized_gb300 as q4k


def fields(c):
    return {n: getattr(c, n) for n, _ in c._fields_ if n not in ("k", "v", "page_table")}


@pytest.mark.parametrize("P,H,S,D", [(5, 1, 4, 64), (5, 3, 1, 64), (1, 2, 8, 128), (1, 1, 1, 64), (4, 2, 3, 256)])
@pytest.mark.parametrize("odd", [0, 1, 3, 1000003])
@pytest.mark.parametrize("B,M", [(3, 1), (1, 4), (1, 1), (2, 2)])
def test_strides_of_single_elements_do_not_count(P, H, S, D, odd, B, M):
    plain = torch.zeros(P, H, S, D, dtype=torch.bfloat16)
    strides = [odd if n == 1 else s for n, s in zip(plain.shape, plain.stride())]
    k = plain.as_strided(plain.shape, strides)
    table = torch.zeros(B, M, dtype=torch.int32)
    odd_table = table.as_strided((B, M), [odd if n == 1 else s for n, s in zip((B, M), (M, 1))])
    want = fields(q4k.kv_cache(plain, plain.clone(), table))
    for kk, vv in ((k, plain), (plain, k), (k, k)):
        got = fields(q4k.kv_cache(kk, vv, odd_table))
        for name, value in got.items():
            if name == "ld_table":
                assert value >= M and (B == 1 or value == M)
            elif not (name == "page_stride" and P == 1 or name == "head_stride" and H == 1 or name == "slot_stride" and S == 1):
                assert value == want[name], name
            elif name in ("page_stride", "head_stride", "slot_stride"):
                assert value >= D and value % 16 == 0, name


def test_strides_that_count_are_still_compared():
    k = torch.zeros(4, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q4k.kv_cache(k, torch.zeros(4, 3, 2, 64, dtype=torch.bfloat16).transpose(1, 2), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        q4k.kv_cache(k, k, torch.zeros(2, 2, dtype=torch.int32).t())
