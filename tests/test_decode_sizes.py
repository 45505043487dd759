"""Sizes that the decode-step operators cannot hold are refused on the host, whichever product of them is too large."""
import ctypes

import pytest

import q4_weight_quantized_gb300 as q4k

A = 1 << 20  # an aligned fake address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


def test_attn_workspace_does_not_wrap(lib):
    """The scores of 2^24 heads of 192 rows over 1.4 * 10^9 slots take more than 2^64 bytes: the size is 0, as for every
    call that is refused, and the call is refused."""
    c = q4k.KvCache(A, A, A, 1 << 20, 1 << 20, 64 * 16 * 256, 64 * 16, 64, 65535, 1 << 20, 1024, 256, 64, q4k.Q4K_KV_BF16, 1.0, 1.0)
    heads, n_q, rows = 256 * 64, 3, 192
    size = lambda ld: lib.q4k_attn_decode_workspace_size(ctypes.byref(c), heads, n_q, ld)  # noqa: E731
    score = 65535 * 256 * rows * 4
    over = -(-2 ** 64 // score)
    assert over < 2 ** 31
    for ld in (over, over + 1, 2 ** 31 - 1, over // 2 + 1):
        assert size(ld) == 0, ld
    for ld in (0, 1, 1 << 20, 4 * 10 ** 18 // score):
        assert score * ld < size(ld) < 2 ** 62, ld
    w = heads * 64
    for ld in (over, 2 ** 31 - 1):
        assert lib.q4k_attn_decode(ctypes.byref(c), A, A, w, heads, n_q, 0.1, 0.0, 0, A, w, A, ld, 1.0, A, 1 << 62, None) == q4k.Q4K_ERR_SHAPE
