"""q4k_norm_residual's ring of rows when a wait runs out: the limit is made so short that the waits give up while rows
are still being copied (no fault, no hang).  The kernel then leaves as a whole after the copies in flight have landed,
the status is reported and cleared, and the next call is right."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    q4k.load()
    yield
    q4k.q4k_set_gemv_wait_limit_ns(0)


@pytest.mark.parametrize("M,D,post,pre", [(4000, 5120, 1, 1), (4000, 768, 0, 2), (700, 10240, 2, 0), (200, 2048, 2, 1)])
def test_a_wait_for_a_row_runs_out(M, D, post, pre):
    g = torch.Generator(device="cuda").manual_seed(D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    y, r, w = rnd(M, D), rnd(M, D), rnd(D)
    out, x = torch.zeros(M, D, device="cuda"), torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")

    def call():
        q4k.q4k_norm_residual(M, D, y, D, post, w, None, 1e-6, None, 0, 0.5, r, out, D, q4k.Q4K_RES_FP32, pre, w, None, 1e-6, x, D)

    q4k.q4k_check_device()
    try:
        assert q4k.q4k_set_gemv_wait_limit_ns(2) == 0
        for _ in range(3):
            call()
        with pytest.raises(q4k.Q4KError) as err:
            q4k.q4k_check_device()
        assert err.value.status == q4k.Q4K_ERR_TIMEOUT
        q4k.q4k_check_device()
    finally:
        q4k.q4k_set_gemv_wait_limit_ns(0)
    call()
    q4k.q4k_check_device()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    h, want = R.norm_residual(f(y), post, f(w), None, 1e-6, None, 0.5, f(r), pre, f(w), None, 1e-6)
    assert np.linalg.norm(f(out) - h) <= np.linalg.norm(h) * 1e-6
    assert np.linalg.norm(f(x) - want) <= np.linalg.norm(want) * (2.0 ** -9 + 1e-6)
