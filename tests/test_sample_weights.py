"""The whole-number weights of q4k_sample, to the last unit: draws at the edge of a token's weight."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R
from tests.test_decode_ops import gen_of, run_sample

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


# without any cut; top-k, top-p or min-p that keep the first two of three tokens, each by another route
ROUTES = [(2, 0, 1.0, 0.0), (3, 2, 1.0, 0.0), (3, 0, 1.0, 0.05), (3, 2, 0.999, 0.0), (3, 0, 0.999, 0.05), (3, 0, 0.999, 0.0),
          (20000, 2, 1.0, 0.0), (20000, 0, 1.0, 0.05), (20000, 0, 0.999, 0.0), (20000, 200, 0.999, 0.0), (20000, 0, 1.0, 0.0)]


@pytest.mark.parametrize("V,k,p,m", ROUTES)
@pytest.mark.parametrize("t", [1.0, 0.7])
def test_a_draw_at_the_edge_of_a_weight(V, k, p, m, t):
    """Token 0 at a distance from the largest, token 1: the last random number that falls on token 0 and the first that
    falls on token 1.  Their targets are 1.5 to 2 units of the weight apart, so a unit more or less shows on many of them."""
    M = 2048 if V < 100 else 256
    g = gen_of(V + k)
    z = torch.full((M, V), -200.0, device="cuda")
    z[:, 1] = torch.randn(M, generator=g, device="cuda") * 3
    z[:, 0] = z[:, 1] - torch.rand(M, generator=g, device="cuda") * 1.5 * t
    rows = z.cpu().numpy()
    f = np.float32
    c = f(f(f(1) / f(t)) * f(1.4426950408889634))
    w = R.sample_weight((rows[:, 1] - rows[:, 0]) * c)
    one = 1 << 40
    first = np.array([-(-int(x) * 2 ** 24 // (int(x) + one)) for x in w])    # the first number whose target is not below w
    for step, want in ((-1, 0), (0, 1)):
        u = (first + step) / 2.0 ** 24
        token, prob = run_sample(z, t, k, p, m, u)
        assert token == [want] * M
        exact = np.where(want, one, w) / (w.astype(np.float64) + one)
        # the sum's and the quotient's rounding
        assert (np.abs(np.array(prob) - exact) <= exact * (2 * 2.0 ** -24 + 2.0 ** -47)).all()
    for i in (0, M - 1):
        assert R.sample(rows[i], float(f(t)), k, float(f(p)), float(f(m)), float(first[i] / 2.0 ** 24))[0] == 1


@pytest.mark.parametrize("V", [15, 700, 9001])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (97, 0.99, 0.0), (40, 1.0, 0.0), (0, 0.9, 0.0), (0, 0.99, 0.1), (0, 1.0, 0.02)])
def test_probabilities_to_two_roundings(V, k, p, m):
    """prob is the exact weight over the exact sum, each rounded (a weight has 24 bits), and their quotient."""
    g = gen_of(V)
    z = torch.randn(24, V, generator=g, device="cuda") * 2.5
    t, u = [1.0, 0.7, 0.3, 2.0, 50.0, 1.3] * 4, torch.rand(24, generator=g, device="cuda").tolist()
    token, prob = run_sample(z, t, k, p, m, u)
    rows, f = z.cpu().numpy(), np.float32
    for i in range(24):
        want, exact = R.sample(rows[i], float(f(t[i])), k, float(f(p)), float(f(m)), float(f(u[i])))
        assert token[i] == want and abs(prob[i] - exact) <= exact * (2 * 2.0 ** -24 + 2.0 ** -47), (i, prob[i], exact)
