"""Attention of chunks where a CTA has many units of one or two tiles of slots each: what is kept by unit (the factors of an e4m3
cache's queries, the marks of values without a number) belongs to the unit that it is used for.  Tolerances are those of
test_attn_chunk.py."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from tests.test_attn_chunk import check, make, reference, run
from tests.test_decode_ops import BF, F8, gen_of, lib  # noqa: F401

pytestmark = pytest.mark.gpu
AT = 5  # the value of a head that is spoilt


def batch(D, dtype, B, longest, gen, window=0):
    """Requests of up to `longest` slots, whose queries' magnitudes differ by powers of two from one request to the next."""
    lens = [1 + i * 29 % longest for i in range(B)]
    new = [min(n, 1 + i * 7 % 30) for i, n in enumerate(lens)]
    k, v, table, ks, vs, starts, q = make(D, dtype, 16, "phsd", 2, 4, new, lens, gen, spare=0)
    of = np.repeat(np.arange(B), new)
    q = (q.float() * torch.exp2(-torch.tensor(of * 5 % 7, device="cuda").float())[:, None, None]).to(BF)
    return k, v, table, ks, vs, starts, q, lens, new


@pytest.mark.parametrize("D,dtype,B,longest,window", [
    (256, F8, 700, 64, 0), (256, F8, 500, 128, 40), (256, BF, 700, 64, 0), (128, F8, 700, 128, 0), (64, F8, 600, 128, 30),
    (128, BF, 500, 256, 0), (64, BF, 700, 128, 0),
])
@pytest.mark.parametrize("spoilt", [False, True])
def test_many_short_units(D, dtype, B, longest, window, spoilt):
    g = gen_of(D + B + longest)
    k, v, table, ks, vs, starts, q, lens, new = batch(D, dtype, B, longest, g)
    want = reference(k, v, table, starts, lens, q, D ** -0.5, 0.0, window, ks, vs)
    none = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    if spoilt:  # in some requests a value that is none, which the first of the new tokens do not see
        nan = torch.full((1,), float("nan"), device="cuda").to(dtype)
        view = (lambda x: x.view(torch.uint8)) if dtype == F8 else (lambda x: x)
        for b in range(0, B, 9):
            j = lens[b] - (new[b] + 1) // 2
            view(v)[int(table[b, j // 16]), 0, j % 16, AT] = view(nan)
            ends = np.arange(lens[b] - new[b] + 1, lens[b] + 1)
            sees = (j < ends) & ((j >= ends - window) if window else True)
            none[starts[b]:starts[b + 1], :4, AT] = torch.tensor(sees, device="cuda")[:, None]
        assert none.any()
    for _ in range(3):
        o = run(k, v, table, starts, lens, q, D ** -0.5, 0.0, window, ks, vs)
        q4k.q4k_check_device()
        assert torch.equal(torch.isnan(o), none)
        o[none] = want[0][none].to(BF)
        check(o, want, D, dtype == F8)
