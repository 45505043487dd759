"""Attention of chunks with soft caps of any size.  The tolerances of test_attn_chunk.py count errors of a score as shares of the
score itself, whatever the cap: c tanh(s / c) must not lose the scores that are small beside c."""
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from tests.test_attn_chunk import check, make, reference, run
from tests.test_decode_ops import BF, F8, gen_of, lib  # noqa: F401

pytestmark = pytest.mark.gpu
SHAPES = [  # D, type, Hkv, G, new tokens, lengths, window: small calls, calls of many sequences or tiles, units of many CTAs
    (128, BF, 2, 4, [33, 1], [200, 77], 0), (128, BF, 2, 4, [900, 1], [3000, 500], 0), (128, F8, 1, 5, [600, 3], [1000, 4000], 0),
    (64, F8, 1, 8, [300], [900], 70), (64, BF, 1, 1, [40] * 35, [200] * 35, 0), (256, BF, 1, 4, [700, 40], [1500, 2500], 0),
    (256, F8, 1, 2, [100], [700], 0), (128, BF, 1, 2, [90], [20000], 0),
]


@pytest.mark.parametrize("D,dtype,Hkv,G,new,lens,window", SHAPES)
@pytest.mark.parametrize("softcap", [3.0, 63.0, 100.0, 511.0, 1e3, 1e5, 1e8, 1e30, 3.4e38])
def test_caps_of_any_size(D, dtype, Hkv, G, new, lens, window, softcap):
    g = gen_of(D + Hkv + len(new))
    k, v, table, ks, vs, starts, q = make(D, dtype, 16, "phsd", Hkv, G, new, lens, g)
    for scale in (1.5 * D ** -0.5, -D ** -0.5):
        o = run(k, v, table, starts, lens, q, scale, softcap, window, ks, vs)
        q4k.q4k_check_device()
        check(o, reference(k, v, table, starts, lens, q, scale, softcap, window, ks, vs), D, dtype == F8)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("softcap", [300.0, 4000.0, 1e5])
def test_scores_on_both_sides_of_a_large_cap(dtype, softcap):
    """Few slots near the cap, many far below it, in units that see all of a tile and units that do not."""
    g = gen_of(int(softcap))
    D, new, lens = 128, [300, 40], [700, 40]
    k, v, table, ks, vs, starts, q = make(D, dtype, 16, "phsd", 1, 2, new, lens, g)
    scale = 0.25 * softcap / 300 * ks   # scores of up to about the cap: their differences matter where they are small
    q = (q.float() * torch.exp2(-torch.randint(0, 14, (q.shape[0], 1, 1), generator=g, device="cuda").float())).to(BF)
    o = run(k, v, table, starts, lens, q, scale, softcap, 0, ks, vs)
    q4k.q4k_check_device()
    check(o, reference(k, v, table, starts, lens, q, scale, softcap, 0, ks, vs), D, dtype == F8, norm=False)


@pytest.mark.parametrize("new,lens", [([40], [170]), ([900, 1], [3000, 500])])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_the_smallest_caps(new, lens, dtype):
    """No score is left: every slot that a row sees counts the same, those of keys or queries of 0, too."""
    g = gen_of(33)
    k, v, table, _, _, starts, q = make(128, dtype, 16, "phsd", 2, 4, new, lens, g)
    (k.view(torch.uint8) if dtype == F8 else k)[int(table[0, 2])] = 0
    q[3] = 0
    for softcap, scale in ((1e-38, 50.0), (1e-42, 50.0), (1e-38, -1e30)):
        o = run(k, v, table, starts, lens, q, scale, softcap)
        check(o, reference(k, v, table, starts, lens, q, 0.0), 128, dtype == F8)
