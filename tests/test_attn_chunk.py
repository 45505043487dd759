"""Attention of chunks of new tokens on the GPU against the plain 64-bit form.

Tolerances are bounds on the kernel's roundings.  With e = the error of a score (D fp32 additions of products that sum to at most
`big` in magnitude, the scale's product and the exponential, 2^-21 of the score together), every weight is off by at most a factor
e^(2 e); it enters the second product rounded to bf16 (2^-8; f16 for an e4m3 cache: 2^-11, and below f16's normal range half
a step of 2^-24 of 2^7 times the weight, the row's largest being at least 1: 2^-32 of it for each slot, so 2^-32 sum_j |v_j| where
p is tiny everywhere but at slots whose value is 0); sums over slots add 2^-24 per addition, at most 2^-11 for the lengths here; o is rounded
to bf16 (2^-8).  Over a whole output the roundings of the weights and of o are independent: their 2-norm is at most
sqrt(2) 2^-8 of o's for values of no common sign."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import step_ref
from tests.test_decode_ops import BF, F8, gen_of, lib, np64, pool, table_of  # noqa: F401

pytestmark = pytest.mark.gpu
GUARD = 77.0


def reference(k, v, table, starts, lens, q, scale, softcap=0.0, window=0, ks=1.0, vs=1.0):
    """o, sum_j p_j |v_j|, max_j scale sum_d |q_d k_jd| and 2^-32 sum_j |v_j| in 64 bits on the GPU (checked against the plain form below)."""
    T, H, D = q.shape
    G = H // k.shape[1]
    o, mag, big, tiny = (torch.zeros(T, H, n, dtype=torch.float64, device="cuda") for n in (D, D, 1, D))
    for b in range(len(lens)):
        lo, hi, L = int(starts[b]), int(starts[b + 1]), max(0, int(lens[b]))
        if hi <= lo:
            continue
        j = torch.arange(L, device="cuda")
        page = table[b][j // k.shape[2]].long()
        end = L - (hi - lo) + 1 + torch.arange(hi - lo, device="cuda")
        seen = (j < end[:, None]) & ((j >= end[:, None] - window) if window else True)
        for h in range(k.shape[1]):
            kk, vv = (x[page, h, j % k.shape[2]].double() * f for x, f in ((k, ks), (v, vs)))
            x = q[lo:hi, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,jd->tgj", x, kk) * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            s = s.masked_fill(~seen[:, None], -float("inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True)) if L else s
            p = torch.where(seen.any(1)[:, None, None], p / p.sum(-1, keepdim=True), torch.zeros_like(p))
            o[lo:hi, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", p, vv)
            tiny[lo:hi, h * G:(h + 1) * G] = (seen.double() @ vv.abs() * 2.0 ** -32)[:, None]
            mag[lo:hi, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", p, vv.abs())
            if L:
                a = torch.einsum("tgd,jd->tgj", x.abs(), kk.abs()) * abs(scale)
                big[lo:hi, h * G:(h + 1) * G] = a.masked_fill(~seen[:, None], 0).amax(-1, keepdim=True)
    return o, mag, big, tiny


def run(k, v, table, starts, lens, q, scale, softcap=0.0, window=0, ks=1.0, vs=1.0, stream=None, ws=None, o=None, pad=0):
    """starts and lens as lists; rows of q and o `pad` values apart."""
    T, H, D = q.shape
    i32 = lambda a: a if torch.is_tensor(a) else torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = q4k.kv_cache(k, v, table, ks, vs)
    size = q4k.q4k_attn_chunk_workspace_size(cache, T, H)
    assert size > 0
    if ws is None:
        ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")  # no call may rely on what is there
    out = torch.full((T, H * D + pad), GUARD, dtype=BF, device="cuda") if o is None else o
    if pad:
        q = torch.cat([q.reshape(T, H * D), torch.full((T, pad), float("nan"), dtype=BF, device="cuda")], 1)
    st, ln = i32(starts), i32(lens)
    torch.cuda.synchronize()
    q4k.q4k_attn_chunk(cache, st, ln, q, T, H * D + pad, H, scale, softcap, window, out, H * D + pad, ws, ws.numel(), stream)
    torch.cuda.synchronize()
    assert (out[:, H * D:] == GUARD).all()
    return out[:, :H * D].reshape(T, H, D)


def check(o, ref, D, e4m3, rows=None, norm=True):
    want, mag, big, tiny = ref
    got = o.double()
    rows = slice(None) if rows is None else rows
    assert torch.isfinite(got).all()
    e = (D * 2.0 ** -24 + 2.0 ** -21) * big
    p = 2.0 ** -11 if e4m3 else 2.0 ** -8
    tol = mag * (2.2 * e + p + 2.0 ** -11) + (tiny if e4m3 else 0) + want.abs() * 2.0 ** -8 + 1e-30
    bad = ((got - want).abs() > tol)[rows]
    assert not bad.any(), (bad.nonzero()[:5].tolist(), float(((got - want).abs() / tol)[rows].max()))
    if norm:
        assert torch.linalg.norm((got - want)[rows]) <= torch.linalg.norm(want[rows]) * (2.0 ** -7.5 + float(e.max()) * 2)


def make(D, dtype, page, layout, Hkv, G, new, lens, gen, spare=1):
    B, per = len(lens), -(-max(max(lens), 1) // page) + spare
    pages = B * per + 2
    k, v = pool((pages, Hkv, page, D), dtype, layout, gen)
    table = table_of(B, per, pages, gen)
    ks, vs = (0.5, 0.25) if dtype == F8 else (1.0, 1.0)
    starts = [0] + np.cumsum(new).tolist()
    q = (torch.randn(starts[-1], Hkv * G, D, generator=gen, device="cuda") * 2 / ks).to(BF)
    return k, v, table, ks, vs, starts, q


CASES = [
    # D, type, page, layout, Hkv, G, new tokens, lengths, window, softcap
    (128, BF, 16, "phsd", 2, 5, [33], [33], 0, 0.0),
    (128, BF, 16, "phsd", 1, 1, [1], [1], 0, 0.0),
    (128, BF, 16, "pshd", 2, 4, [1, 1, 1, 1], [1, 17, 128, 129], 0, 0.0),
    (128, BF, 1, "phsd", 1, 1, [300, 0, 5], [300, 40, 200], 0, 0.0),
    (128, BF, 24, "mixed", 2, 8, [40, 129, 1, 0, 64], [400, 129, 700, 0, 65], 0, 0.0),
    (128, BF, 64, "phsd", 1, 7, [100, 7], [100, 263], 37, 0.0),
    (128, BF, 128, "pshd", 2, 2, [257, 128], [300, 513], 130, 5.0),
    (128, BF, 16, "phsd", 1, 16, [70], [5], 0, 0.0),                 # more new tokens than slots: rows that read nothing
    (64, BF, 16, "phsd", 2, 4, [65, 200, 3], [65, 700, 3], 0, 0.0),
    (64, BF, 7, "mixed", 3, 3, [129, 31], [300, 31], 50, 0.0),
    (64, BF, 32, "pshd", 1, 1, [513], [600], 0, 20.0),
    (256, BF, 16, "phsd", 2, 2, [65, 200, 3], [65, 500, 3], 0, 0.0),
    (256, BF, 24, "mixed", 1, 5, [100, 1, 40], [100, 300, 41], 33, 0.0),
    (256, BF, 64, "pshd", 1, 16, [17, 33], [400, 64], 0, 3.0),
    (128, F8, 16, "phsd", 2, 5, [33, 1, 200], [33, 500, 300], 0, 0.0),
    (128, F8, 64, "pshd", 1, 8, [100], [513], 0, 0.0),
    (128, F8, 5, "mixed", 1, 6, [130, 2], [300, 2], 40, 4.0),
    (64, F8, 16, "phsd", 2, 8, [100, 1], [100, 900], 0, 0.0),
    (64, F8, 24, "mixed", 1, 3, [200], [333], 70, 0.0),
    (256, F8, 32, "phsd", 1, 4, [65, 1], [300, 700], 0, 0.0),
    (256, F8, 16, "mixed", 2, 3, [90, 43], [90, 100], 64, 10.0),
]


@pytest.mark.parametrize("D,dtype,page,layout,Hkv,G,new,lens,window,softcap", CASES)
def test_chunk(D, dtype, page, layout, Hkv, G, new, lens, window, softcap):
    g = gen_of(D + page + G)
    k, v, table, ks, vs, starts, q = make(D, dtype, page, layout, Hkv, G, new, lens, g)
    ref = reference(k, v, table, starts, lens, q, D ** -0.5, softcap, window, ks, vs)
    o = run(k, v, table, starts, lens, q, D ** -0.5, softcap, window, ks, vs)
    q4k.q4k_check_device()
    check(o, ref, D, dtype == F8)
    # the same call again, rows farther apart: the same bits
    o2 = run(k, v, table, starts, lens, q, D ** -0.5, softcap, window, ks, vs, pad=8)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))


def test_the_reference_is_the_plain_form():
    g = gen_of(3)
    k, v, table, ks, vs, starts, q = make(64, BF, 8, "phsd", 2, 2, [9, 0, 20], [9, 4, 12], g)
    for window, cap in ((0, 0.0), (5, 2.0)):
        a = reference(k, v, table, starts, [9, 4, 12], q, 0.3, cap, window)
        b = step_ref.attn_chunk(np64(k), np64(v), table.cpu().numpy(), starts, [9, 4, 12], np64(q), 0.3, cap, window)
        for x, y in zip(a, (b[0], b[1], b[2][:, :, None])):
            assert np.allclose(np64(x), y, rtol=1e-12, atol=1e-13)


LONG = [
    (128, BF, 16, 2, 4, [1500, 2, 700], [1500, 3000, 2500], 0, 0.0),
    (128, BF, 32, 2, 8, [1] * 12 + [200, 333], [4000, 17, 1200, 300, 5000, 1, 129, 128, 127, 2048, 999, 64, 2000, 333], 0, 0.0),
    (128, BF, 64, 1, 5, [1], [30001], 0, 0.0),                   # one row tile, split over the GPU
    (128, F8, 64, 2, 5, [64], [20000], 0, 0.0),
    (64, BF, 16, 4, 4, [1100, 900], [1100, 1500], 256, 0.0),
    (64, F8, 16, 2, 2, [1, 700], [9000, 3000], 0, 0.0),
    (256, BF, 32, 1, 4, [500, 1], [2000, 6000], 0, 0.0),
    (256, F8, 16, 2, 1, [300], [3000], 1000, 30.0),
]


@pytest.mark.parametrize("D,dtype,page,Hkv,G,new,lens,window,softcap", LONG)
def test_chunk_long(D, dtype, page, Hkv, G, new, lens, window, softcap):
    """Many units a CTA, units of many CTAs, and both in a call."""
    g = gen_of(D + G)
    k, v, table, ks, vs, starts, q = make(D, dtype, page, "phsd", Hkv, G, new, lens, g)
    ref = reference(k, v, table, starts, lens, q, D ** -0.5, softcap, window, ks, vs)
    o = run(k, v, table, starts, lens, q, D ** -0.5, softcap, window, ks, vs)
    q4k.q4k_check_device()
    check(o, ref, D, dtype == F8)
    for _ in range(3):
        assert torch.equal(run(k, v, table, starts, lens, q, D ** -0.5, softcap, window, ks, vs), o)


@pytest.mark.parametrize("D,dtype,Hkv,G,new,lens,window,softcap", [
    (128, BF, 2, 4, [900, 1], [3000, 500], 0, 15.0), (128, F8, 1, 5, [600, 3], [1000, 4000], 0, 4.0),
    (64, BF, 2, 2, [1400], [2500], 700, 30.0), (64, F8, 1, 8, [300], [9000], 0, 8.0),
    (256, BF, 1, 4, [700, 40], [1500, 2500], 0, 50.0), (256, F8, 2, 2, [500], [2000], 300, 2.0),
    (128, BF, 4, 8, [20], [9000], 0, 10.0), (128, BF, 1, 1, [40] * 35, [200] * 35, 0, 6.0),
])
def test_chunk_softcap_in_the_weights_pass(D, dtype, Hkv, G, new, lens, window, softcap):
    """Calls of more than a few tiles for a CTA, and small ones, with scores on both sides of the cap."""
    g = gen_of(D + Hkv + len(new))
    k, v, table, ks, vs, starts, q = make(D, dtype, 16, "phsd", Hkv, G, new, lens, g)
    scale = 2.5 * D ** -0.5
    ref = reference(k, v, table, starts, lens, q, scale, softcap, window, ks, vs)
    o = run(k, v, table, starts, lens, q, scale, softcap, window, ks, vs)
    q4k.q4k_check_device()
    check(o, ref, D, dtype == F8)
    assert torch.equal(run(k, v, table, starts, lens, q, scale, softcap, window, ks, vs), o)


def test_chunk_many_sequences():
    """More sequences than threads of the CTA that lists them, many without new tokens."""
    g = gen_of(21)
    B, Hkv, G, D, page = 1500, 1, 2, 64, 8
    lens = [0 if i % 3 == 1 or 300 < i < 700 else (i * 37) % 157 for i in range(B)]
    new = [min(n, (i * 11) % 23) if i % 5 else 0 for i, n in enumerate(lens)]
    k, v, table, ks, vs, starts, q = make(D, BF, page, "phsd", Hkv, G, new, lens, g, spare=0)
    o = run(k, v, table, starts, lens, q, D ** -0.5)
    q4k.q4k_check_device()
    check(o, reference(k, v, table, starts, lens, q, D ** -0.5), D, False)


def test_chunk_agrees_with_the_decode_step():
    """Chunks of equal length: the same rows as q4k_attn_decode's, to both calls' roundings."""
    g = gen_of(22)
    D, n, lens, H = 128, 4, [300, 77, 4], 8
    k, v, table, ks, vs, starts, q = make(D, BF, 16, "phsd", 2, 4, [n] * 3, lens, g)
    cache = q4k.kv_cache(k, v, table)
    ws = torch.empty(q4k.q4k_attn_decode_workspace_size(cache, H, n, 0), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    q4k.q4k_attn_decode(cache, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, H * D, H, n, D ** -0.5, 0.0, 0, o, H * D, None, 0,
                        1.0, ws, ws.numel())
    got = run(k, v, table, starts, lens, q, D ** -0.5)
    ref = reference(k, v, table, starts, lens, q, D ** -0.5)
    assert ((got.double() - o.double()).abs() <= ref[1] * 2.0 ** -7.8 + ref[0].abs() * 2.0 ** -6.9).all()


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("D,lens,new", [(128, [40, 300, 129, 20], [7, 200, 129, 1]), (64, [500], [300]), (256, [130, 70], [100, 3])])
def test_chunk_what_is_masked_has_no_part(dtype, bad, D, lens, new):
    """Slots past a length, before every window or of later tokens may hold anything, in the same page and tile."""
    g = gen_of(11)
    page, window = 16, 60
    k, v, table, _, _, starts, q = make(D, dtype, page, "phsd", 2, 3, new, lens, g)
    clean = run(k, v, table, starts, lens, q, 0.1, window=window)
    value = bad if dtype == BF else (bad if bad != bad else 448.0 if bad > 0 else -448.0)
    poison = torch.full((1,), value, device="cuda").to(dtype)
    view = (lambda x: x.view(torch.uint8)) if dtype == F8 else (lambda x: x)
    def put(b, j):
        at = int(table[b, j // page])
        view(k)[at, :, j % page] = view(poison)
        view(v)[at, :, j % page] = view(poison)
    for b, n in enumerate(lens):
        for j in list(range(0, max(0, n - new[b] + 1 - window))) + list(range(n, table.shape[1] * page)):
            put(b, j)
    assert torch.equal(run(k, v, table, starts, lens, q, 0.1, window=window), clean)
    # the last token, and one in the middle of the chunk: only rows that see them change
    for b, n in enumerate(lens):
        put(b, n - 1)
        if new[b] > 60:
            put(b, n - 40)
    o = run(k, v, table, starts, lens, q, 0.1, window=window)
    for b, n in enumerate(lens):
        first = new[b] - (40 if new[b] > 60 else 1)  # the first row of the chunk that sees one of them
        assert torch.equal(o[starts[b]:starts[b] + first], clean[starts[b]:starts[b] + first])
        if dtype == BF and abs(bad) != 3e38 or bad != bad:
            assert not torch.isfinite(o[starts[b + 1] - 1].float()).any()
    q4k.q4k_check_device()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_an_infinite_value_reaches_those_that_see_it(D):
    """Values (not keys) of one slot: infinite where the slot's are, in the rows from its token on; other values as without it."""
    g = gen_of(12)
    n, page = 200, 16
    k, v, table, _, _, starts, q = make(D, BF, page, "phsd", 1, 2, [n], [n], g)
    j = 150
    v[int(table[0, j // page]), 0, j % page] = 0.0
    ref = reference(k, v, table, starts, [n], q, 0.1)
    v[int(table[0, j // page]), 0, j % page, 5] = float("inf")
    v[int(table[0, j // page]), 0, j % page, 9] = -float("inf")
    o = run(k, v, table, starts, [n], q, 0.1)
    assert (o[j:, :, 5] == float("inf")).all() and (o[j:, :, 9] == -float("inf")).all()
    o[j:, :, 5], o[j:, :, 9] = ref[0][j:, :, 5].to(BF), ref[0][j:, :, 9].to(BF)
    check(o, ref, D, False)


def test_chunk_a_query_without_a_number_keeps_to_itself():
    g = gen_of(9)
    for dtype in (BF, F8):
        k, v, table, _, _, starts, q = make(128, dtype, 16, "phsd", 1, 5, [40], [700], g)
        clean = run(k, v, table, starts, [700], q, 0.1)
        q[7, 2] = float("nan")
        o = run(k, v, table, starts, [700], q, 0.1)
        assert torch.isnan(o[7, 2]).all()
        o[7, 2] = clean[7, 2]
        assert torch.equal(o, clean)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3e4, -1e30, 1e-30])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_chunk_scales(scale, dtype):
    """No scale, a negative one, one that makes scores of millions, one that makes one slot take all, one that makes all equal."""
    g = gen_of(14)
    D, n = 128, 150
    k, v, table, _, _, starts, q = make(D, dtype, 16, "phsd", 1, 2, [n], [n + 130], g)
    o = run(k, v, table, starts, [n + 130], q, scale)
    ref = reference(k, v, table, starts, [n + 130], q, scale)
    assert torch.isfinite(o.float()).all()
    if abs(scale) < 1e3:
        return check(o, ref, D, dtype == F8)
    # differences of scores are at least 2^-24 of their size: each row takes one slot (or none is far ahead, at the roundings)
    top = (torch.einsum("tgd,jd->tgj", q.double(), k[table[0].long(), 0].reshape(-1, D)[:n + 130].double()) * (1 if scale > 0 else -1))
    seen = torch.arange(n + 130, device="cuda") < (131 + torch.arange(n, device="cuda"))[:, None]
    best = top.masked_fill(~seen[:, None], -float("inf")).topk(2, -1)
    clear = (best.values[..., 0] - best.values[..., 1]) > best.values[..., 0].abs() * 2.0 ** -12 + 200 / abs(scale)
    vv = v[table[0].long(), 0].reshape(-1, D)[best.indices[..., 0]].double()
    assert clear.float().mean() > 0.5
    assert ((o.double() - vv).abs() <= vv.abs() * 2.0 ** -7)[clear].all()


def test_chunk_e4m3_small_and_large_queries():
    """Queries of any bf16 magnitude reach an e4m3 cache's keys exactly."""
    g = gen_of(13)
    k, v, table, _, _, starts, base = make(64, F8, 16, "phsd", 1, 3, [40], [128], g)
    base = base.clamp(-8, 8)
    one = run(k, v, table, starts, [128], base, 0.5)
    for e in (-115, -90, -40, 30, 90):
        q = (base.float() * 2.0 ** e).to(BF)
        assert torch.equal(run(k, v, table, starts, [128], q, 0.5 * 2.0 ** -e), one), e


def test_chunk_tiny_queries_and_a_tiny_scale():
    """Scores that are 0 to any precision: every slot that a row sees counts the same, masked ones not at all."""
    g = gen_of(19)
    for dtype in (BF, F8):
        k, v, table, _, _, starts, q = make(128, dtype, 16, "phsd", 1, 3, [40], [170], g)
        q = (q.float() * 2.0 ** -118).to(BF)
        o = run(k, v, table, starts, [170], q, 1e-36)
        ref = reference(k, v, table, starts, [170], q, 0.0)
        check(o, ref, 128, dtype == F8)


def test_chunk_values_of_any_size():
    """A score far above those of the tiles before, and values near 2^100."""
    g = gen_of(20)
    k, v, table, _, _, starts, q = make(128, BF, 16, "phsd", 1, 2, [90], [700], g)
    v *= 2.0 ** 100
    for j, f in ((300, 3.0), (301, 5.0), (450, 9.0), (640, 40.0)):  # each above the one before by more than a step
        k[int(table[0, j // 16]), 0, j % 16] *= f
    o = run(k, v, table, starts, [700], q, 0.3)
    check(o, reference(k, v, table, starts, [700], q, 0.3), 128, False)


def test_chunk_bad_indices_are_reported_and_left_out():
    g = gen_of(15)
    D, page, n, L = 128, 16, 30, 200
    k, v, table, _, _, starts, q = make(D, BF, page, "phsd", 1, 4, [n, n], [L, L], g, spare=0)
    def reported():
        with pytest.raises(q4k.Q4KError) as e:
            q4k.q4k_check_device()
        assert e.value.status == q4k.Q4K_ERR_INDEX
    pages = k.shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1], t[0, 9] = bad, bad
        o = run(k, v, t, starts, [L, L], q, 0.2)
        reported()
        # as if those pages' slots were not there
        keep = torch.cat([table[0, :1], table[0, 2:9], table[0, 10:]])[None]
        ref = reference(k, v, keep, [0, n], [L - 32], q[:n], 0.2)
        check(o[:n], ref, D, False)
        check(o[n:], reference(k, v, table[1:], [0, n], [L], q[n:], 0.2), D, False)
    # lengths beyond the table are clamped, negative ones count as none
    cap = table.shape[1] * page
    o = run(k, v, table, starts, [10 ** 6, -7], q, 0.2)
    reported()
    check(o, reference(k, v, table, starts, [cap, 0], q, 0.2), D, False)
    assert (o[n:] == 0).all()
    # starts that go back or beyond T
    o = run(k, v, table, [5, 2 * n + 9, 3], [L, L], q, 0.2)
    reported()
    check(o[5:], reference(k, v, table[:1], [0, 2 * n - 5], [L], q[5:], 0.2), D, False)
    assert (o[:5] == GUARD).all()
    q4k.q4k_check_device()


@pytest.mark.parametrize("D,G,new", [
    (128, 8, [1] * 31), (128, 8, [1] * 32),                                # sequences
    (128, 8, [31 * 32]), (128, 8, [31 * 32 + 1]),                          # row tiles
    (128, 8, [1] * 16 + [15 * 32 + 15]), (128, 8, [1] * 16 + [16 * 32]),   # the bound on them from both
    (256, 4, [1] * 31), (256, 4, [31 * 32 + 1]), (64, 1, [31 * 256]), (64, 1, [31 * 256, 0, 2]),
])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_chunk_either_side_of_a_small_call(dtype, D, G, new):
    """Each CTA lists the work of a call with less than 32 sequences and at most 32 row tiles; a kernel does for more."""
    g = gen_of(len(new) + D)
    lens = [n + 41 * i % 199 for i, n in enumerate(new)]
    k, v, table, ks, vs, starts, q = make(D, dtype, 16, "phsd", 1, G, new, lens, g)
    ref = reference(k, v, table, starts, lens, q, D ** -0.5, 0.0, 0, ks, vs)
    o = run(k, v, table, starts, lens, q, D ** -0.5, 0.0, 0, ks, vs)
    q4k.q4k_check_device()
    check(o, ref, D, dtype == F8)


@pytest.mark.parametrize("B", [31, 32, 2100])
def test_chunk_bad_starts_and_lengths_of_many_sequences(B):
    g = gen_of(B)
    D, page, L = 64, 8, 24
    k, v, table, _, _, _, q = make(D, BF, page, "phsd", 1, 2, [2] * B, [L] * B, g, spare=0)
    cap = table.shape[1] * page
    starts, lens = [2 * b for b in range(B + 1)], [L] * B
    starts[3], starts[7], starts[B] = 1, 2 ** 31 - 1, -5   # back; beyond T, so that all later ones go back; negative
    lens[1], lens[2], lens[5] = cap + 1, -2 ** 31, 2 ** 31 - 1
    o = run(k, v, table, starts, lens, q, 0.2)
    with pytest.raises(q4k.Q4KError) as e:
        q4k.q4k_check_device()
    assert e.value.status == q4k.Q4K_ERR_INDEX
    T = 2 * B
    as_if = [0, 2, 4, 4, 8, 10, 12] + [T] * (B - 6)
    check(o, reference(k, v, table, as_if, [min(max(n, 0), cap) for n in lens], q, 0.2), D, False)


def test_chunk_rows_of_no_sequence_are_left_alone():
    g = gen_of(16)
    k, v, table, _, _, _, q = make(128, BF, 16, "phsd", 2, 2, [100], [100], g)
    table = table.repeat(2, 1)
    o = run(k, v, table, [10, 40, 70], [60, 90], q, 0.2)
    assert (o[:10] == GUARD).all() and (o[70:] == GUARD).all()
    check(o[10:70], reference(k, v, table, [0, 30, 60], [60, 90], q[10:70], 0.2), 128, False)
    o = run(k, v, table, [0, 0, 0], [60, 90], q, 0.2)  # nothing to do
    assert (o == GUARD).all()
    q4k.q4k_check_device()


def test_chunk_offsets_past_32_bits():
    """Pages more than 2^32 bytes apart."""
    page, D = 16, 128
    stride = (1 << 30) // 8 * 8 + 4096           # elements: 2 GiB a page
    g = gen_of(17)
    pools = []
    for _ in range(2):
        raw = torch.empty(3 * stride + page * D, dtype=BF, device="cuda")
        x = raw.as_strided((4, 1, page, D), (stride, page * D, D, 1))
        x.copy_(torch.randn(4, 1, page, D, generator=g, device="cuda"))
        pools.append(x)
    k, v = pools
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    q = torch.randn(20, 4, D, generator=g, device="cuda").to(BF)
    o = run(k, v, table, [0, 20], [61], q, 0.2)
    q4k.q4k_check_device()
    check(o, reference(k, v, table, [0, 20], [61], q, 0.2), D, False)


def test_chunk_on_another_stream_and_in_two_graphs_that_share_a_workspace():
    g = gen_of(18)
    k, v, table, _, _, starts, q = make(128, BF, 16, "phsd", 2, 4, [60, 1], [300, 900], g)
    lens, st = torch.tensor([300, 900], dtype=torch.int32, device="cuda"), torch.tensor(starts, dtype=torch.int32, device="cuda")
    want = run(k, v, table, starts, [300, 900], q, 0.2)
    side = torch.cuda.Stream()
    assert torch.equal(run(k, v, table, starts, [300, 900], q, 0.2, stream=side), want)
    cache = q4k.kv_cache(k, v, table)
    ws = torch.empty(q4k.q4k_attn_chunk_workspace_size(cache, 61, 8), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(q), torch.zeros_like(q)], []
    for o, scale in zip(outs, (0.2, 0.4)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            q4k.q4k_attn_chunk(cache, st, lens, q, 61, 1024, 8, scale, 0.0, 0, o, 1024, ws, ws.numel())
        graphs.append(graph)
    # replayed in turn, with other lengths, chunks and queries
    for new_starts, new_lens in (([0, 1, 61], [40, 920]), ([0, 61, 61], [61, 5])):
        lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        st.copy_(torch.tensor(new_starts, dtype=torch.int32))
        q.copy_(torch.randn(61, 8, 128, generator=g, device="cuda"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, scale in zip(outs, (0.2, 0.4)):
            assert torch.equal(o, run(k, v, table, new_starts, new_lens, q, scale))
    q4k.q4k_check_device()
