"""The decode-step operators on the GPU against the plain 64-bit forms.

Tolerances are bounds on the kernels' roundings.  Attention: with e = the error of a
score (D fp32 additions of products that sum to at most `big` in magnitude, and the
exponential's 2^-22 of the score), every weight is off by at most a factor e^(2 e), the
weights enter the second product to 2^-15, and o is rounded to bf16.  Sums over slots add
2^-24 per addition, at most 2^-14 for the lengths here.
"""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R

pytestmark = pytest.mark.gpu
F8, BF = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


def pool(shape, dtype, layout, gen, fill=None):
    """Keys and values [pages][heads][size][D] over memory ordered by `layout`."""
    P, H, S, D = shape
    if layout == "phsd":
        k, v = (torch.empty(P, H, S, D, dtype=BF, device="cuda") for _ in range(2))
    elif layout == "pshd":
        k, v = (torch.empty(P, S, H, D, dtype=BF, device="cuda").transpose(1, 2) for _ in range(2))
    else:  # keys and values interleaved, rows padded
        m = torch.empty(P, H, 2, S, D + 32, dtype=BF, device="cuda")
        k, v = m[:, :, 0, :, :D], m[:, :, 1, :, :D]
    if dtype == F8:
        k, v = (torch.empty_strided(x.shape, x.stride(), dtype=F8, device="cuda") if layout != "mixed" else x for x in (k, v))
        if layout == "mixed":
            m = torch.empty(P, H, 2, S, D + 32, dtype=F8, device="cuda")
            k, v = m[:, :, 0, :, :D], m[:, :, 1, :, :D]
    for x in (k, v):
        x.copy_(torch.randn(shape, generator=gen, device="cuda") if fill is None else torch.full(shape, fill, device="cuda"))
    return k, v


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def table_of(B, per, pages, gen):
    return torch.randperm(pages, generator=gen, device="cuda")[:B * per].to(torch.int32).view(B, per)


def np64(t):
    return t.double().cpu().numpy()


ATTN = [
    # D, type, page, layout, Hkv, group, n_q, lens, window, softcap, weights
    (128, BF, 16, "phsd", 2, 5, 1, [1, 0, 2, 15, 16, 17, 63, 64, 65, 1000], 0, 0.0, True),
    (128, BF, 1, "pshd", 1, 1, 1, [5, 129, 64], 0, 0.0, False),
    (64, BF, 24, "mixed", 3, 8, 1, [100, 3, 257], 0, 0.0, True),
    (256, BF, 32, "phsd", 1, 16, 1, [300, 33, 0], 0, 0.0, False),
    (128, BF, 16, "phsd", 2, 4, 4, [4, 3, 1, 0, 100, 515], 0, 0.0, True),          # fewer slots than new tokens
    (128, BF, 64, "phsd", 1, 7, 5, [200, 64, 70], 0, 0.0, True),                    # 35 rows: three row tiles
    (64, BF, 16, "pshd", 2, 2, 3, [400, 50, 2, 90], 37, 0.0, True),                 # a window
    (128, BF, 16, "phsd", 2, 4, 1, [2000, 10], 100, 5.0, False),                    # window and soft cap
    (256, BF, 7, "mixed", 1, 3, 6, [61, 6, 700], 50, 0.0, True),
    (128, F8, 16, "phsd", 2, 5, 1, [1, 0, 31, 32, 33, 127, 128, 129, 1500], 0, 0.0, True),
    (64, F8, 64, "pshd", 2, 8, 2, [100, 1, 900], 0, 0.0, True),
    (256, F8, 16, "phsd", 1, 4, 1, [64, 65, 333], 0, 0.0, False),
    (128, F8, 5, "mixed", 1, 6, 4, [300, 2, 77], 40, 0.0, True),
    (256, F8, 16, "phsd", 1, 2, 3, [130, 40], 33, 3.0, True),
    (64, BF, 16, "phsd", 1, 8, 3, [90, 200, 2], 0, 0.0, True),                      # 24 rows of one row tile
    (64, F8, 16, "phsd", 2, 16, 2, [140, 33], 20, 0.0, True),                       # 32
    (256, F8, 24, "pshd", 1, 16, 2, [100, 31], 0, 0.0, True),                       # two row tiles of 16
    (256, BF, 16, "phsd", 2, 6, 7, [77, 300], 0, 0.0, False),                       # three
    (128, F8, 16, "mixed", 1, 12, 6, [65, 500], 0, 0.0, True),                      # three of 32
    (128, BF, 16, "phsd", 1, 1, 64, [64, 100], 0, 0.0, True),                       # the most new tokens
]


def run_attn(k, v, table, lens, q, n_q, scale, softcap=0.0, window=0, weights=None, decay=1.0, ks=1.0, vs=1.0, stream=None,
             ws=None):
    cache = q4k.kv_cache(k, v, table, ks, vs)
    B, _, H, D = q.shape
    ld = weights.shape[2] if weights is not None else 0
    size = q4k.q4k_attn_decode_workspace_size(cache, H, n_q, ld)
    assert size > 0
    if ws is None:
        ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")  # no call may rely on what is there
    o = torch.full_like(q, float("nan"))
    q4k.q4k_attn_decode(cache, lens, q, H * D, H, n_q, scale, softcap, window, o, H * D, weights, ld, decay, ws, ws.numel(),
                        stream)
    return o


def check_attn(o, w, ref, D, n):
    want, wref, mag, big = ref
    e = D * 2.0 ** -24 * big + 2.0 ** -20 * big
    tol = mag * (2 * e[..., None] * 1.1 + 2.0 ** -14) + np.abs(want) * 2.0 ** -8 + 1e-30
    got = np64(o)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    if wref is not None:
        tol = np.abs(wref) * (2 * e.max() * 1.1 + 2.0 ** -14) + 1e-30
        assert (np.abs(np64(w) - wref) <= tol).all(), float((np.abs(np64(w) - wref) / tol).max())


@pytest.mark.parametrize("D,dtype,page,layout,Hkv,G,n_q,lens,window,softcap,weigh", ATTN)
def test_attn(D, dtype, page, layout, Hkv, G, n_q, lens, window, softcap, weigh):
    g = gen_of(D + page)
    B, per = len(lens), -(-max(lens) // page) + 1
    pages = B * per + 2
    k, v = pool((pages, Hkv, page, D), dtype, layout, g)
    table = table_of(B, per, pages, g)
    ks, vs = (0.5, 0.25) if dtype == F8 else (1.0, 1.0)
    q = (torch.randn(B, n_q, Hkv * G, D, generator=g, device="cuda") * 2 / ks).to(BF)
    w0 = torch.rand(B, Hkv, per * page, generator=g, device="cuda") if weigh else None
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = R.attn_decode(np64(k), np64(v), table.cpu().numpy(), lens, np64(q), n_q, D ** -0.5, softcap, window, ks, vs,
                        None if w0 is None else np64(w0), 0.9)
    w = None if w0 is None else w0.clone()
    o = run_attn(k, v, table, lt, q, n_q, D ** -0.5, softcap, window, w, 0.9, ks, vs)
    q4k.q4k_check_device()
    check_attn(o, w, ref, D, max(lens))
    # the same call again: the same bits
    w2 = None if w0 is None else w0.clone()
    o2 = run_attn(k, v, table, lt, q, n_q, D ** -0.5, softcap, window, w2, 0.9, ks, vs)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and (w is None or torch.equal(w, w2))


@pytest.mark.parametrize("D,dtype,page,layout,Hkv,G,n_q,lens,window,softcap", [
    (256, F8, 32, "phsd", 1, 16, 4, [83, 2793], 0, 0.0),      # 64 rows in four tiles, a few units in many parts
    (64, BF, 16, "pshd", 2, 16, 4, [17, 569, 300], 0, 0.0),   # whole units, 64 rows
    (128, BF, 16, "phsd", 1, 5, 1, [1500, 1025], 0, 0.0),
    (128, F8, 24, "mixed", 1, 40, 3, [3000, 3, 517], 700, 30.0),  # 120 rows; chunks before the window's begin
    (64, BF, 16, "phsd", 3, 7, 5, [257, 256, 255, 4097], 0, 0.0),
])
def test_attn_weights_of_many_rows(D, dtype, page, layout, Hkv, G, n_q, lens, window, softcap):
    """Weights of few slots, whose rows are dealt to groups of threads, and (m, l) of several octets at once."""
    test_attn(D, dtype, page, layout, Hkv, G, n_q, lens, window, softcap, True)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_attn_many_and_long(dtype):
    """Ragged lengths over two orders of magnitude (units of one CTA, of many, of none), and one long sequence."""
    g = gen_of(7)
    for lens, Hkv, G in (([0, 1, 30, 9000, 64, 700, 2, 4000, 333] * 7, 2, 4), ([70001], 1, 8)):
        B, page, D = len(lens), 16, 128
        per = -(-max(lens) // page)
        k, v = pool((B * per, Hkv, page, D), dtype, "phsd", g)
        table = table_of(B, per, B * per, g)
        q = (torch.randn(B, 1, Hkv * G, D, generator=g, device="cuda") * 2).to(BF)
        w = torch.zeros(B, Hkv, per * page, device="cuda")
        o = run_attn(k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, 1, D ** -0.5, weights=w)
        ref = R.attn_decode(np64(k), np64(v), table.cpu().numpy(), lens, np64(q), 1, D ** -0.5, weights=np.zeros(w.shape))
        check_attn(o, w, ref, D, max(lens))
    q4k.q4k_check_device()


def test_attn_more_sequences_than_threads():
    """Several sequences a thread when the work is shared out, many of them empty."""
    g = gen_of(8)
    B, Hkv, G, D, page, per = 700, 2, 3, 64, 8, 20
    lens = [0 if i % 3 == 1 or 200 < i < 420 else (i * 37) % 157 for i in range(B)]
    k, v = pool((B * per, Hkv, page, D), BF, "phsd", g)
    table = table_of(B, per, B * per, g)
    q = torch.randn(B, 1, Hkv * G, D, generator=g, device="cuda").to(BF)
    w = torch.ones(B, Hkv, per * page, device="cuda")
    o = run_attn(k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, 1, D ** -0.5, weights=w, decay=0.5)
    q4k.q4k_check_device()
    check_attn(o, w, R.attn_decode(np64(k), np64(v), table.cpu().numpy(), lens, np64(q), 1, D ** -0.5, weights=np.ones(w.shape),
                                   decay=0.5), D, 160)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("n", [40, 5000])
def test_attn_a_query_without_a_number_keeps_to_itself(dtype, n):
    g = gen_of(9)
    D, page, per = 128, 16, 320
    k, v = pool((per, 1, page, D), dtype, "phsd", g)
    table = table_of(1, per, per, g)
    q = torch.randn(1, 1, 5, D, generator=g, device="cuda").to(BF)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    clean = run_attn(k, v, table, lens, q, 1, 0.1)
    q[0, 0, 2] = float("nan")
    o = run_attn(k, v, table, lens, q, 1, 0.1)
    assert torch.isnan(o[0, 0, 2]).all()
    assert torch.equal(o[0, 0, [0, 1, 3, 4]], clean[0, 0, [0, 1, 3, 4]])


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_attn_what_is_masked_has_no_part(dtype, bad):
    """Slots past a length, outside the window or of later tokens may hold anything, in the same page and tile."""
    g = gen_of(11)
    Hkv, G, n_q, D, page, lens, window = 2, 3, 3, 128, 16, [40, 7, 90, 17], 25
    B, per = len(lens), 6
    k, v = pool((B * per, Hkv, page, D), dtype, "phsd", g)
    table = table_of(B, per, B * per, g)
    q = torch.randn(B, n_q, Hkv * G, D, generator=g, device="cuda").to(BF)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = run_attn(k, v, table, lt, q, n_q, 0.1, window=window)
    if dtype == F8 and bad != bad:
        poison = torch.full((1,), float("nan"), device="cuda").to(F8)
    else:
        poison = torch.full((1,), bad if dtype == BF else (448.0 if bad > 0 else -448.0), device="cuda").to(dtype)
    kb, vb = (x.view(torch.uint8) if dtype == F8 else x for x in (k, v))
    pb = poison.view(torch.uint8) if dtype == F8 else poison
    for b, n in enumerate(lens):
        first = max(0, n - n_q + 1 - window)
        for j in list(range(0, first)) + list(range(n, per * page)):
            pg = int(table[b, j // page])
            kb[pg, :, j % page] = pb
            vb[pg, :, j % page] = pb
    assert torch.equal(run_attn(k, v, table, lt, q, n_q, 0.1, window=window), clean)
    # the last token: only its own query sees it
    for b, n in enumerate(lens):
        pg = int(table[b, (n - 1) // page])
        vb[pg, :, (n - 1) % page] = pb
        kb[pg, :, (n - 1) % page] = pb
    o = run_attn(k, v, table, lt, q, n_q, 0.1, window=window)
    assert torch.equal(o[:, :2], clean[:, :2])
    q4k.q4k_check_device()


def test_attn_extreme_scores():
    """Scores that overflow e^s by far, and keys of the type's largest value."""
    g = gen_of(12)
    k, v = pool((8, 1, 16, 128), BF, "phsd", g)
    table = table_of(1, 8, 8, g)
    q = torch.randn(1, 1, 2, 128, generator=g, device="cuda").to(BF) * 300
    k[3] *= 1e3
    lens = torch.tensor([128], dtype=torch.int32, device="cuda")
    o = run_attn(k, v, table, lens, q, 1, 1.0)
    ref = R.attn_decode(np64(k), np64(v), table.cpu().numpy(), [128], np64(q), 1, 1.0)
    assert np.isfinite(np64(o)).all()
    # one slot takes all: its value, rounded
    assert (np.abs(np64(o) - ref[0]) <= np.abs(ref[0]) * 2.0 ** -8 + 1e-30).all()


def test_attn_e4m3_small_and_large_queries():
    """Queries of any bf16 magnitude reach an e4m3 cache's keys exactly."""
    g = gen_of(13)
    k, v = pool((8, 1, 16, 64), F8, "phsd", g)
    table = table_of(1, 8, 8, g)
    lens = torch.tensor([128], dtype=torch.int32, device="cuda")
    base = torch.randn(1, 1, 3, 64, generator=g, device="cuda").to(BF)
    one = run_attn(k, v, table, lens, base, 1, 0.5)
    for e in (-90, -40, 30, 90):
        q = (base.float() * 2.0 ** e).to(BF)
        assert torch.equal(run_attn(k, v, table, lens, q, 1, 0.5 * 2.0 ** -e), one)


def test_attn_bad_indices_are_reported_and_left_out():
    g = gen_of(14)
    page, D, B, per = 16, 64, 2, 4
    k, v = pool((B * per, 1, page, D), BF, "phsd", g)
    table = table_of(B, per, B * per, g)
    q = torch.randn(B, 1, 4, D, generator=g, device="cuda").to(BF)
    for bad in (-1, B * per, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        o = run_attn(k, v, t, torch.tensor([60, 60], dtype=torch.int32, device="cuda"), q, 1, 0.3)
        with pytest.raises(q4k.Q4KError) as e:
            q4k.q4k_check_device()
        assert e.value.status == q4k.Q4K_ERR_INDEX
        # as if the page's slots were not there: the other 44 in their order
        keep = torch.cat([table[0, :1], table[0, 2:]])[None]
        short = torch.cat([k[keep[0].long()].reshape(-1, D)[:44], torch.zeros(4, D, device="cuda", dtype=BF)]).view(3, 1, page, D)
        shortv = torch.cat([v[keep[0].long()].reshape(-1, D)[:44], torch.zeros(4, D, device="cuda", dtype=BF)]).view(3, 1, page, D)
        ref = R.attn_decode(np64(short), np64(shortv), np.array([[0, 1, 2]]), [44], np64(q[:1]), 1, 0.3)
        check_attn(o[:1], None, ref, D, 44)
    # lengths beyond the table are clamped, negative ones count as none
    o = run_attn(k, v, table, torch.tensor([1000, -5], dtype=torch.int32, device="cuda"), q, 1, 0.3)
    with pytest.raises(q4k.Q4KError):
        q4k.q4k_check_device()
    ref = R.attn_decode(np64(k), np64(v), table.cpu().numpy(), [64, 0], np64(q), 1, 0.3)
    check_attn(o, None, ref, D, 64)
    q4k.q4k_check_device()


def test_attn_offsets_past_32_bits():
    """Pages more than 2^32 bytes apart."""
    page, D = 16, 128
    stride = (1 << 30) // 8 * 8 + 4096           # elements: 2 GiB a page
    raw = torch.empty(3 * stride + page * D, dtype=BF, device="cuda")
    k = raw.as_strided((4, 1, page, D), (stride, page * D, D, 1))
    vraw = torch.empty(3 * stride + page * D, dtype=BF, device="cuda")
    v = vraw.as_strided((4, 1, page, D), (stride, page * D, D, 1))
    g = gen_of(15)
    for x in (k, v):
        x.copy_(torch.randn(4, 1, page, D, generator=g, device="cuda"))
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 4, D, generator=g, device="cuda").to(BF)
    lens = torch.tensor([61], dtype=torch.int32, device="cuda")
    o = run_attn(k, v, table, lens, q, 1, 0.2)
    kc, vc = k.contiguous(), v.contiguous()
    ref = R.attn_decode(np64(kc), np64(vc), table.cpu().numpy(), [61], np64(q), 1, 0.2)
    check_attn(o, None, ref, D, 61)
    # eviction moves rows between such pages
    w = torch.arange(64, dtype=torch.float32, device="cuda").view(1, 1, 64).contiguous()
    p = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 1, 64).contiguous()
    cache = q4k.kv_cache(k, v, table)
    ws = torch.empty(q4k.q4k_kv_evict_workspace_size(cache, 64), dtype=torch.uint8, device="cuda")
    q4k.q4k_kv_evict(cache, lens, lens, 32, 0, 0, w, p, w, p, 64, ws, ws.numel())
    q4k.q4k_check_device()
    _, take = R.kv_evict([61], np.arange(64.0).reshape(1, 1, 64), np.arange(64).reshape(1, 1, 64), 32, 0, 0)
    rows = kc[table[0].long(), 0].reshape(-1, D)
    assert torch.equal(k[table[0, :2].long(), 0].reshape(-1, D), rows[torch.tensor(take[0][0], device="cuda")])
    assert int(lens[0]) == 32


def test_attn_on_another_stream_and_in_a_graph():
    g = gen_of(16)
    k, v = pool((8, 2, 16, 128), BF, "phsd", g)
    table = table_of(2, 4, 8, g)
    q = torch.randn(2, 1, 8, 128, generator=g, device="cuda").to(BF)
    lens = torch.tensor([50, 20], dtype=torch.int32, device="cuda")
    want = run_attn(k, v, table, lens, q, 1, 0.2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cache = q4k.kv_cache(k, v, table)
    ws = torch.empty(q4k.q4k_attn_decode_workspace_size(cache, 8, 1, 0), dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(q)
    call = lambda s: q4k.q4k_attn_decode(cache, lens, q, 1024, 8, 1, 0.2, 0.0, 0, o, 1024, None, 0, 1.0, ws, ws.numel(), s)  # noqa: E731
    call(side)
    side.synchronize()
    assert torch.equal(o, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(None)
    # a graph replayed with other lengths, queries and table contents
    lens.copy_(torch.tensor([64, 3], dtype=torch.int32))
    q.copy_(torch.randn(2, 1, 8, 128, generator=g, device="cuda"))
    want = run_attn(k, v, table, lens, q, 1, 0.2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("D,dtype,layout,rot,pairs,offset", [
    (128, BF, "phsd", 128, False, 0), (64, F8, "pshd", 32, True, 0), (256, BF, "mixed", 128, False, 0),
    (128, F8, "phsd", 0, False, 0), (64, BF, "phsd", 30, False, 0), (128, F8, "phsd", 128, True, 1),
    (128, BF, "pshd", 6, True, 3)])
@pytest.mark.parametrize("T", [1, 37])
def test_append(D, dtype, layout, rot, pairs, offset, T):
    g = gen_of(D + rot)
    B, Hkv, G, page, per = 5, 2, 3, 12, 4
    Hq = Hkv * G
    k, v = pool((B * per + 1, Hkv, page, D), dtype, layout, g)
    table = table_of(B, per, B * per + 1, g)
    at = torch.randperm(B * per * page, generator=g, device="cuda")[:T]
    seq, slot = (at // (per * page)).int(), (at % (per * page)).int()
    pos = torch.randint(0, 500, (T,), generator=g, device="cuda", dtype=torch.int32)
    width = (Hq + 2 * Hkv) * D + offset
    raw = torch.randn(T * width + offset, generator=g, device="cuda") * 30
    x = raw[offset:].view(T, width)              # odd offsets: no row is 16-byte aligned
    rope = torch.randn(500, rot, generator=g, device="cuda").contiguous() if rot else None
    ld = per * page
    w = torch.ones(B, Hkv, ld, device="cuda")
    p = torch.zeros(B, Hkv, ld, dtype=torch.int32, device="cuda")
    q = torch.full((T, Hq, D), float("nan"), dtype=BF, device="cuda")
    wantk, wantv = k.clone(), v.clone()
    ks, vs = (0.5, 0.125) if dtype == F8 else (1.0, 1.0)
    cache = q4k.kv_cache(k, v, table, ks, vs)
    q4k.q4k_kv_append(cache, T, Hq, x.data_ptr(), width, x.data_ptr() + 4 * Hq * D, width,
                      x.data_ptr() + 4 * (Hq + Hkv) * D, width, seq, slot, pos, rope, 500, rot,
                      q4k.Q4K_ROPE_PAIRS if pairs else q4k.Q4K_ROPE_HALF, q, Hq * D, w, p, ld)
    q4k.q4k_check_device()
    rows = x[:, :(Hq + 2 * Hkv) * D].reshape(T, -1, D).cpu().numpy()
    tab = np.zeros((T, 0), np.float32) if rope is None else rope[pos.long()].cpu().numpy()
    rq = torch.from_numpy(R.rope(rows[:, :Hq], tab, rot, pairs))
    rk = torch.from_numpy(R.rope(rows[:, Hq:Hq + Hkv], tab, rot, pairs)) * (1 / ks)
    rv = torch.from_numpy(rows[:, Hq + Hkv:]) * (1 / vs)
    assert torch.equal(q.cpu(), rq.to(BF))
    stored = (lambda t: t.clamp(-448, 448).to(F8)) if dtype == F8 else (lambda t: t.to(BF))
    for want, new in ((wantk, rk), (wantv, rv)):
        for t in range(T):
            pg = table[seq[t], slot[t] // page]
            want[pg, :, slot[t] % page] = stored(new[t]).cuda()
    u8 = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(u8(k), u8(wantk)) and torch.equal(u8(v), u8(wantv))
    ww, wp = torch.ones_like(w), torch.zeros_like(p)
    ww[seq.long(), :, slot.long()] = 0.0
    wp[seq.long(), :, slot.long()] = pos[:, None]
    assert torch.equal(w, ww) and torch.equal(p, wp)


def test_append_values_without_a_number_and_without_queries():
    """NaN, infinities and values beyond e4m3; keys and values only."""
    g = gen_of(21)
    k, v = pool((2, 1, 4, 64), F8, "phsd", g)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    x = torch.randn(1, 64, device="cuda", generator=g)
    x[0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30, -449.0, -0.0])
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = q4k.kv_cache(k, v, table)
    q4k.q4k_kv_append(cache, 1, 0, None, 0, x, 64, x, 64, i, i + 5, i, None, 0, 0, q4k.Q4K_ROPE_HALF, None, 0)
    q4k.q4k_check_device()
    for c in (k, v):
        row = c[0, 0, 1].float()
        assert torch.isnan(row[0]) and row[1:5].tolist() == [448.0, -448.0, 448.0, -448.0]
        assert torch.equal(row[5:], x[0, 5:].to(F8).float())


def test_append_bad_indices():
    g = gen_of(22)
    k, v = pool((4, 2, 4, 64), BF, "phsd", g)
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    T = 8
    seq = torch.tensor([0, -1, 2, 0, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
    slot = torch.tensor([0, 0, 0, 8, -3, 5, 1, 2], dtype=torch.int32, device="cuda")   # token 5: page id 9
    pos = torch.tensor([0, 0, 0, 0, 0, 0, 10, -1], dtype=torch.int32, device="cuda")   # 6, 7: no such position
    x = torch.randn(T, 4 * 64, generator=g, device="cuda")
    q = torch.full((T, 2, 64), float("nan"), dtype=BF, device="cuda")
    rope = torch.randn(10, 64, generator=g, device="cuda")
    k0, v0 = k.clone(), v.clone()
    w = torch.ones(2, 2, 8, device="cuda")
    cache = q4k.kv_cache(k, v, table)
    q4k.q4k_kv_append(cache, T, 2, x, 256, x.data_ptr() + 4 * 128, 256, x.data_ptr() + 4 * 128, 256, seq, slot, pos, rope,
                      10, 64, q4k.Q4K_ROPE_HALF, q, 128, w, None, 8)
    with pytest.raises(q4k.Q4KError) as e:
        q4k.q4k_check_device()
    assert e.value.status == q4k.Q4K_ERR_INDEX
    k0[0, :, 0] = k[0, :, 0]
    v0[0, :, 0] = v[0, :, 0]
    assert torch.equal(k, k0) and torch.equal(v, v0)
    assert (q[1:] == 0).all() and (q[0] != 0).any()
    assert w.sum() == 32 - 2
    q4k.q4k_check_device()


# ---------------------------------------------------------------- evict

def run_evict(c, lens, budget, sinks, recent, w, p, in_place=False):
    ld = w.shape[2]
    ws = torch.full((q4k.q4k_kv_evict_workspace_size(c, ld),), 0x5A, dtype=torch.uint8, device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = lt if in_place else torch.full_like(lt, -7)
    wo, po = (w, p) if in_place else (torch.full_like(w, -1), torch.full_like(p, -1))
    q4k.q4k_kv_evict(c, lt, new, budget, sinks, recent, w, p, wo, po, ld, ws, ws.numel())
    return new, wo, po


@pytest.mark.parametrize("dtype,D,page,layout,Hkv,lens,budget,sinks,recent,kind", [
    (BF, 128, 16, "phsd", 2, [0, 5, 64, 65, 66, 200, 1], 64, 4, 16, "random"),
    (BF, 64, 1, "pshd", 3, [300, 299, 17], 100, 0, 0, "random"),
    (F8, 256, 24, "mixed", 1, [500, 120, 3000], 119, 2, 60, "ties"),
    (F8, 64, 16, "phsd", 2, [1025, 2049], 1024, 4, 1020, "equal"),       # everything kept is protected
    (BF, 64, 16, "phsd", 1, [700, 40], 30, 10, 20, "equal"),
    (BF, 64, 64, "phsd", 2, [2000, 1999], 1, 0, 1, "random"),
    (BF, 64, 64, "phsd", 2, [2000, 900], 700, 0, 5, "odd"),              # infinities, NaN, signed zeros, negatives
    (BF, 64, 128, "phsd", 1, [30000, 21000, 20480], 9000, 4, 100, "ties"),  # longer than what a CTA's registers hold
    (BF, 64, 128, "phsd", 1, [9000, 17001], 8192, 4, 100, "random"),
    (BF, 64, 128, "phsd", 1, [60000, 49153], 30000, 4, 100, "random"),      # longer than the shared memory's keys
    (BF, 64, 16, "phsd", 1, [400], 200, 0, 50, "one position"),          # all protected: cut by weight all the same
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(dtype, D, page, layout, Hkv, lens, budget, sinks, recent, kind, in_place):
    g = gen_of(budget)
    B, per = len(lens), -(-max(max(lens), 1) // page) + 1
    k, v = pool((B * per, Hkv, page, D), dtype, layout, g)
    table = table_of(B, per, B * per, g)
    ld = per * page - 3 if per * page - 3 >= max(lens) else per * page
    w = torch.rand(B, Hkv, ld, generator=g, device="cuda")
    if kind == "ties":
        w = torch.floor(w * 5)
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "odd":
        w = w - 0.5
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-40)):
            w[:, :, i::37] = x
    p = torch.stack([torch.randperm(ld, generator=g, device="cuda") for _ in range(B * Hkv)]).view(B, Hkv, ld).int()
    if kind == "one position":
        p.fill_(3)
    new, take = R.kv_evict(lens, w.cpu().numpy(), p.cpu().numpy(), budget, sinks, recent)
    u8 = lambda t: t.view(torch.uint8) if t.dtype == F8 else t  # noqa: E731
    k0, v0, w0, p0 = k.clone(), v.clone(), w.clone(), p.clone()
    got, wo, po = run_evict(q4k.kv_cache(k, v, table), lens, budget, sinks, recent, w, p, in_place)
    q4k.q4k_check_device()
    assert got.tolist() == new.tolist()
    for b in range(B):
        for h in range(Hkv):
            t = torch.tensor(take[b][h], dtype=torch.long, device="cuda")
            m = len(take[b][h])
            to = torch.arange(m, device="cuda")
            for now, was in ((k, k0), (v, v0)):
                want = u8(was)[table[b][t // page].long(), h, t % page]
                assert torch.equal(u8(now)[table[b][to // page].long(), h, to % page], want)
            assert torch.equal(wo[b, h, :m].view(torch.int32), w0[b, h, t].view(torch.int32))
            assert torch.equal(po[b, h, :m], p0[b, h, t])
            if not in_place:
                assert (wo[b, h, m:] == -1).all() and (po[b, h, m:] == -1).all()
    # slots at or above the budget, and pages of nobody, are as they were
    for b, n in enumerate(lens):
        j = torch.arange(min(int(new[b]), n), per * page, device="cuda")
        for now, was in ((k, k0), (v, v0)):
            pg = table[b][j // page].long()
            assert torch.equal(u8(now)[pg, :, j % page], u8(was)[pg, :, j % page])


@pytest.mark.parametrize("n", [1100, 4090, 9001, 20011, 30001, 50021])
@pytest.mark.parametrize("part", [0.01, 0.5, 0.99])
def test_evict_equal_weights_over_many_slots(n, part):
    """Far more equal weights than are ranked at once: those in the lowest slots go, however far in they end."""
    g = gen_of(n)
    page, D = 64, 64
    per = -(-n // page)
    k, v = pool((per, 1, page, D), BF, "phsd", g)
    table = table_of(1, per, per, g)
    ld = per * page
    w = torch.floor(torch.rand(1, 1, ld, generator=g, device="cuda") * 1.5)  # two thirds 0
    p = torch.randperm(ld, generator=g, device="cuda").view(1, 1, ld).int()
    budget, was = n - max(1, int(part * 0.6 * n)), p[0, 0].tolist()
    _, take = R.kv_evict([n], w.cpu().numpy(), p.cpu().numpy(), budget, 1, 5)
    got, wo, po = run_evict(q4k.kv_cache(k, v, table), [n], budget, 1, 5, w, p, True)
    q4k.q4k_check_device()
    assert got.tolist() == [budget] and po[0, 0, :budget].tolist() == [was[j] for j in take[0][0]]


@pytest.mark.parametrize("kind", ["random", "ties", "equal"])
@pytest.mark.parametrize("most", [300, 4096])
def test_evict_more_heads_than_sms(kind, most):
    """More sequences and heads than a GPU has SMs, which smaller CTAs take."""
    lens = [(37 * i) % 90 + 1 for i in range(78)] + [most, most - 1]
    test_evict(BF, 64, 16, "phsd", 4, lens, 32, 2, 8, kind, True)


def test_evict_bad_indices():
    g = gen_of(31)
    k, v = pool((4, 1, 16, 64), BF, "phsd", g)
    table = torch.tensor([[0, 1], [2, 77]], dtype=torch.int32, device="cuda")
    w = torch.rand(2, 1, 32, generator=g, device="cuda")
    p = torch.arange(32, dtype=torch.int32, device="cuda").expand(2, 1, 32).contiguous()
    k0 = k.clone()
    new, _, _ = run_evict(q4k.kv_cache(k, v, table), [10, 32], 8, 0, 0, w, p)
    with pytest.raises(q4k.Q4KError) as e:
        q4k.q4k_check_device()
    assert e.value.status == q4k.Q4K_ERR_INDEX
    assert new.tolist() == [8, 8] and torch.equal(k[3], k0[3])
    run_evict(q4k.kv_cache(k, v, table[:1]), [100], 8, 0, 0, w[:1], p[:1])
    with pytest.raises(q4k.Q4KError):
        q4k.q4k_check_device()
    q4k.q4k_check_device()


def test_attend_append_evict_keep_the_cache_consistent():
    """A cache at its budget over several steps: positions stay with their keys, and the set of slots is what a cache
    without pages would hold."""
    g = gen_of(32)
    B, Hkv, D, page, per, budget = 2, 2, 64, 4, 3, 9
    k, v = pool((B * per, Hkv, page, D), BF, "phsd", g)
    table = table_of(B, per, B * per, g)
    ld = per * page
    w = torch.zeros(B, Hkv, ld, device="cuda")
    p = torch.full((B, Hkv, ld), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache = q4k.kv_cache(k, v, table)
    ws = torch.empty(max(q4k.q4k_attn_decode_workspace_size(cache, 4, 1, ld), q4k.q4k_kv_evict_workspace_size(cache, ld)),
                     dtype=torch.uint8, device="cuda")
    keys = torch.randn(20, B, Hkv, D, generator=g, device="cuda")
    seq = torch.arange(B, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 4, D, dtype=BF, device="cuda")
    o = torch.zeros_like(q)
    for t in range(20):
        x = torch.cat([torch.randn(B, 4 * D, generator=g, device="cuda"), keys[t].reshape(B, -1), keys[t].reshape(B, -1)], 1).contiguous()
        at = x.data_ptr()
        q4k.q4k_kv_append(cache, B, 4, at, x.shape[1], at + 16 * D, x.shape[1], at + 24 * D, x.shape[1], seq, lens,
                          torch.full((B,), t, dtype=torch.int32, device="cuda"), None, 0, 0, q4k.Q4K_ROPE_HALF, q, 4 * D, w, p, ld)
        lens += 1
        q4k.q4k_attn_decode(cache, lens, q, 4 * D, 4, 1, D ** -0.5, 0.0, 0, o, 4 * D, w, ld, 1.0, ws, ws.numel())
        q4k.q4k_kv_evict(cache, lens, lens, budget, 1, 3, w, p, w, p, ld, ws, ws.numel())
        q4k.q4k_check_device()
        for b in range(B):
            for h in range(Hkv):
                n = int(lens[b])
                held = p[b, h, :n].tolist()
                assert n == min(t + 1, budget) and len(set(held)) == n
                assert {0, t, max(t - 1, 0), max(t - 2, 0)} <= set(held)
                j = torch.arange(n, device="cuda")
                rows = k[table[b][j // page].long(), h, j % page]
                assert torch.equal(rows, keys[torch.tensor(held, device="cuda"), b, h].to(BF))


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("M,D,off", [(1, 1, 0), (3, 7, 0), (2, 64, 0), (5, 768, 0), (3, 2048, 0), (2, 5120, 0), (2, 5121, 0),
                                     (4, 1000, 1), (2, 16384, 0), (2, 16385, 0), (1, 40000, 0)])
@pytest.mark.parametrize("post,pre,gate,res,bias", [
    ("rms", "rms", None, torch.float32, False), ("layer", "rms", "row", BF, True), ("none", "layer", "all", torch.float32, True),
    ("layer", "none", "row", BF, False), ("rms", "layer", None, BF, True)])
def test_norm(M, D, off, post, pre, gate, res, bias):
    """fp32 arithmetic: a few roundings of 2^-24 of each term, a sum of D squares in a tree of depth log2 D + 64 per thread
    at most, and the outputs' own rounding (bf16: 2^-9)."""
    g = gen_of(D + M)
    kind = {"none": 0, "rms": 1, "layer": 2}
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ld = D + off
    y = (rnd(M * ld + off) * 5 + 1)[off:].view(M, ld)
    r = (rnd(M * ld + off) * 2)[off:].to(res).view(M, ld)
    if off:
        r = torch.empty(M * ld + off, dtype=res, device="cuda")[off:].view(M, ld).copy_(r)
    vec = lambda: rnd(D + off)[off:]  # noqa: E731
    pw, qw = 1 + 0.2 * vec(), 1 + 0.2 * vec()
    pb, qb = (vec(), vec()) if bias else (None, None)
    gt = None if gate is None else rnd(1 if gate == "row" else M, D)
    r_out = torch.zeros(M, ld, dtype=res, device="cuda")
    x = torch.zeros(M, ld, dtype=BF, device="cuda")
    q4k.q4k_norm_residual(M, D, y, ld, kind[post], pw, pb, 1e-5, gt, 0 if gate != "all" else D, 0.7, r, r_out, ld,
                          q4k.Q4K_RES_FP32 if res == torch.float32 else q4k.Q4K_RES_BF16, kind[pre], qw, qb, 1e-6, x, ld)
    f = lambda t: None if t is None else np64(t)  # noqa: E731
    h, want = R.norm_residual(f(y)[:, :D], kind[post], f(pw), f(pb), 1e-5, f(gt), 0.7, f(r)[:, :D], kind[pre], f(qw), f(qb), 1e-6)
    terms = np.abs(h) + np.abs(h - f(r)[:, :D]) + np.abs(f(r)[:, :D]) + (0 if pb is None else np.abs(f(pb) * 0.7 * (1 if gt is None else f(gt))))
    tol = terms * 100 * 2.0 ** -24 + (np.abs(h) * 2.0 ** -8 if res == BF else 0)
    assert (np.abs(np64(r_out)[:, :D] - h) <= tol).all()
    scale = np.abs(want) + (0 if pb is None or pre == "none" else np.abs(f(qb))) + terms * (
        1 if pre == "none" else np.abs(f(qw)) / np.sqrt((((h - h.mean(1, keepdims=True)) if pre == "layer" else h) ** 2).mean(1, keepdims=True) + 1e-6))
    assert (np.abs(np64(x)[:, :D] - want) <= scale * 200 * 2.0 ** -24 + np.abs(want) * 2.0 ** -8).all()
    assert (x[:, D:] == 0).all() and (r_out[:, D:] == 0).all()


@pytest.mark.parametrize("D", [8, 64, 300, 768, 1000, 5120, 10240])
@pytest.mark.parametrize("post,pre,gate,res,bias", [
    ("rms", "rms", "row", BF, False), ("layer", "rms", None, torch.float32, True), ("none", "layer", "all", torch.float32, True),
    ("rms", "none", "all", BF, True), ("rms", "layer", "row", torch.float32, True)])
def test_norm_many_rows_are_each_row_alone(D, post, pre, gate, res, bias):
    """Enough rows for every CTA to walk several: each equals the same row in a call of its own to a few roundings (the
    orders of summation and of the factors differ), the outputs' own rounding aside; the last rows and r_out = r_in."""
    g = gen_of(D)
    M, kind = 1401, {"none": 0, "rms": 1, "layer": 2}
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    y, r0 = rnd(M, D) * 3, (rnd(M, D) * 2).to(res)
    pw, qw = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
    pb, qb = (rnd(D), rnd(D)) if bias else (None, None)
    gt = None if gate is None else rnd(1 if gate == "row" else M, D)
    t = q4k.Q4K_RES_FP32 if res == torch.float32 else q4k.Q4K_RES_BF16

    def call(y, gt, r, r_out, x):
        q4k.q4k_norm_residual(y.shape[0], D, y, D, kind[post], pw, pb, 1e-5, gt, D if gate == "all" else 0, 0.7, r, r_out, D, t,
                              kind[pre], qw, qb, 1e-6, x, D)

    r, x = r0.clone(), torch.zeros(M, D, dtype=BF, device="cuda")
    call(y, gt, r, r, x)
    q4k.q4k_check_device()
    for m in [0, 1, 303, 304, 700, M - 2, M - 1]:
        r1, x1 = torch.zeros(1, D, dtype=res, device="cuda"), torch.zeros(1, D, dtype=BF, device="cuda")
        call(y[m:m + 1], gt[m:m + 1] if gate == "all" else gt, r0[m:m + 1], r1, x1)
        for got, want in ((r[m], r1[0]), (x[m], x1[0])):
            scale = want.double().abs() + want.double().pow(2).mean().sqrt()
            tol = scale * 100 * 2.0 ** -24 + (want.double().abs() * 2.0 ** -7 if want.dtype == BF else 0)  # (one step of bf16)
            assert ((got.double() - want.double()).abs() <= tol).all()
    full = R.norm_residual(np64(y), kind[post], np64(pw), None if pb is None else np64(pb), 1e-5, None if gt is None else np64(gt),
                           0.7, np64(r0), kind[pre], np64(qw), None if qb is None else np64(qb), 1e-6)
    for got, want in ((np64(r), full[0]), (np64(x), full[1])):
        assert np.linalg.norm(got - want) <= np.linalg.norm(want) * (2.0 ** -9 + 1e-6)


@pytest.mark.parametrize("res", [torch.float32, BF])
@pytest.mark.parametrize("D", [96, 101, 20000])
def test_norm_in_place_and_parts(res, D):
    """r_out = r_in; no block output; no residual kept; no next norm."""
    g = gen_of(41)
    y, r0 = torch.randn(6, D, generator=g, device="cuda"), torch.randn(6, D, generator=g, device="cuda").to(res)
    t = q4k.Q4K_RES_FP32 if res == torch.float32 else q4k.Q4K_RES_BF16
    a, b, x, x2 = r0.clone(), torch.zeros_like(r0), torch.zeros(6, D, dtype=BF, device="cuda"), torch.zeros(6, D, dtype=BF, device="cuda")
    call = lambda y, r, ro, x: q4k.q4k_norm_residual(6, D, y, D, 1, None, None, 1e-6, None, 0, 0.5, r, ro, D, t, 1, None, None, 1e-6, x, D)  # noqa: E731
    call(y, r0, b, x)
    call(y, a, a, x2)
    assert torch.equal(a, b) and torch.equal(x, x2)
    call(y, r0, None, x2)
    assert torch.equal(x, x2)
    c = torch.zeros_like(r0)
    call(y, r0, c, None)
    assert torch.equal(c, b)
    call(None, r0, c, x)
    want = R.norm_residual(None, 1, None, None, 0, None, 1.0, np64(r0), 1, None, None, 1e-6)[1]
    assert torch.equal(c, r0) and (np.abs(np64(x) - want) <= np.abs(want) * 2.0 ** -8 + 1e-6).all()


def test_norm_large_means_and_rows_without_a_number():
    """A mean far above the spread; a row with NaN or infinity stays its own affair."""
    g = gen_of(42)
    y = torch.randn(4, 512, generator=g, device="cuda") + 1e4
    y[2, 5], y[3, 7] = float("nan"), float("inf")
    r = torch.zeros(4, 512, device="cuda")
    out, x = torch.zeros_like(r), torch.zeros(4, 512, dtype=BF, device="cuda")
    q4k.q4k_norm_residual(4, 512, y, 512, 2, None, None, 0.0, None, 0, 1.0, r, out, 512, q4k.Q4K_RES_FP32, 0, None, None, 0.0, x, 512)
    want = R.norm_residual(np64(y[:2]), 2, None, None, 0.0, None, 1.0, np.zeros((2, 512)), 0, None, None, 0)[0]
    # the mean is known to 2^-24 * 1e4 * (depth 16): that much, in units of the spread, is left in every value
    assert np.abs(np64(out[:2]) - want).max() <= 1e4 * 16 * 2.0 ** -24
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).any()


@pytest.mark.parametrize("D", [256, 776, 1536, 2048, 4096, 8192])
@pytest.mark.parametrize("post,pre,gate,res,bias", [
    ("layer", "layer", None, BF, True), ("layer", "rms", "all", BF, True), ("rms", "layer", "row", torch.float32, False)])
def test_norm_many_rows_of_more_widths(D, post, pre, gate, res, bias):
    """Widths that fill every thread and widths that do not; biases beside the ring, and rings that they leave no room for."""
    test_norm_many_rows_are_each_row_alone(D, post, pre, gate, res, bias)


@pytest.mark.parametrize("D", [768, 1000, 5120])
def test_norm_many_rows_with_large_means(D):
    """The mean is known to 2^-24 of itself and each addition on the way (up to 16 of a thread's values, 5 and 5 of a tree,
    and as many for the warps' parts)."""
    g = gen_of(42)
    M, shift = 700, 1e4
    y = torch.randn(M, D, generator=g, device="cuda") + shift
    y[5, 0] = -3e5  # far from all others
    r, x = torch.zeros(M, D, device="cuda"), torch.zeros(M, D, dtype=BF, device="cuda")
    q4k.q4k_norm_residual(M, D, y, D, 2, None, None, 0.0, None, 0, 1.0, r, r, D, q4k.Q4K_RES_FP32, 0, None, None, 0.0, x, D)
    want = R.norm_residual(np64(y), 2, None, None, 0.0, None, 1.0, np.zeros((M, D)), 0, None, None, 0)[0]
    spread = np64(y).std(axis=1, keepdims=True)
    assert (np.abs(np64(r) - want) * spread <= shift * 32 * 2.0 ** -24 + np.abs(want) * spread * 64 * 2.0 ** -24).all()


# ---------------------------------------------------------------- sample

def run_sample(z, t=None, k=None, p=None, m=None, u=None, ld=None):
    M, V = z.shape
    f = lambda a: None if a is None else torch.as_tensor(a, dtype=torch.float32, device="cuda").expand(M).contiguous()  # noqa: E731
    k = None if k is None else torch.as_tensor(k, dtype=torch.int32, device="cuda").expand(M).contiguous()
    token = torch.full((M,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((M,), -9.0, device="cuda")
    q4k.q4k_sample(z, M, V, z.stride(0), f(t), k, f(p), f(m), f(u), token, prob)
    return token.tolist(), prob.tolist()


def check_sample(z, t, k, p, m, u, got=None):
    token, prob = got or run_sample(z, t, k, p, m, u)
    rows = z.cpu().numpy()
    at = lambda a, i, none: none if a is None else float(np.float32(a[i] if hasattr(a, "__len__") else a))  # noqa: E731
    for i in range(len(rows)):
        want, pw = R.sample(rows[i], at(t, i, 1.0), int(at(k, i, 0)), at(p, i, 1.0), at(m, i, 0.0), at(u, i, 0.0))
        assert token[i] == want, (i, token[i], want)
        assert abs(prob[i] - pw) <= 3 * 2.0 ** -24 * pw, (i, prob[i], pw)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.9, 0.0), (1.3, 0, 0.95, 0.02), (0.9, 7, 1.0, 0.1), (0.0, 9, 0.5, 0.3), (1.0, 1, 0.3, 0.0),
            (100.0, 700, 1.0, 0.0), (100.0, 0, 0.37, 0.0), (0.01, 0, 0.999, 0.0), (1.0, 0, 0.0, 0.0), (3.0, 900, 0.6, 0.5)]


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4096, 4097, 9001, 20003])
@pytest.mark.parametrize("t,k,p,m", SETTINGS)
def test_sample(V, t, k, p, m):
    g = gen_of(V)
    M = 3
    z = torch.randn(M, V, generator=g, device="cuda") * 2.5
    z[:, ::max(1, V // 7)] += 5
    u = torch.rand(M, generator=g, device="cuda").tolist()
    check_sample(z, t, k, p, m, u)


@pytest.mark.parametrize("kind", ["equal", "two values", "ties at the cut", "one", "masked", "none", "inf", "nan", "wide", "zeros",
                                  "close"])
@pytest.mark.parametrize("V", [700, 6001, 30011])
def test_sample_hard_rows(kind, V):
    """Rows in which many logits are equal, masked, infinite, no number, or a few units in the last place apart."""
    g = gen_of(V + 1)
    z = torch.randn(4, V, generator=g, device="cuda")
    if kind == "equal":
        z.fill_(-3.25)
    elif kind == "two values":
        z = torch.where(z > 0.5, 1.0, 0.75)
    elif kind == "ties at the cut":
        z = torch.round(z * 2) / 2
    elif kind == "one":
        z.fill_(-float("inf"))
        z[:, V // 3] = -1e30
    elif kind == "masked":
        z[:, V // 9:] = torch.finfo(torch.float32).min
        z[1, :] = torch.finfo(torch.float32).min
    elif kind == "none":
        z.fill_(-float("inf"))
        z[1] = float("nan")
    elif kind == "inf":
        z[:, ::50] = float("inf")
        z[1] = -float("inf")
        z[1, 5] = float("inf")
    elif kind == "nan":
        z[:, ::3] = float("nan")
    elif kind == "wide":
        z *= 1e30
    elif kind == "zeros":
        z = torch.where(z > 0, 0.0, -0.0)
    elif kind == "close":
        z = 1.0 + torch.randint(0, 400, (4, V), generator=g, device="cuda") * 2.0 ** -23
    z = z.float().contiguous()
    for t, k, p, m in ((1.0, 0, 1.0, 0.0), (1.0, 40, 0.9, 0.0), (0.8, 0, 0.5, 0.0), (1.0, 601, 0.99, 0.01), (0.0, 0, 1.0, 0.0)):
        check_sample(z, t, k, p, m, [0.0, 0.3, 0.77, 1 - 2.0 ** -24])


def test_sample_long_rows_strides_and_row_settings():
    """A vocabulary beyond the shared memory, odd strides, and each row with its own settings."""
    g = gen_of(51)
    for V, M in ((200003, 4), (151936, 3)):
        raw = torch.randn(M, V + 3, generator=g, device="cuda") * 2.2
        z = raw[:, 1:V + 1] if V % 2 else raw[:, :V]
        check_sample(z, [0.7, 1.0, 0.0, 1.2][:M], [50, 0, 3, 5000][:M], [0.9, 0.95, 1.0, 0.5][:M], [0.0, 0.02, 0.0, 0.0][:M],
                     torch.rand(M, generator=g, device="cuda").tolist())


def test_sample_settings_out_of_range():
    g = gen_of(52)
    z = torch.randn(8, 500, generator=g, device="cuda")
    nan = float("nan")
    check_sample(z, [nan, -1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0], [0, 0, -5, 10 ** 9, 0, 0, 0, 0], [1.0, 1.0, nan, 7.0, -2.0, 0.9, 1.0, 1.0],
                 [0.0, 0.0, nan, 0.0, 0.0, 2.0, -1.0, 0.0], [0.5, 0.5, 0.5, 0.5, 0.5, nan, 1.0, -3.0])


def test_sample_defaults_and_no_prob():
    g = gen_of(53)
    z = torch.randn(2, 3000, generator=g, device="cuda")
    u = torch.tensor([0.2, 0.9], device="cuda")
    token = torch.zeros(2, dtype=torch.int32, device="cuda")
    q4k.q4k_sample(z, 2, 3000, 3000, None, None, None, None, u, token)
    check_sample(z, None, None, None, None, u.tolist(), (token.tolist(), run_sample(z, u=u)[1]))


@pytest.mark.parametrize("order", ["falling", "rising", "runs"])
@pytest.mark.parametrize("V", [128, 1500, 6001, 40003])
def test_sample_rows_in_order(order, V):
    """Logits in order, so that the largest of a stretch say little about the k-th; k about the largest that they bound."""
    g = gen_of(V + 2)
    z = torch.sort(torch.randn(4, V, generator=g, device="cuda") * 2, dim=1, descending=order == "falling").values
    if order == "runs":
        z = z.view(4, -1).roll(V // 3, 1)
    z = z.contiguous()
    for k in (1, 2, 95, 96, 97, 128):
        for p, m in ((1.0, 0.0), (0.9, 0.0), (0.97, 0.05), (1.0, 0.2)):
            check_sample(z, [1.0, 0.5, 2.0, 0.9], k, p, m, [0.0, 0.4, 0.8, 1 - 2.0 ** -24])


@pytest.mark.parametrize("near", [254, 255, 256, 257, 2000])
def test_sample_tokens_that_min_p_keeps(near):
    """As many tokens in reach of min-p as are ranked at once, one more, and many; top-p ends before, at and beyond them."""
    V = 12007
    g = gen_of(near)
    for bulk in (-3.0, -9.0):
        z = bulk + 0.1 * torch.randn(6, V, generator=g, device="cuda").clamp(-3, 3)
        at = torch.randperm(V, generator=g, device="cuda")[:near + 1]
        z[:, at] = -0.5 * torch.rand(6, near + 1, generator=g, device="cuda")
        z[:, at[0]] = 0.0
        z = z.contiguous()
        u = [0.0, 0.2, 0.5, 0.7, 0.95, 1 - 2.0 ** -24]
        for p in (0.05, 0.5, 0.9, 0.999, 1.0):
            for k in (0, 60, near):
                check_sample(z, 1.0, k, p, 0.3, u)


@pytest.mark.parametrize("V", [4097, 9001, 17003, 39001, 80021])
def test_sample_many_rows(V):
    """So many rows that fewer CTAs share one."""
    g = gen_of(V + 3)
    M = 310 if V < 5000 else 160
    z = torch.randn(M, V, generator=g, device="cuda") * 2.5
    k = [(0, 50, 1, 300)[i % 4] for i in range(M)]
    p = [(0.9, 1.0, 0.5)[i % 3] for i in range(M)]
    m = [(0.0, 0.02, 0.0, 0.0, 0.1)[i % 5] for i in range(M)]
    check_sample(z, 0.8, k, p, m, torch.rand(M, generator=g, device="cuda").tolist())


@pytest.mark.parametrize("M,V", [(21, 156011), (2, 390001)])
def test_sample_rows_beyond_shared_memory(M, V):
    g = gen_of(V)
    z = torch.randn(M, V, generator=g, device="cuda") * 2.2
    k = [(50, 0, 3, 5000)[i % 4] for i in range(M)]
    p = [(0.9, 0.95, 1.0)[i % 3] for i in range(M)]
    m = [(0.0, 0.02)[i % 2] for i in range(M)]
    check_sample(z, 1.0, k, p, m, torch.rand(M, generator=g, device="cuda").tolist())


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_sample_rows_off_16_bytes(offset):
    """What lies before and behind a row in its first and last 16 bytes is no part of it."""
    g = gen_of(60 + offset)
    for V in (1, 2, 3, 4, 5, 6, 7, 1030, 4098, 16391):
        raw = torch.full((3, V + 8), float("inf"), device="cuda")
        z = raw[:, offset:offset + V]
        z.copy_(torch.randn(3, V, generator=g, device="cuda") * 2)
        for k, p, m in ((0, 1.0, 0.0), (2, 1.0, 0.0), (0, 0.8, 0.0), (0, 0.9, 0.1)):
            check_sample(z, 1.0, k, p, m, torch.rand(3, generator=g, device="cuda").tolist())
