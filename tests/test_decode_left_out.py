"""Paged caches with page ids out of range: what lies in such a page is left out of every result, and no result holds
what an earlier call or nobody wrote."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import decode_ref as R
from tests.test_decode_ops import BF, F8, gen_of, np64, pool, run_attn, run_evict, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


def attend(k, v, table, lens, q, scale, window, weights, decay, ks, vs):
    """Attention over the slots whose pages are there, in 64 bits: o, weights, sum p |v|, and the largest sum of products."""
    B, n_q, H, D = q.shape
    pages, Hkv, page, _ = k.shape
    o, mag, big, w = np.zeros(q.shape), np.zeros(q.shape), 0.0, weights.copy()
    for b in range(B):
        n = lens[b]
        w[b, :, :n] *= decay
        j = np.arange(n)
        there = (table[b][j // page] >= 0) & (table[b][j // page] < pages)
        for h in range(H):
            for i in range(n_q):
                end = n - n_q + 1 + i
                begin = max(0, end - window) if window else 0
                at = j[there & (j >= begin) & (j < end)]
                if len(at) == 0:
                    continue
                g = h * Hkv // H
                kk, vv = k[table[b][at // page], g, at % page] * ks, v[table[b][at // page], g, at % page] * vs
                s = kk @ q[b, i, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o[b, i, h], mag[b, i, h] = p @ vv, p @ np.abs(vv)
                big = max(big, (np.abs(kk) @ np.abs(q[b, i, h])).max() * scale)
                w[b, g, at] += p
    return o, w, mag, big


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("n_q,G,window", [(1, 4, 0), (3, 4, 0), (2, 16, 70)])
def test_attn_weights_without_the_slots_of_bad_pages(dtype, D, page, n_q, G, window):
    """Slots of a bad page get decay * weight and nothing else, the others what a cache without them gives: whole steps
    of a warp are missing (pages of 16 and more), whole tiles, and every slot of a sequence.

    Errors: e of a score as for every attention test (D additions of products that sum to big at most, the exponential),
    weights off by e^(2 e); p enters the second product to 2^-16 (e4m3: 2^-11), and o is rounded to bf16."""
    g = gen_of(D + page + n_q)
    Hkv, lens, decay = 2, [5 * page - 3, 8 * page, 3 * page + 1, 700], 0.75
    B, per = len(lens), -(-max(lens) // page)
    pages = B * per
    k, v = pool((pages, Hkv, page, D), dtype, "phsd", g)
    table = table_of(B, per, pages, g)
    bad = table.clone()
    bad[0, 1] = -1
    bad[1, :] = pages                                  # nothing of this sequence is there
    bad[2, 3] = 2 ** 31 - 1                            # the new tokens themselves
    bad[3, 2:5] = -2 ** 31
    bad[3, -(-700 // page) - 2] = pages + 7
    ks, vs = (0.5, 0.25) if dtype == F8 else (1.0, 1.0)
    q = (torch.randn(B, n_q, Hkv * G, D, generator=g, device="cuda") * 2 / ks).to(BF)
    w0 = torch.rand(B, Hkv, per * page, generator=g, device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ids, scale = bad.cpu().numpy(), D ** -0.5
    want, ww, mag, big = attend(np64(k), np64(v), ids, lens, np64(q), scale, window, np64(w0), decay, ks, vs)
    first = None
    for fill in (0x5A, 0x00, 0xFF):                    # whatever the workspace held
        cache = q4k.kv_cache(k, v, bad, ks, vs)
        ws = torch.full((q4k.q4k_attn_decode_workspace_size(cache, Hkv * G, n_q, per * page),), fill, dtype=torch.uint8, device="cuda")
        w = w0.clone()
        o = run_attn(k, v, bad, lt, q, n_q, scale, window=window, weights=w, decay=decay, ks=ks, vs=vs, ws=ws)
        with pytest.raises(q4k.Q4KError) as err:
            q4k.q4k_check_device()
        assert err.value.status == q4k.Q4K_ERR_INDEX
        for b, n in enumerate(lens):
            j = np.arange(per * page)
            page_id = ids[b][j // page]
            out = torch.from_numpy((j < n) & ((page_id < 0) | (page_id >= pages))).cuda()
            assert torch.equal(w[b][:, out], w0[b][:, out] * decay)
            assert torch.equal(w[b, :, n:], w0[b, :, n:])
        e = D * 2.0 ** -24 * big + 2.0 ** -20 * big
        assert (np.abs(np64(w) - ww) <= ww * (2.2 * e + 2.0 ** -14)).all()
        near = 2.2 * e + 2.0 ** -14 + (2.0 ** -11 if dtype == F8 else 0.0)
        assert (np.abs(np64(o) - want) <= mag * near + np.abs(want) * 2.0 ** -8 + 2.0 ** -20).all()
        first = first if first is not None else (o, w)
        assert torch.equal(o, first[0]) and torch.equal(w, first[1])


@pytest.mark.parametrize("dtype", [BF, F8])
def test_attn_scores_of_an_earlier_call_are_not_read(dtype):
    """The same workspace after a call over the whole cache: a page that then goes bad gets no weight from it."""
    g = gen_of(3)
    D, page, per = 128, 64, 6
    k, v = pool((per, 1, page, D), dtype, "phsd", g)
    table = table_of(1, per, per, g)
    q = torch.randn(1, 1, 4, D, generator=g, device="cuda").to(BF)
    lens = torch.tensor([per * page], dtype=torch.int32, device="cuda")
    cache = q4k.kv_cache(k, v, table)
    ws = torch.empty(q4k.q4k_attn_decode_workspace_size(cache, 4, 1, per * page), dtype=torch.uint8, device="cuda")
    w = torch.zeros(1, 1, per * page, device="cuda")
    run_attn(k, v, table, lens, q, 1, 0.1, weights=w, ws=ws)
    q4k.q4k_check_device()
    assert abs(float(w.sum()) - 4) < 1e-3
    table[0, 2] = -1
    w.zero_()
    run_attn(k, v, table, lens, q, 1, 0.1, weights=w, ws=ws)
    with pytest.raises(q4k.Q4KError):
        q4k.q4k_check_device()
    assert (w[0, 0, 2 * page:3 * page] == 0).all() and abs(float(w.sum()) - 4) < 1e-3


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF, 64), (F8, 128)])
@pytest.mark.parametrize("bad", ["from", "to", "both"])
def test_evict_makes_a_move_whole_or_not_at_all(bad, dtype, D, in_place):
    """A move between pages of which one is out of range is not made: the hole keeps its token, key, value, weight and
    position alike, and every other move is made."""
    g = gen_of(5)
    B, Hkv, page, per, budget = 2, 2, 16, 20, 150
    lens = [300, 290]
    k, v = pool((B * per, Hkv, page, D), dtype, "phsd", g)
    table = table_of(B, per, B * per, g)
    if bad != "to":
        table[0, 12], table[1, 15] = -1, B * per         # slots from the budget on: moves come from there
    if bad != "from":
        table[0, 3], table[1, 0] = 2 ** 31 - 1, -7       # slots below it: moves go there
    w = torch.rand(B, Hkv, per * page, generator=g, device="cuda")
    p = torch.stack([torch.randperm(per * page, generator=g, device="cuda") for _ in range(B * Hkv)]).view(B, Hkv, -1).int()
    new, take = R.kv_evict(lens, w.cpu().numpy(), p.cpu().numpy(), budget, 4, 16)
    u8 = lambda t: t.view(torch.uint8) if t.dtype == F8 else t  # noqa: E731
    k0, v0, w0, p0 = u8(k).clone(), u8(v).clone(), w.clone(), p.clone()
    got, wo, po = run_evict(q4k.kv_cache(k, v, table), lens, budget, 4, 16, w, p, in_place)
    with pytest.raises(q4k.Q4KError) as err:
        q4k.q4k_check_device()
    assert err.value.status == q4k.Q4K_ERR_INDEX and got.tolist() == new.tolist()
    ids, refused = table.cpu().numpy(), 0
    for b in range(B):
        for h in range(Hkv):
            for i, j in enumerate(take[b][h]):
                to, at = ids[b, i // page], ids[b, j // page]
                ok = 0 <= to < B * per and 0 <= at < B * per
                refused += not ok and i != j
                j = j if ok else i
                assert wo[b, h, i] == w0[b, h, j] and po[b, h, i] == p0[b, h, j], (b, h, i)
                if 0 <= to < B * per:
                    for now, was in ((u8(k), k0), (u8(v), v0)):
                        assert torch.equal(now[to, h, i % page], was[ids[b, j // page], h, j % page]), (b, h, i)
    assert refused > 4
