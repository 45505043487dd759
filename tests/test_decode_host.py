"""Refusals of the decode-step operators: every call checks its arguments before it touches a device."""
import ctypes

import pytest
import torch

import q4_weight_quantized_gb300 as q4k

A = 1 << 20  # an aligned fake address; never dereferenced by these calls
N, S, L, W = q4k.Q4K_ERR_NULL, q4k.Q4K_ERR_SHAPE, q4k.Q4K_ERR_ALIGN, q4k.Q4K_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


def cache(**a):
    c = dict(k=A, v=A, page_table=A, ld_table=8, n_pages=64, page_stride=2 * 16 * 128, head_stride=16 * 128, slot_stride=128,
             batch=4, max_pages=8, page_size=16, n_kv_heads=2, head_dim=128, dtype=q4k.Q4K_KV_BF16, k_scale=1.0, v_scale=1.0)
    assert not set(a) - set(c)
    return q4k.KvCache(**{**c, **a})


BAD_CACHE = [(dict(k=None), N), (dict(v=None), N), (dict(page_table=None), N), (dict(ld_table=7), S), (dict(n_pages=0), S),
             (dict(page_stride=0), S), (dict(head_stride=-8), S), (dict(slot_stride=64), S), (dict(batch=0), S),
             (dict(batch=65536), S), (dict(max_pages=0), S), (dict(page_size=0), S), (dict(page_size=1 << 28, max_pages=8), S),
             (dict(n_kv_heads=0), S), (dict(n_kv_heads=1025), S), (dict(head_dim=96), S), (dict(dtype=2), S),
             (dict(k_scale=0.0), S), (dict(v_scale=float("nan")), S), (dict(v_scale=float("inf")), S), (dict(k=A + 8), L),
             (dict(v=A + 2), L), (dict(page_table=A + 2), L), (dict(slot_stride=132), L), (dict(head_stride=2052), L),
             (dict(page_stride=4100), L), (dict(dtype=q4k.Q4K_KV_E4M3, slot_stride=136), L)]


def append(lib, c=None, T=4, n_heads=4, q=A, ldq=512, k=A, ldk=256, v=A, ldv=256, seq=A, slot=A, pos=A, rope=A, n_pos=100,
           rope_dim=128, mode=0, q_out=A, ldqo=512, weights=A, positions=A, ld_meta=128):
    return lib.q4k_kv_append(ctypes.byref(c or cache()), T, n_heads, q, ldq, k, ldk, v, ldv, seq, slot, pos, rope, n_pos, rope_dim,
                             mode, q_out, ldqo, weights, positions, ld_meta, None)


def attn(lib, c=None, lens=A, q=A, ldq=512, n_heads=4, n_q=1, scale=0.1, softcap=0.0, window=0, o=A, ldo=512, weights=None,
         ld_weights=0, decay=1.0, ws=A, ws_bytes=1 << 30):
    return lib.q4k_attn_decode(ctypes.byref(c or cache()), lens, q, ldq, n_heads, n_q, scale, softcap, window, o, ldo, weights,
                               ld_weights, decay, ws, ws_bytes, None)


def evict(lib, c=None, lens=A, new=A, budget=64, sinks=4, recent=16, w=A, p=A, wo=A, po=A, ld=128, ws=A, ws_bytes=1 << 30):
    return lib.q4k_kv_evict(ctypes.byref(c or cache()), lens, new, budget, sinks, recent, w, p, wo, po, ld, ws, ws_bytes, None)


def norm(lib, M=2, D=64, y=A, ldy=64, post=1, post_w=A, post_b=A, post_eps=1e-6, gate=A, ld_gate=0, scale=1.0, r=A, r_out=A,
         ldr=64, r_dtype=0, pre=1, pre_w=A, pre_b=A, pre_eps=1e-6, x=A, ldx=64):
    return lib.q4k_norm_residual(M, D, y, ldy, post, post_w, post_b, post_eps, gate, ld_gate, scale, r, r_out, ldr, r_dtype, pre,
                                 pre_w, pre_b, pre_eps, x, ldx, None)


def sample(lib, z=A, M=2, V=100, ldl=100, t=A, k=A, p=A, m=A, u=A, token=A, prob=A):
    return lib.q4k_sample(z, M, V, ldl, t, k, p, m, u, token, prob, None)


@pytest.mark.parametrize("call", [append, attn, evict])
@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_cache(lib, call, change, status):
    assert call(lib, c=cache(**change)) == status


def test_no_cache(lib):
    assert lib.q4k_kv_append(None, 1, 1, A, 128, A, 256, A, 256, A, A, A, None, 0, 0, 0, A, 128, None, None, 0, None) == N
    assert lib.q4k_attn_decode(None, A, A, 512, 4, 1, 0.1, 0.0, 0, A, 512, None, 0, 1.0, A, 1 << 30, None) == N
    assert lib.q4k_kv_evict(None, A, A, 64, 0, 0, A, A, A, A, 128, A, 1 << 30, None) == N
    assert lib.q4k_attn_decode_workspace_size(None, 4, 1, 0) == 0 and lib.q4k_kv_evict_workspace_size(None, 128) == 0


@pytest.mark.parametrize("change,status", [
    (dict(k=None), N), (dict(v=None), N), (dict(seq=None), N), (dict(slot=None), N), (dict(pos=None), N), (dict(rope=None), N),
    (dict(q=None), N), (dict(q_out=None), N), (dict(T=0), S), (dict(T=1 << 31), S), (dict(n_heads=0), S), (dict(ldq=511), S),
    (dict(ldqo=511), S), (dict(ldk=255), S), (dict(ldv=255), S), (dict(rope_dim=130), S), (dict(rope_dim=3), S), (dict(rope_dim=-2), S),
    (dict(n_pos=0), S), (dict(mode=2), S), (dict(ld_meta=0), S), (dict(q=A + 2), L), (dict(k=A + 1), L), (dict(v=A + 2), L),
    (dict(seq=A + 2), L), (dict(rope=A + 2), L), (dict(q_out=A + 1), L), (dict(weights=A + 2), L), (dict(positions=A + 1), L)])
def test_append_refusals(lib, change, status):
    assert append(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(lens=None), N), (dict(q=None), N), (dict(o=None), N), (dict(ws=None), N), (dict(n_heads=3), S), (dict(n_heads=0), S),
    (dict(n_q=0), S), (dict(n_q=65), S), (dict(ldq=511), S), (dict(ldo=504), S), (dict(scale=float("nan")), S),
    (dict(softcap=-1.0), S), (dict(softcap=float("inf")), S), (dict(window=-1), S), (dict(weights=A, ld_weights=0), S),
    (dict(weights=A, ld_weights=128, decay=float("nan")), S), (dict(q=A + 8), L), (dict(o=A + 4), L), (dict(ldq=516), L),
    (dict(ldo=514), L), (dict(weights=A + 2, ld_weights=128), L), (dict(ws=A + 16), L), (dict(lens=A + 1), L), (dict(ws_bytes=1000), W),
    (dict(n_heads=2 * 64, ldq=2 * 64 * 128, ldo=2 * 64 * 128, n_q=32), S)])
def test_attn_refusals(lib, change, status):
    assert attn(lib, **change) == status


def test_attn_workspace(lib):
    c = ctypes.byref(cache())
    a, b = lib.q4k_attn_decode_workspace_size(c, 4, 1, 0), lib.q4k_attn_decode_workspace_size(c, 4, 1, 128)
    assert 0 < a and a % 256 == 0 and b >= a + 4 * 4 * 128 * 4
    assert attn(lib, weights=A, ld_weights=128, ws_bytes=a) == W
    for bad in ((3, 1, 0), (4, 0, 0), (4, 65, 0), (4, 1, -1), (4, 1, 1 << 31)):
        assert lib.q4k_attn_decode_workspace_size(c, *bad) == 0


@pytest.mark.parametrize("change,status", [
    (dict(lens=None), N), (dict(new=None), N), (dict(w=None), N), (dict(p=None), N), (dict(wo=None), N), (dict(po=None), N),
    (dict(ws=None), N), (dict(budget=0), S), (dict(budget=1 << 31), S), (dict(sinks=-1), S), (dict(recent=-1), S),
    (dict(sinks=40, recent=25), S), (dict(sinks=65, recent=0), S), (dict(ld=0), S), (dict(w=A + 2), L), (dict(po=A + 1), L),
    (dict(ws=A + 128), L), (dict(ws_bytes=64), W)])
def test_evict_refusals(lib, change, status):
    assert evict(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(r=None), N), (dict(r_out=None, x=None), N), (dict(M=0), S), (dict(D=0), S), (dict(D=(1 << 20) + 1), S), (dict(ldy=63), S),
    (dict(ldr=63), S), (dict(ldx=63), S), (dict(ld_gate=5), S), (dict(post=3), S), (dict(pre=-1), S), (dict(r_dtype=2), S),
    (dict(post_eps=-1.0), S), (dict(pre_eps=float("nan")), S), (dict(y=A + 2), L), (dict(gate=A + 1), L), (dict(r=A + 2), L),
    (dict(r=A + 2, r_dtype=1, r_out=A + 1), L), (dict(x=A + 1), L), (dict(pre_w=A + 2), L), (dict(post_b=A + 2), L)])
def test_norm_refusals(lib, change, status):
    assert norm(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(z=None), N), (dict(u=None), N), (dict(token=None), N), (dict(M=0), S), (dict(V=0), S), (dict(V=(1 << 22) + 1), S),
    (dict(ldl=99), S), (dict(z=A + 2), L), (dict(t=A + 1), L), (dict(k=A + 2), L), (dict(u=A + 2), L), (dict(token=A + 2), L)])
def test_sample_refusals(lib, change, status):
    assert sample(lib, **change) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device status; a GPU is present")
@pytest.mark.parametrize("call", [append, attn, evict, norm, sample])
def test_no_device(lib, call):
    assert call(lib) == q4k.Q4K_ERR_DEVICE


def test_status_and_descriptor(lib):
    assert q4k.status_string(q4k.Q4K_ERR_INDEX) != q4k.status_string(99)
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    c = q4k.kv_cache(k, k.clone(), torch.zeros(3, 2, dtype=torch.int32), 0.5, 2.0)
    assert (c.n_pages, c.n_kv_heads, c.page_size, c.head_dim, c.batch, c.max_pages, c.dtype) == (6, 2, 16, 64, 3, 2, q4k.Q4K_KV_BF16)
    assert (c.page_stride, c.head_stride, c.slot_stride) == (2 * 16 * 64, 16 * 64, 64) and (c.k_scale, c.v_scale) == (0.5, 2.0)
    for bad in (dict(k=k.float()), dict(v=k[:3]), dict(t=torch.zeros(3, 2)), dict(t=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            q4k.kv_cache(bad.get("k", k), bad.get("v", bad.get("k", k)), bad.get("t", torch.zeros(3, 2, dtype=torch.int32)))
    with pytest.raises(ValueError):
        q4k.kv_cache(k, k, torch.zeros(1, 2, dtype=torch.int32).expand(3, 2))  # one row for all sequences
    wide = torch.zeros(3, 8, dtype=torch.int32)[:, :2]
    assert q4k.kv_cache(k, k, wide).ld_table == 8
