"""Refusals of the operators of a mixed step: every call checks its arguments before it touches a device."""
import ctypes

import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from tests.test_decode_host import A, BAD_CACHE, L, N, S, W, cache, lib  # noqa: F401


def plan(lib, c=None, lens=A, new=A, first=A, held=A, held_out=A, free=A, count=A, count_out=A, T=8, after=A, starts=A, seq=A,
         slot=A, pos=A, ws=A, ws_bytes=1 << 20):
    return lib.q4k_batch_plan(ctypes.byref(c or cache()), lens, new, first, held, held_out, free, count, count_out, T, after,
                              starts, seq, slot, pos, ws, ws_bytes, None)


def norm8(lib, M=2, D=64, y=A, ldy=64, post=1, post_w=A, post_b=A, post_eps=1e-6, gate=A, ld_gate=0, scale=1.0, r=A, r_out=A,
          ldr=64, r_dtype=0, pre=1, pre_w=A, pre_b=A, pre_eps=1e-6, x=A, ldx=64, q=A, s=A):
    return lib.q4k_norm_residual_x8(M, D, y, ldy, post, post_w, post_b, post_eps, gate, ld_gate, scale, r, r_out, ldr, r_dtype,
                                    pre, pre_w, pre_b, pre_eps, x, ldx, q, s, None)


def lora(lib, n=4, N=64, K=64, R=16, a=A, b=A, ranks=A, scales=A, ids=A, x=A, T=8, ldx=64, y=A, ldy=64, ws=A, ws_bytes=1 << 20):
    return lib.q4k_lora_add(n, N, K, R, a, b, ranks, scales, ids, x, T, ldx, y, ldy, ws, ws_bytes, None)


def chunk(lib, c=None, starts=A, lens=A, q=A, T=8, ldq=512, n_heads=4, scale=0.1, softcap=0.0, window=0, o=A, ldo=512, ws=A,
          ws_bytes=1 << 30):
    return lib.q4k_attn_chunk(ctypes.byref(c or cache()), starts, lens, q, T, ldq, n_heads, scale, softcap, window, o, ldo, ws,
                              ws_bytes, None)


@pytest.mark.parametrize("call", [plan, chunk])
@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_cache(lib, call, change, status):  # noqa: F811
    assert call(lib, c=cache(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(starts=None), N), (dict(lens=None), N), (dict(q=None), N), (dict(o=None), N), (dict(ws=None), N), (dict(T=0), S),
    (dict(T=1 << 31), S), (dict(T=1 << 29), S), (dict(n_heads=3), S), (dict(n_heads=0), S), (dict(ldq=511), S), (dict(ldo=504), S),
    (dict(n_heads=2050, ldq=1 << 19, ldo=1 << 19), S), (dict(scale=float("nan")), S), (dict(softcap=-1.0), S),
    (dict(softcap=float("inf")), S), (dict(window=-1), S), (dict(q=A + 8), L), (dict(o=A + 4), L), (dict(ldq=516), L),
    (dict(ldo=514), L), (dict(ws=A + 16), L), (dict(lens=A + 1), L), (dict(starts=A + 2), L), (dict(ws_bytes=1000), W)])
def test_chunk_refusals(lib, change, status):  # noqa: F811
    assert chunk(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(lens=None), N), (dict(new=None), N), (dict(held=None), N), (dict(held_out=None), N), (dict(free=None), N),
    (dict(count=None), N), (dict(count_out=None), N), (dict(after=None), N), (dict(starts=None), N), (dict(seq=None), N),
    (dict(slot=None), N), (dict(pos=None), N), (dict(ws=None), N), (dict(T=0), S), (dict(T=1 << 31), S), (dict(lens=A + 2), L),
    (dict(first=A + 1), L), (dict(free=A + 2), L), (dict(count_out=A + 2), L), (dict(pos=A + 1), L), (dict(ws=A + 64), L),
    (dict(ws_bytes=256), W)])
def test_plan_refusals(lib, change, status):  # noqa: F811
    assert plan(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(r=None), N), (dict(q=None), N), (dict(s=None), N), (dict(M=0), S), (dict(D=0), S), (dict(D=48, ldy=64), S),
    (dict(D=(1 << 20) + 32), S), (dict(ldy=63), S), (dict(ldr=63), S), (dict(ldx=63), S), (dict(ld_gate=5), S), (dict(post=3), S),
    (dict(pre=-1), S), (dict(r_dtype=2), S), (dict(post_eps=-1.0), S), (dict(pre_eps=float("nan")), S), (dict(y=A + 2), L),
    (dict(x=A + 1), L), (dict(q=A + 2), L), (dict(s=A + 2), L)])
def test_norm8_refusals(lib, change, status):  # noqa: F811
    assert norm8(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(a=None), N), (dict(b=None), N), (dict(ids=None), N), (dict(x=None), N), (dict(y=None), N), (dict(ws=None), N),
    (dict(n=0), S), (dict(n=1025), S), (dict(N=0), S), (dict(N=(1 << 21) + 1, ldy=1 << 22), S), (dict(K=60), S), (dict(K=0), S),
    (dict(R=12), S), (dict(R=0), S), (dict(R=136), S), (dict(T=0), S), (dict(T=(1 << 23) + 1), S), (dict(ldx=56), S),
    (dict(ldy=63), S), (dict(a=A + 8), L), (dict(b=A + 2), L), (dict(x=A + 8), L), (dict(ldx=68), L), (dict(y=A + 2), L),
    (dict(ids=A + 2), L), (dict(ranks=A + 1), L), (dict(scales=A + 2), L), (dict(ws=A + 16), L), (dict(ws_bytes=64), W)])
def test_lora_refusals(lib, change, status):  # noqa: F811
    assert lora(lib, **change) == status


def test_workspaces(lib):  # noqa: F811
    assert lib.q4k_batch_plan_workspace_size(None) == 0
    assert lib.q4k_batch_plan_workspace_size(ctypes.byref(cache(head_dim=96))) == 0
    assert lib.q4k_batch_plan_workspace_size(ctypes.byref(cache())) % 256 == 0
    c = ctypes.byref(cache())
    a = lib.q4k_attn_chunk_workspace_size(c, 8, 4)
    assert a > 0 and a % 256 == 0 and lib.q4k_attn_chunk_workspace_size(c, 1 << 20, 4) >= a + (1 << 20) * 2 // 256 * 12
    for bad in ((0, 4), (8, 3), (1 << 31, 4), (8, 0)):
        assert lib.q4k_attn_chunk_workspace_size(c, *bad) == 0
    assert lib.q4k_attn_chunk_workspace_size(None, 8, 4) == 0
    assert lib.q4k_lora_add_workspace_size(4, 64, 64, 16, 8) >= 8 * 16 * 4
    assert lib.q4k_lora_add_workspace_size(4, 64, 64, 16, 1000) >= 1000 * (16 + 1) * 4
    for bad in ((0, 64, 64, 16, 8), (4, 0, 64, 16, 8), (4, 64, 60, 16, 8), (4, 64, 64, 15, 8), (4, 64, 64, 16, 0)):
        assert lib.q4k_lora_add_workspace_size(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device status; a GPU is present")
@pytest.mark.parametrize("call", [plan, norm8, lora, chunk])
def test_no_device(lib, call):  # noqa: F811
    assert call(lib) == q4k.Q4K_ERR_DEVICE
