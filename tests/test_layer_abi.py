"""Refusals of the norm, cache and attention entry points: every argument is
checked on the host before any HIP call.  Pointer arguments are fake addresses
that are never touched."""
import ctypes

import pytest

from ternary_weight_linear_forward_amd import bitlinear as bl

A, B, C, D, E, F, G = (0x10000 + i * 0x40000000 for i in range(7))  # far apart, 16-byte aligned
BAD, UNS, WS = bl.ERR_INVALID_ARG, bl.ERR_UNSUPPORTED, bl.ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    a = dict(X=A, x_dtype=bl.BF16, M=4, K=100, ldx=100, R=B, ldr=100, w=C, eps=1e-5, H=D, h_dtype=bl.F32, ldh=100, Xq=E,
             q_dtype=bl.I8, ldq=112, layout=bl.LAYOUT_I2, beta=F, stream=None)
    a.update(kw)
    return bl.bitlinear_norm_quantize(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), BAD), (dict(Xq=None), BAD), (dict(beta=None), BAD), (dict(x_dtype=bl.I8), BAD), (dict(h_dtype=bl.I32), BAD),
    (dict(q_dtype=bl.F32), BAD), (dict(M=0), BAD), (dict(M=bl.MAX_M + 1), BAD), (dict(K=0), BAD),
    (dict(K=bl.MAX_K + 1, ldx=1 << 20, ldr=1 << 20, ldh=1 << 20, ldq=1 << 20), BAD), (dict(ldx=99), BAD), (dict(ldr=99), BAD),
    (dict(ldh=99), BAD), (dict(ldq=96), BAD), (dict(ldq=104), BAD), (dict(ldx=1 << 41), BAD), (dict(ldr=1 << 41), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(X=A + 1), BAD), (dict(R=B + 2), BAD),
    (dict(H=D + 2), BAD), (dict(w=C + 2), BAD), (dict(Xq=E + 8), BAD), (dict(beta=F + 2), BAD), (dict(Xq=A + 16), BAD),
    (dict(beta=B + 16), BAD), (dict(H=B + 4), BAD), (dict(H=B, ldh=104), BAD), (dict(H=A, ldh=100), BAD), (dict(w=E), BAD),
    (dict(H=C), BAD), (dict(q_dtype=bl.I8_TILED, layout=9), BAD),
    (dict(q_dtype=bl.I8_TILED, K=65552, ldx=65552, ldr=65552, ldh=65552), UNS),
])
def test_norm_quantize_rejects(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(Xq=None), dict(beta=None), dict(V=None), dict(v_dtype=bl.I8), dict(M=0), dict(K=0), dict(ldq=99), dict(ldv=99),
    dict(V=C + 2), dict(beta=B + 2), dict(V=A + 64), dict(V=B), dict(ldq=1 << 41), dict(M=bl.MAX_M + 1),
])
def test_dequantize_rejects(kw):
    a = dict(Xq=A, ldq=112, beta=B, M=4, K=100, V=C, v_dtype=bl.F32, ldv=100, stream=None)
    a.update(kw)
    assert bl.bitlinear_dequantize_act(**a) == BAD


def bwd(**kw):
    a = dict(dY=A, lddy=100, H=B, h_dtype=bl.BF16, ldh=100, w=C, eps=1e-5, dH=D, lddh=100, M=4, K=100, dX=E, lddx=100, dW=F,
             ws=G, ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return bl.bitlinear_norm_backward(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(dY=None), BAD), (dict(H=None), BAD), (dict(dX=None), BAD), (dict(h_dtype=bl.I8), BAD), (dict(M=0), BAD),
    (dict(K=0), BAD), (dict(lddy=99), BAD), (dict(ldh=99), BAD), (dict(lddh=99), BAD), (dict(lddx=99), BAD),
    (dict(eps=-1e-9), BAD), (dict(eps=NAN), BAD), (dict(dY=A + 2), BAD), (dict(H=B + 1), BAD), (dict(dX=E + 1), BAD),
    (dict(dW=F + 2), BAD), (dict(ws=None), WS), (dict(ws_bytes=3), WS), (dict(ws=G + 4), BAD), (dict(dX=B), BAD),
    (dict(dX=A), BAD), (dict(dW=C), BAD), (dict(dX=D, lddx=104), BAD), (dict(dX=D + 2), BAD), (dict(ws=A), BAD),
    (dict(dW=E), BAD), (dict(dW=D), BAD), (dict(lddy=1 << 41), BAD),
])
def test_norm_backward_rejects(kw, status):
    assert bwd(**kw) == status


def test_norm_backward_workspace():
    assert bl.bitlinear_norm_backward_workspace_bytes(4, 100, 0) == 0
    assert bl.bitlinear_norm_backward_workspace_bytes(4, 100, 1) >= 400
    assert bl.bitlinear_norm_backward_workspace_bytes(0, 100, 1) == -1
    assert bl.bitlinear_norm_backward_workspace_bytes(4, bl.MAX_K + 1, 1) == -1


def test_cache_bytes():
    assert bl.bitlinear_cache_bytes(3, 64, 8, 128) == 3 * 64 * 8 * 128
    assert bl.bitlinear_cache_bytes(3, 128, 32, 100) == 3 * 128 * 32 * 112
    for bad in [(0, 64, 8, 128), (1, 0, 8, 128), (1, 96, 8, 128), (1, 32, 8, 128), (1, 64, 0, 128), (1, 64, 4097, 128),
                (1, 64, 8, 0), (1, 64, 8, 257), (1, 1 << 21, 8, 128), (1 << 31, 64, 8, 128), (1 << 30, 128, 1, 16)]:
        assert bl.bitlinear_cache_bytes(*bad) == -1, bad


def test_cache_block_count():
    assert bl.bitlinear_cache_bytes(1 << 26, 64, 31, 16) == (1 << 26) * 64 * 31 * 16
    assert bl.bitlinear_cache_bytes(1 << 26, 64, 32, 16) == -1


def cache(**kw):
    a = dict(K=A, K_scale=B, V=C, V_scale=D, pages=4, page_tokens=64, heads=2, head_dim=128)
    a.update(kw)
    return bl.Cache(**a)


BAD_CACHES = [dict(K=None), dict(V=None), dict(K_scale=None), dict(V_scale=None), dict(K=A + 8), dict(V=C + 4),
              dict(K_scale=B + 2), dict(page_tokens=65), dict(heads=0), dict(head_dim=300), dict(pages=0), dict(V=A),
              dict(K_scale=A), dict(V_scale=B)]


def write(c=None, **kw):
    a = dict(K=E, ldk_token=256, ldk_head=128, V=F, ldv_token=256, ldv_head=128, dtype=bl.BF16, tokens=7, slots=G, stream=None)
    a.update(kw)
    return bl.bitlinear_cache_write(c or cache(), **a)


def read(c=None, **kw):
    a = dict(slots=G, tokens=7, K=E, ldk_token=256, ldk_head=128, V=F, ldv_token=256, ldv_head=128, dtype=bl.BF16, stream=None)
    a.update(kw)
    return bl.bitlinear_cache_read(c or cache(), **a)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_descriptions_are_checked(kw):
    assert write(cache(**kw)) == BAD and read(cache(**kw)) == BAD and attn(cache(**kw)) == BAD
    assert write(cache(**kw), tokens=0) == BAD


@pytest.mark.parametrize("kw", [dict(K=None), dict(V=None), dict(slots=None), dict(dtype=bl.I8), dict(tokens=-1),
                                dict(tokens=(1 << 24) + 1), dict(K=E + 1), dict(slots=G + 4), dict(ldk_token=-1),
                                dict(ldv_head=1 << 41), dict(K=A), dict(V=B), dict(slots=C)])
def test_cache_write_rejects(kw):
    assert write(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(K=None), dict(V=None), dict(slots=None), dict(dtype=bl.I8), dict(tokens=-1),
                                dict(K=E + 1), dict(slots=G + 4), dict(ldk_token=128), dict(ldk_head=64), dict(ldk_head=0),
                                dict(ldv_token=200), dict(V=E + 256), dict(K=A), dict(V=D), dict(K=G)])
def test_cache_read_rejects(kw):
    assert read(**kw) == BAD


def test_no_tokens_do_nothing():
    assert write(tokens=0) == bl.OK and read(tokens=0) == bl.OK
    assert bl.bitlinear_cache_write(ctypes.POINTER(bl.Cache)(), E, 256, 128, F, 256, 128, bl.F32, 0, G, None) == BAD


def attn(c=None, **kw):
    a = dict(Q=E, dtype=bl.BF16, tokens=6, heads=8, ldq_token=1024, ldq_head=128, seqs=3, q_start=None, max_q=2,
             own_pages=F, ld_pages=2, own_len=F + 0x1000, max_own=100, prefix_pages=F + 0x2000, prefix_len=70, scale=0.1,
             O=G, ldo_token=1024, ldo_head=128, lse=G + 0x1000000, ws=G + 0x2000000, ws_bytes=1 << 28, stream=None)
    a.update(kw)
    return bl.bitlinear_attention(c or cache(), **a)


@pytest.mark.parametrize("kw", [
    dict(Q=None), dict(O=None), dict(own_len=None), dict(own_pages=None), dict(prefix_pages=None), dict(dtype=bl.I32),
    dict(scale=NAN), dict(scale=INF), dict(tokens=0), dict(tokens=5), dict(heads=7), dict(heads=1), dict(heads=0), dict(seqs=0),
    dict(max_q=0), dict(max_own=-1), dict(prefix_len=-1), dict(max_own=(1 << 30) + 1), dict(ld_pages=1), dict(heads=8192),
    dict(prefix_len=(1 << 30) + 1), dict(Q=E + 1), dict(O=G + 1), dict(own_len=F + 2), dict(lse=G + 0x1000002),
    dict(ldo_token=900), dict(ldo_head=100), dict(ldo_head=0), dict(ldq_token=-1), dict(O=E), dict(O=A), dict(lse=G),
    dict(lse=B), dict(O=F), dict(tokens=1 << 20, seqs=1 << 20, max_q=1 << 20, q_start=F + 0x100),
])
def test_attention_rejects(kw):
    assert attn(**kw) == BAD


def test_attention_workspace():
    args = (6, 8, 2, 128, 3, 2, 100, 70)
    need = bl.bitlinear_attention_workspace_bytes(*args)
    assert need >= 0
    if need > 0:
        assert attn(ws=None) == WS and attn(ws_bytes=need - 1) == WS and attn(ws=G + 0x2000004) == BAD
        assert attn(ws=E) == BAD and attn(ws=C) == BAD
    for i, v in [(0, 0), (1, 7), (2, 0), (3, 257), (4, 0), (5, 0), (6, -1), (7, -1)]:
        bad = list(args)
        bad[i] = v
        assert bl.bitlinear_attention_workspace_bytes(*bad) == -1, (i, v)
