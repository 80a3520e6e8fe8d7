"""Refusals of the 8-bit entry points, on the host (fake pointers, no GPU)."""
import ctypes

import pytest
import torch

import block_wise_diffusion_b200 as tt
from block_wise_diffusion_b200 import build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build.build()
    return tt.lib()


def _d(**kw):
    base = dict(B=8, S=16, Hq=32, Hkv=2, dh=128, V=131072, L_cap=4096)
    base.update(kw)
    return tt.Dims(base["B"], base["S"], base["Hq"], base["Hkv"], base["dh"],
                   base.get("H", base["Hq"] * base["dh"]), base["V"], base["L_cap"])


def attn(L, d, f, ptrs=(FAKE,) * 9, ws=FAKE, ws_bytes=1 << 40):
    return L.tt_block_denoise_attn_q8(ctypes.byref(d), f if f is None else ctypes.byref(f), *ptrs,
                                      ws, ws_bytes, None)


def test_workspaces(L):
    d = _d()
    assert tt.tt_workspace_bytes(d, tt.TT_WS_ATTN_Q8) >= 256
    assert tt.tt_workspace_bytes(d, tt.TT_WS_APPEND_Q8) >= 256
    # 128 rows of int8 y, and 16 bytes per row and vocabulary tile
    assert tt.tt_workspace_bytes(d, tt.TT_WS_VOCAB_I8) >= 128 * 4096 + 128 * 16 * (131072 // 224)
    assert L.tt_workspace_bytes(ctypes.byref(d), 7) == 0
    assert tt.tt_linear_i8_workspace_bytes(128, 4608, 4096) >= 128 * 4096 + 128 * 4


@pytest.mark.parametrize("kw,code", [(dict(S=8), 2), (dict(dh=96), 2), (dict(B=0), 1),
                                     (dict(Hkv=3), 1), (dict(L_cap=-1), 1)])
def test_bad_dims(L, kw, code):
    assert attn(L, _d(**kw), tt.q8("int8", 128)) == code
    assert L.tt_workspace_bytes(ctypes.byref(_d(**kw)), tt.TT_WS_ATTN_Q8) == 0


def test_bad_formats(L):
    for f, code in ((tt.Q8(2, 128), 2), (tt.Q8(-1, 128), 2), (tt.Q8(0, 0), 2), (tt.Q8(0, 8), 2),
                    (tt.Q8(1, 48), 2), (tt.Q8(1, 256), 2)):
        assert attn(L, _d(), f) == code
    assert attn(L, _d(), None) == 1
    with pytest.raises(KeyError):
        tt.q8("int4", 128)


@pytest.mark.parametrize("i,name,align", [(0, "q_blk", 16), (1, "k_blk", 16), (2, "v_blk", 16),
                                          (3, "k_ctx", 16), (4, "v_ctx", 16), (5, "k_scale", 4),
                                          (6, "v_scale", 4), (7, "ctx_len", 4), (8, "out", 16)])
def test_attention_pointers(L, i, name, align):
    p = [FAKE] * 9
    p[i] = None
    assert attn(L, _d(), tt.q8("int8", 64), p) == 1 and name in tt.tt_last_error()
    p[i] = FAKE + align // 2
    assert attn(L, _d(), tt.q8("int8", 64), p) == 1 and "aligned" in tt.tt_last_error()


def test_longest_context(L):
    """Lengths are rounded up to whole tiles in 32 bits."""
    d, st = _d(B=1, Hq=2, dh=64, L_cap=(1 << 31) - 1), (64, 64, 64)
    d.Hkv, d.Hq, d.H = 1, 1, 64
    for f in (tt.q8("int8", 16), tt.q8("e4m3", 128)):
        assert attn(L, d, f) == 2 and "L_cap" in tt.tt_last_error()
        assert append(L, d=d, f=f, st=st) == 2 and "L_cap" in tt.tt_last_error()


def test_attention_workspace(L):
    need = tt.tt_workspace_bytes(_d(), tt.TT_WS_ATTN_Q8)
    assert attn(L, _d(), tt.q8("int8", 64), ws_bytes=need - 1) == 3
    assert attn(L, _d(), tt.q8("int8", 64), ws=FAKE + 16, ws_bytes=need) == 1
    assert attn(L, _d(), tt.q8("int8", 64), ws=None, ws_bytes=need) == 1


def append(L, d=None, f=None, n=16, new_len=None, k=FAKE, v=FAKE, st=(1024, 64, 8), caches=None,
           ws_bytes=1 << 20):
    s = tt._RowStrides(*st) if st is not None else None
    return L.tt_append_ctx_q8(ctypes.byref(d or _d()), ctypes.byref(f or tt.q8("e4m3", 32)), n,
                              new_len, k, v, None if s is None else ctypes.byref(s),
                              *(caches or [FAKE] * 5), FAKE, ws_bytes, None)


def test_append_refusals(L):
    assert append(L, n=0) == 1 and append(L, n=4097) == 1 and append(L, n=-3) == 1
    assert append(L, d=_d(L_cap=0), n=1) == 1
    assert append(L, k=None) == 1 and append(L, v=FAKE + 8) == 1
    assert append(L, new_len=FAKE + 2) == 1 and "new_len" in tt.tt_last_error()
    assert append(L, st=None) == 1 and "strides" in tt.tt_last_error()
    for st in ((1028, 64, 8), (1024, 68, 8), (1024, 64, 4)):
        assert append(L, st=st) == 1 and "multiples of 8" in tt.tt_last_error()
    assert append(L, f=tt.Q8(0, 17)) == 2
    assert append(L, ws_bytes=255) == 3
    for i in range(5):
        c = [FAKE] * 5
        c[i] = None
        assert append(L, caches=c) == 1


def test_linear_and_quantise_refusals(L):
    q = lambda r, k, x=FAKE, c=FAKE, s=FAKE: L.tt_quantize_rows_i8(r, k, x, c, s, None)  # noqa: E731
    assert q(0, 64) == 1 and q(-1, 64) == 1 and q(4, 0) == 1
    assert q(4, 24) == 2 and q(4, 131088) == 2 and q(1 << 24, 16) == 2
    assert q(4, 64, x=None) == 1 and q(4, 64, c=FAKE + 8) == 1 and q(4, 64, s=FAKE + 2) == 1
    lin = lambda m, n, k, p=(FAKE,) * 4, wsb=1 << 40: L.tt_linear_i8(m, n, k, *p, FAKE, wsb, None)  # noqa: E731
    assert lin(0, 8, 64) == 1 and lin(8, 0, 64) == 1 and lin(8, 8, 40) == 2
    assert lin(8, 1 << 24, 64) == 2
    for i in range(4):
        p = [FAKE] * 4
        p[i] = FAKE + 8
        assert lin(8, 8, 64, p) == 1 and "aligned" in tt.tt_last_error()
    assert lin(8, 8, 64, wsb=255) == 3
    assert L.tt_linear_i8_workspace_bytes(8, 8, 40) == 0
    with pytest.raises(tt.TTError):
        tt.tt_linear_i8_workspace_bytes(0, 8, 64)


def test_vocab_refusals(L):
    d = _d()
    need = tt.tt_workspace_bytes(d, tt.TT_WS_VOCAB_I8)

    def call(gamma=0.8, scale=1.0, y=FAKE, w=FAKE, ws=FAKE, tok=FAKE, m=FAKE, wsb=need, dd=d):
        return L.tt_vocab_confidence_commit_i8(ctypes.byref(dd), y, w, ws, gamma, scale, tok, m,
                                               FAKE, FAKE, FAKE, FAKE, wsb, None)
    assert call(gamma=0.0) == 1 and call(gamma=1.5) == 1 and call(scale=0.0) == 1
    assert call(scale=float("inf")) == 1 and call(y=None) == 1 and call(w=FAKE + 4) == 1
    assert call(ws=FAKE + 8) == 1 and call(tok=None) == 1 and call(m=None) == 1
    assert call(wsb=need - 1) == 3 and call(dd=_d(V=1)) == 1


def test_binding_checks_shapes(L):
    d, f = _d(B=2, Hq=4, Hkv=2, dh=64, V=1000, L_cap=50), tt.q8("int8", 16)
    R, ctx, ns = 32, 2 * 2 * 50 * 64, 2 * 2 * 4 * 4
    need = dict(q_blk=R * 4 * 64 * 2, k_blk=R * 2 * 64 * 2, v_blk=R * 2 * 64 * 2, k_ctx=ctx,
                v_ctx=ctx, k_scale=ns, v_scale=ns, ctx_len=8, out=R * 4 * 64 * 2)
    for name, nbytes in need.items():
        for n, message in ((nbytes, "CUDA tensors only"), (nbytes - 1, "holds")):
            kw = {k: FAKE for k in need}
            kw[name] = torch.zeros(n, dtype=torch.uint8)
            with pytest.raises(ValueError, match=message):
                tt.tt_block_denoise_attn_q8(d, f, **kw, ws=FAKE, stream=0)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        x = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)
        tt.tt_append_ctx_q8(d, f, 3, None, x, x, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0)
    lin = dict(x=4 * 64 * 2, w_q=10 * 64, w_scale=40, out=4 * 10 * 2)
    for name, nbytes in lin.items():
        kw = {k: FAKE for k in lin}
        kw[name] = torch.zeros(nbytes - 1, dtype=torch.uint8)
        with pytest.raises(ValueError, match="holds"):
            tt.tt_linear_i8(4, 10, 64, **kw, ws=FAKE, stream=0)
