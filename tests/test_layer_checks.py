"""Argument checks of the layer and norm calls, on a machine without a GPU: a table is stood in for
by a record laid out like ``struct lora_table``, whose pointers are never followed by a call that the
checks refuse.  A call that passes every check gets as far as asking for the current device, which
fails here (LORA_ERR_CUDA); with a device present these tests are skipped."""
import ctypes

import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the stand-in table must not reach a device")

P = 1 << 20          # any aligned address
OK = L.LORA_ERR_CUDA


class Table(ctypes.Structure):
    """``struct lora_table`` (lora_internal.h); the four vectors and the last one are not touched."""

    _fields_ = ([(k, ctypes.c_int32) for k in ("n", "h", "o", "dtype", "max_rank", "min_rank", "device", "pad")]
                + [("d_desc", ctypes.c_void_p), ("d_status", ctypes.c_void_p), ("vectors", ctypes.c_uint8 * 96)]
                + [(k, ctypes.c_void_p) for k in ("d_tmaps", "d_tmaps_pfA", "d_tmaps_pfB")]
                + [("sigma_kind", ctypes.c_int32), ("tail", ctypes.c_uint8 * 64)])


def table(dtype=L.LORA_BF16, **kw):
    t = Table(n=4, h=256, o=512, dtype=dtype, max_rank=16, min_rank=16, device=0, d_desc=P, d_status=P, d_tmaps=P,
              d_tmaps_pfA=P, d_tmaps_pfB=P)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def code(fn, *a):
    try:
        fn(*a)
    except L.LoraError as e:
        return e.code
    return L.LORA_OK


def bgmv(t=None, ids=P, T=8, x=2 * P, ldx=256, W=3 * P, ldw=256, epi=None, y=4 * P, ldy=512, off=0, ws=5 * P,
         ws_bytes=1 << 19):
    t = t or table()
    return code(L.lora_bgmv_layer, ctypes.addressof(t), ids, T, x, ldx, W, ldw, epi, y, ldy, off, ws, ws_bytes, 0)


def sgmv(t=None, perm=None, ptr=P, T=8, x=2 * P, ldx=256, W=3 * P, ldw=256, epi=None, y=4 * P, ldy=512, off=0,
         ws=5 * P, ws_bytes=1 << 19):
    t = t or table()
    seg = L.make_segments(perm, ptr, P, P, T, 4)
    return code(L.lora_sgmv_layer, ctypes.addressof(t), seg, x, ldx, W, ldw, epi, y, ldy, off, ws, ws_bytes, 0)


@pytest.mark.parametrize("call", [bgmv, sgmv])
def test_layer_arguments(call):
    I, U, WS = L.LORA_ERR_INVALID_ARG, L.LORA_ERR_UNSUPPORTED, L.LORA_ERR_WORKSPACE
    assert call() == OK
    assert call(T=0) == L.LORA_OK
    assert call(T=-1) == I
    assert call(x=None) == I and call(y=None) == I and call(W=None) == I
    assert call(ldx=248) == I and call(ldw=248) == I and call(ldy=504) == I and call(off=8) == I and call(off=-8) == I
    assert call(x=2 * P + 8) == U and call(W=3 * P + 2) == U and call(y=4 * P + 4) == U
    assert call(ldx=260) == U and call(ldw=260) == U and call(ldy=516) == U and call(ldy=600, off=4) == U
    assert call(ws=None) == WS and call(ws_bytes=256) == WS and call(ws=5 * P + 8) == U
    assert call(t=table(dtype=L.LORA_F32, d_tmaps_pfA=None, d_tmaps_pfB=None)) == U
    assert call(t=table(sigma_kind=L.LORA_SIGMA_DIAG)) == U
    assert call(t=table(d_desc=None)) == I
    # wide strides and a slice of a fused output
    assert call(ldx=1024, ldw=264, ldy=2048, off=1024) == OK


def test_layer_forms():
    assert sgmv(perm=P) == L.LORA_ERR_UNSUPPORTED
    assert sgmv(ptr=None) == L.LORA_ERR_INVALID_ARG
    # a table that the tensor-core path of long segments does not take still has the per-token form
    t = table(d_tmaps_pfA=None, d_tmaps_pfB=None, max_rank=128)
    assert sgmv(t=t) == L.LORA_ERR_UNSUPPORTED and bgmv(t=t) == OK
    assert bgmv(ids=None, ws=None, ws_bytes=0) == OK


@pytest.mark.parametrize("call", [bgmv, sgmv])
def test_epilogue_arguments(call):
    I, U = L.LORA_ERR_INVALID_ARG, L.LORA_ERR_UNSUPPORTED
    E = L.make_epilogue
    assert call(epi=E(bias=6 * P, act=L.LORA_ACT_GELU, mul=7 * P, ldmul=512, residual=8 * P, ldres=520)) == OK
    assert call(epi=E(act=5)) == I and call(epi=E(act=-1)) == I
    assert call(epi=E(mul=7 * P, ldmul=504)) == I and call(epi=E(residual=7 * P, ldres=504)) == I
    assert call(epi=E(mul=7 * P, ldmul=516)) == U and call(epi=E(residual=7 * P, ldres=516)) == U
    assert call(epi=E(bias=6 * P + 2)) == U and call(epi=E(mul=6 * P + 2, ldmul=512)) == U
    assert call(epi=E(residual=6 * P + 2, ldres=512)) == U
    # an update in place, and nothing else that touches y
    y = 4 * P
    assert call(epi=E(residual=y, ldres=512)) == OK and call(epi=E(mul=y, ldmul=512)) == OK
    assert call(epi=E(residual=y + 16, ldres=512)) == I and call(epi=E(residual=y - 1024, ldres=512)) == I
    assert call(epi=E(mul=y + 2048, ldmul=1024)) == I
    # y is columns [512, 1024) of a fused buffer; its neighbours are free, columns that meet it are not
    fused = dict(ldy=1536, off=512)
    assert call(epi=E(residual=y, ldres=1536), **fused) == OK
    assert call(epi=E(residual=y + 2048, ldres=1536), **fused) == OK
    assert call(epi=E(residual=y + 1024, ldres=1536), **fused) == OK          # y itself
    assert call(epi=E(residual=y + 1040, ldres=1536), **fused) == I
    assert call(epi=E(residual=y + 16, ldres=1536), **fused) == I
    assert call(x=y, ldx=1536, **fused) == OK
    assert call(x=y + 1024, ldx=1536, **fused) == I and call(x=y + 640, ldx=1536, **fused) == I


def before(t=None, ids=P, T=8, d=256, x=2 * P, ldx=256, norm="rms", h=3 * P, ldh=256):
    t = t or table()
    if norm == "rms":
        norm = L.make_norm(L.LORA_NORM_RMS, 1e-5, gain=6 * P)
    return code(L.lora_norm_before, ctypes.addressof(t), ids, T, d, x, ldx, norm, h, ldh, 0)


def test_norm_before_arguments():
    I, U = L.LORA_ERR_INVALID_ARG, L.LORA_ERR_UNSUPPORTED
    N = L.make_norm
    assert before() == OK and before(ids=None) == OK and before(T=0) == L.LORA_OK
    assert before(t=table(dtype=L.LORA_F32), d=4, ldx=4, ldh=4) == OK
    assert before(T=-1) == I and before(d=0) == I and before(norm=None) == I
    assert before(d=252) == U and before(d=16392, ldx=16392, ldh=16392) == U
    assert before(d=16384, ldx=16384, ldh=16384) == OK
    assert before(x=None) == I and before(h=None) == I and before(ldx=248) == I and before(ldh=248) == I
    assert before(x=2 * P + 2) == U and before(h=3 * P + 8) == U and before(ldx=260) == U and before(ldh=260) == U
    assert before(norm=N(0, 1e-5)) == I and before(norm=N(3, 1e-5)) == I
    for eps in (-1e-5, float("nan"), float("inf")):
        assert before(norm=N(L.LORA_NORM_RMS, eps)) == I
    assert before(norm=N(L.LORA_NORM_LAYER, 0.0)) == OK
    assert before(norm=N(L.LORA_NORM_RMS, 1e-5, gain=6 * P, ld=248)) == I
    assert before(norm=N(L.LORA_NORM_RMS, 1e-5, gain=6 * P, ld=260)) == U
    assert before(norm=N(L.LORA_NORM_RMS, 1e-5, shift=6 * P + 2)) == U
    assert before(norm=N(L.LORA_NORM_RMS, 1e-5, gain=6 * P, shift=7 * P, ld=264)) == OK
    assert before(h=2 * P) == OK                                # in place
    assert before(h=2 * P + 16) == I and before(h=2 * P, ldh=512) == I
    assert before(x=2 * P, ldx=512, h=2 * P + 512, ldh=512) == OK   # two halves of one buffer


def after(t=None, ids=P, T=8, d=256, z=2 * P, ldz=256, norm="rms", res="res", r=3 * P, ldr=256, nxt="rms", h=4 * P,
          ldh=256):
    t = t or table()
    if norm == "rms":
        norm = L.make_norm(L.LORA_NORM_RMS, 1e-5, gain=6 * P)
    if nxt == "rms":
        nxt = L.make_norm(L.LORA_NORM_RMS, 1e-5, gain=6 * P)
    if res == "res":
        res = L.make_residual(residual=5 * P, ldres=256)
    return code(L.lora_norm_after, ctypes.addressof(t), ids, T, d, z, ldz, norm, res, r, ldr, nxt, h, ldh, 0)


def test_norm_after_arguments():
    I, U = L.LORA_ERR_INVALID_ARG, L.LORA_ERR_UNSUPPORTED
    R = L.make_residual
    assert after() == OK and after(norm=None) == OK and after(r=None) == OK and after(nxt=None, h=None) == OK
    assert after(res=None) == I and after(nxt=None) == I and after(h=None) == I and after(nxt=None, h=None, r=None) == I
    assert after(res=R()) == OK
    assert after(res=R(residual=5 * P, ldres=248)) == I and after(res=R(residual=5 * P + 2, ldres=256)) == U
    A, T = L.LORA_GATE_ADAPTER, L.LORA_GATE_TOKEN
    assert after(res=R(gate_kind=A)) == I and after(res=R(gate_kind=3, gate=7 * P)) == I
    assert after(res=R(gate_kind=A, gate=7 * P)) == OK and after(res=R(gate_kind=T, gate=7 * P)) == I
    assert after(res=R(gate_kind=T, gate=7 * P, ldgate=256)) == OK
    assert after(res=R(gate_kind=A, gate=7 * P, ldgate=248)) == I
    assert after(res=R(gate_kind=A, gate=7 * P + 2, ldgate=256)) == U
    # r and h in place of an input, but not of each other
    assert after(r=2 * P) == OK and after(r=5 * P) == OK and after(h=2 * P) == OK and after(r=5 * P, h=2 * P) == OK
    assert after(r=4 * P) == I and after(r=2 * P + 16) == I and after(h=5 * P + 512) == I
    assert after(res=R(gate_kind=T, gate=3 * P, ldgate=256)) == OK
    assert after(res=R(gate_kind=T, gate=3 * P + 16, ldgate=256)) == I


def test_null_tables():
    assert code(L.lora_bgmv_layer, None, P, 1, P, 8, P, 8, None, P, 8, 0, P, 0, 0) == L.LORA_ERR_INVALID_ARG
    assert code(L.lora_sgmv_layer, None, L.lora_segments(), P, 8, P, 8, None, P, 8, 0, P, 0, 0) == \
        L.LORA_ERR_INVALID_ARG
    n = L.make_norm(L.LORA_NORM_RMS, 0.0)
    assert code(L.lora_norm_before, None, P, 1, 8, P, 8, n, P, 8, 0) == L.LORA_ERR_INVALID_ARG
    assert code(L.lora_norm_after, None, P, 1, 8, P, 8, n, L.make_residual(), P, 8, None, None, 0, 0) == \
        L.LORA_ERR_INVALID_ARG
