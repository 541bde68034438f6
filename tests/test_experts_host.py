"""Refusals of the expert products: every wrong argument is an error before
any kernel is launched (no GPU needed, host memory stands for the matrices
and is never read)."""
import ctypes

import pytest
import torch

import communication_gemm_amd as agg
from communication_gemm_amd import _native

lib = _native.lib
BUF = (ctypes.c_char * 4096)()
P = (ctypes.addressof(BUF) + 255) // 256 * 256
BF16, FP8, F32, F16 = agg.TYPE_BF16, agg.TYPE_FP8, agg.TYPE_F32, agg.TYPE_F16
INVALID, UNSUPPORTED = agg.AGG_E_INVALID, agg.AGG_E_UNSUPPORTED

GROUPED = dict(type=BF16, x=P, ldx=64, w=P, ldw=32, ws=64 * 32, trans=0, off=P, groups=4, y=P,
               ldy=32, out=BF16, T=16, K=64, N=32, st=None)
WGRAD = dict(type=BF16, x=P, ldx=64, dy=P, lddy=32, off=P, groups=4, dw=P, lddw=32, dws=64 * 32,
             out=F32, T=16, K=64, N=32, st=None)
DENSE = dict(a=P, lda=256, sa=P, ldas=2, b=P, ldb=256, sb=P, ldbs=2, c=P, ldc=32, out=BF16, M=16,
             K=256, N=32, st=None)
GFP8 = dict(a=P, lda=256, sa=P, ldas=2, b=P, ldb=256, bst=256 * 32, sb=P, ldbs=2, bsst=2, off=P,
            groups=4, c=P, ldc=32, out=BF16, T=16, K=256, N=32, st=None)
QUANT = dict(type=BF16, x=P, ldx=256, q=P, ldq=256, s=P, lds=2, br=1, M=16, K=256, st=None)


@pytest.mark.parametrize("fn,good,changes,status", [
    (fn, good, ch, status)
    for fn, good, table in (
        ("ag_gemm_grouped", GROUPED, [
            (dict(type=F32), INVALID), (dict(type=FP8), INVALID), (dict(type=1), INVALID),
            (dict(out=F16), INVALID), (dict(out=9), INVALID), (dict(x=None), INVALID),
            (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(off=None), INVALID),
            (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID),
            (dict(groups=0), INVALID), (dict(ldx=63), INVALID), (dict(ldw=31), INVALID),
            (dict(trans=1, ldw=63), INVALID), (dict(ldy=31), INVALID), (dict(ws=-1), INVALID),
            (dict(x=P + 1), UNSUPPORTED), (dict(w=P + 1), UNSUPPORTED),
            (dict(y=P + 2, out=F32), UNSUPPORTED), (dict(off=P + 2), UNSUPPORTED),
            (dict(T=2 ** 31 - 1), UNSUPPORTED), (dict(K=2 ** 20 + 1, ldx=2 ** 21), UNSUPPORTED),
            (dict(N=2 ** 20 + 1, ldw=2 ** 21, ldy=2 ** 21), UNSUPPORTED),
            (dict(ldx=2 ** 21 + 1), UNSUPPORTED), (dict(groups=65537), UNSUPPORTED)]),
        ("ag_gemm_grouped_wgrad", WGRAD, [
            (dict(type=FP8), INVALID), (dict(out=F16), INVALID), (dict(x=None), INVALID),
            (dict(dy=None), INVALID), (dict(dw=None), INVALID), (dict(off=None), INVALID),
            (dict(lddy=31), INVALID), (dict(lddw=31), INVALID), (dict(dws=64 * 32 - 1), INVALID),
            (dict(dw=P + 2), UNSUPPORTED), (dict(dy=P + 1), UNSUPPORTED)]),
        ("ag_gemm_fp8_block", DENSE, [
            (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID),
            (dict(sb=None), INVALID), (dict(c=None), INVALID), (dict(out=FP8), INVALID),
            (dict(ldas=1), INVALID), (dict(ldbs=1), INVALID), (dict(lda=255), INVALID),
            (dict(M=-1), INVALID), (dict(sa=P + 2), UNSUPPORTED), (dict(c=P + 1), UNSUPPORTED)]),
        ("ag_gemm_grouped_fp8_block", GFP8, [
            (dict(off=None), INVALID), (dict(bst=-1), INVALID), (dict(bsst=-1), INVALID),
            (dict(groups=-3), INVALID), (dict(off=P + 1), UNSUPPORTED)]),
        ("ag_gemm_quant_fp8_block", QUANT, [
            (dict(type=FP8), INVALID), (dict(br=64), INVALID), (dict(x=None), INVALID),
            (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(lds=1), INVALID),
            (dict(ldq=255), INVALID), (dict(K=0), INVALID), (dict(type=F32, x=P + 2), UNSUPPORTED)]))
    for ch, status in table])
def test_refused(fn, good, changes, status):
    assert getattr(lib, fn)(*{**good, **changes}.values()) == status


@pytest.mark.parametrize("fn,good", [("ag_gemm_grouped", GROUPED), ("ag_gemm_grouped_fp8_block", GFP8)])
def test_no_rows_is_no_work(fn, good):
    null = {k: None for k in ("x", "y", "a", "sa", "c") if k in good}
    assert getattr(lib, fn)(*{**good, **null, "T": 0}.values()) == 0
    assert lib.ag_gemm_fp8_block(*{**DENSE, "M": 0}.values()) == 0
    assert lib.ag_gemm_quant_fp8_block(*{**QUANT, "M": 0}.values()) == 0


def test_binding_refuses_wrong_tensors():
    """The checks that need no device: types and shapes."""
    x, w = torch.empty(4, 8, dtype=torch.bfloat16), torch.empty(2, 8, 16, dtype=torch.bfloat16)
    y, off = torch.empty(4, 16, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        agg.ag_gemm_grouped(x.float(), w, off, y)
    with pytest.raises(ValueError):
        agg.ag_gemm_grouped(x, w.half(), off, y)
    with pytest.raises(ValueError):
        agg.ag_gemm_grouped(x, w, off, y.half())
    with pytest.raises(ValueError):
        agg.ag_gemm_grouped(x, w, off, y)          # on the host
    with pytest.raises(ValueError):
        agg.ag_gemm_grouped_wgrad(x, x, off, y)
    with pytest.raises(ValueError):
        agg.ag_gemm_quant_fp8_block(x, x, torch.empty(4, 1))
    with pytest.raises(ValueError):
        agg.ag_gemm_quant_fp8_block(x, x.to(torch.float8_e4m3fn), torch.empty(4, 1), 64)
