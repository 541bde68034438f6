"""Refusals of the operators around the expert products: every wrong argument
is an error before any kernel is launched (no GPU needed, host memory stands
for the matrices and is never read)."""
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

SORT = dict(ids=P, size=8, ldi=2, T=16, top=2, experts=8, off=P, place=P, ws=None, wsb=0, st=None)
DISPATCH = dict(type=BF16, x=P, ldx=64, place=P, top=2, xs=P, ldxs=64, rows=32, T=16, K=64, st=None)
COMBINE = dict(type=BF16, h=P, ldh=64, rows=32, place=P, top=2, w=P, ldw=2, y=P, ldy=64, out=BF16,
               T=16, K=64, st=None)
CGRAD = dict(type=BF16, dy=P, lddy=64, h=P, ldh=64, rows=32, place=P, top=2, w=P, ldw=2, dh=P,
             lddh=64, dw=P, lddw=2, T=16, K=64, st=None)
NORM = dict(type=BF16, x=P, ldx=256, res=P, ldr=256, w=P, h=P, ldh=256, y=P, ldy=256, q=P, ldq=256,
            scale=P, lds=2, rstd=P, eps=1e-6, T=16, K=256, st=None)
NGRAD = dict(type=BF16, dy=P, lddy=256, h=P, ldh=256, w=P, rstd=P, dh=P, lddh=256, dx=P, lddx=256,
             dw=P, dwt=F32, ws=P, wsb=1 << 20, T=16, K=256, st=None)
MXQ = dict(type=BF16, x=P, ldx=256, q=P, ldq=128, s=P, lds=8, M=16, K=256, st=None)
MXD = dict(q=P, ldq=128, s=P, lds=8, y=P, ldy=256, type=BF16, M=16, K=256, st=None)
MX = dict(a=P, lda=128, sa=P, ldas=8, b=P, ldb=128, sb=P, ldbs=8, c=P, ldc=32, out=BF16, M=16, K=256,
          N=32, st=None)
GMX = dict(a=P, lda=128, sa=P, ldas=8, b=P, ldb=128, bst=128 * 32, sb=P, ldbs=8, bsst=256, off=P,
           groups=4, c=P, ldc=32, out=BF16, T=16, K=256, N=32, st=None)

TABLE = (
    ("ag_gemm_expert_sort", SORT, [
        (dict(ids=None), INVALID), (dict(size=2), INVALID), (dict(ldi=1), INVALID), (dict(T=-1), INVALID),
        (dict(top=0), INVALID), (dict(experts=0), INVALID), (dict(off=None), INVALID),
        (dict(place=None), INVALID), (dict(T=20000), INVALID), (dict(T=20000, ws=P, wsb=4), INVALID),
        (dict(T=20000, ws=P + 2, wsb=1 << 20), UNSUPPORTED), (dict(ids=P + 4), UNSUPPORTED),
        (dict(place=P + 1), UNSUPPORTED), (dict(off=P + 2), UNSUPPORTED),
        (dict(experts=4097), UNSUPPORTED), (dict(top=1025, ldi=1025), UNSUPPORTED),
        (dict(T=2 ** 30), UNSUPPORTED), (dict(T=2 ** 62), UNSUPPORTED)]),
    ("ag_gemm_expert_dispatch", DISPATCH, [
        (dict(type=1), INVALID), (dict(x=None), INVALID), (dict(place=None), INVALID),
        (dict(xs=None), INVALID), (dict(ldx=63), INVALID), (dict(ldxs=63), INVALID),
        (dict(rows=-1), INVALID), (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(top=0), INVALID),
        (dict(x=P + 1), UNSUPPORTED), (dict(place=P + 2), UNSUPPORTED), (dict(top=1025), UNSUPPORTED),
        (dict(T=2 ** 30), UNSUPPORTED), (dict(rows=2 ** 31), UNSUPPORTED),
        (dict(K=2 ** 20 + 1, ldx=2 ** 21, ldxs=2 ** 21), UNSUPPORTED), (dict(ldx=2 ** 21 + 1), UNSUPPORTED)]),
    ("ag_gemm_expert_combine", COMBINE, [
        (dict(type=FP8), INVALID), (dict(out=F16), INVALID), (dict(h=None), INVALID),
        (dict(place=None), INVALID), (dict(y=None), INVALID), (dict(ldw=1), INVALID),
        (dict(ldh=63), INVALID), (dict(ldy=63), INVALID), (dict(type=F32, out=BF16), INVALID),
        (dict(w=P + 2), UNSUPPORTED), (dict(out=F32, y=P + 2), UNSUPPORTED), (dict(h=P + 1), UNSUPPORTED)]),
    ("ag_gemm_expert_combine_grad", CGRAD, [
        (dict(type=FP8), INVALID), (dict(dy=None), INVALID), (dict(h=None), INVALID),
        (dict(w=None), INVALID), (dict(dh=None, dw=None), INVALID), (dict(place=None), INVALID),
        (dict(lddh=63), INVALID), (dict(lddw=1), INVALID), (dict(dw=P + 2), UNSUPPORTED),
        (dict(dh=P + 1), UNSUPPORTED)]),
    ("ag_gemm_rmsnorm", NORM, [
        (dict(type=FP8), INVALID), (dict(x=None), INVALID), (dict(y=None, q=None, scale=None), INVALID),
        (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(eps=-1.0), INVALID),
        (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(ldx=255), INVALID),
        (dict(ldr=255), INVALID), (dict(ldh=255), INVALID), (dict(ldy=255), INVALID),
        (dict(ldq=255), INVALID), (dict(lds=1), INVALID), (dict(T=-1), INVALID), (dict(K=0), INVALID),
        (dict(x=P + 256, h=P + 256, ldh=264), INVALID), (dict(x=P + 1), UNSUPPORTED),
        (dict(w=P + 1), UNSUPPORTED), (dict(rstd=P + 2), UNSUPPORTED), (dict(scale=P + 2), UNSUPPORTED)]),
    ("ag_gemm_rmsnorm_grad", NGRAD, [
        (dict(type=FP8), INVALID), (dict(dwt=F16), INVALID), (dict(dy=None), INVALID),
        (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID),
        (dict(ws=None), INVALID), (dict(wsb=16 * 256 * 4 - 1), INVALID), (dict(lddx=255), INVALID),
        (dict(lddh=255), INVALID), (dict(ws=P + 4), UNSUPPORTED), (dict(dw=P + 2), UNSUPPORTED)]),
    ("ag_gemm_quant_mxfp4", MXQ, [
        (dict(type=FP8), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
        (dict(K=255), INVALID), (dict(ldq=127), INVALID), (dict(lds=7), INVALID), (dict(M=-1), INVALID),
        (dict(x=P + 1), UNSUPPORTED)]),
    ("ag_gemm_dequant_mxfp4", MXD, [
        (dict(type=FP8), INVALID), (dict(y=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
        (dict(K=255), INVALID), (dict(ldy=255), INVALID), (dict(type=F32, y=P + 2), UNSUPPORTED)]),
    ("ag_gemm_mxfp4", MX, [
        (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID), (dict(sb=None), INVALID),
        (dict(c=None), INVALID), (dict(out=FP8), INVALID), (dict(K=255), INVALID), (dict(lda=127), INVALID),
        (dict(ldbs=7), INVALID), (dict(ldc=31), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
        (dict(c=P + 1), UNSUPPORTED), (dict(M=2 ** 31 - 1), UNSUPPORTED)]),
    ("ag_gemm_grouped_mxfp4", GMX, [
        (dict(off=None), INVALID), (dict(bst=-1), INVALID), (dict(bsst=-1), INVALID),
        (dict(groups=0), INVALID), (dict(off=P + 1), UNSUPPORTED), (dict(groups=65537), UNSUPPORTED)]))


@pytest.mark.parametrize("fn,good,changes,status",
                         [(fn, good, ch, st) for fn, good, table in TABLE for ch, st in table])
def test_refused(fn, good, changes, status):
    assert getattr(lib, fn)(*{**good, **changes}.values()) == status


def test_no_rows_is_no_work():
    for fn, good, null in (("ag_gemm_expert_dispatch", DISPATCH, ("x", "place")),
                           ("ag_gemm_expert_combine", COMBINE, ("place", "w", "y")),
                           ("ag_gemm_expert_combine_grad", CGRAD, ("dy", "place", "w", "dw")),
                           ("ag_gemm_rmsnorm", NORM, ("x", "res", "h", "y", "q", "scale", "rstd")),
                           ("ag_gemm_grouped_mxfp4", GMX, ("a", "sa", "c"))):
        assert getattr(lib, fn)(*{**good, **{k: None for k in null}, "T": 0}.values()) == 0, fn
    assert lib.ag_gemm_rmsnorm_grad(*{**NGRAD, "T": 0, "dy": None, "dw": None}.values()) == 0
    for fn, good in (("ag_gemm_quant_mxfp4", MXQ), ("ag_gemm_dequant_mxfp4", MXD), ("ag_gemm_mxfp4", MX)):
        assert getattr(lib, fn)(*{**good, "M": 0}.values()) == 0, fn


def test_workspaces():
    """By the rules in the header: none up to 8192 assignments, counts of at
    most 256 chunks after that; a float32 row for each of at most 512 parts."""
    assert agg.expert_sort_workspace_bytes(4096, 2, 64) == 0
    assert agg.expert_sort_workspace_bytes(4097, 2, 64) == 9 * 64 * 4
    assert agg.expert_sort_workspace_bytes(1 << 20, 8, 64) == 256 * 64 * 4
    assert agg.expert_sort_workspace_bytes(1 << 40, 8, 64) == 0
    assert agg.expert_sort_workspace_bytes(1 << 20, 8, 4097) == 0
    assert agg.rmsnorm_grad_workspace_bytes(3, 100) == 3 * 100 * 4
    assert agg.rmsnorm_grad_workspace_bytes(100000, 100) == 512 * 100 * 4
    assert agg.rmsnorm_grad_workspace_bytes(0, 100) == 0


def test_binding_refuses_wrong_tensors():
    """The checks that need no device: types, shapes, tensors on the host."""
    x, ids = torch.empty(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    xs, w = torch.empty(8, 64, dtype=torch.bfloat16), torch.empty(4, 2)
    off, place = torch.zeros(9, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    q, s = torch.empty(4, 32, dtype=torch.uint8), torch.empty(4, 2, dtype=torch.uint8)
    for call in (lambda: agg.ag_gemm_expert_sort(ids.short(), 8, off, place),
                 lambda: agg.ag_gemm_expert_sort(ids.flatten(), 8, off, place),
                 lambda: agg.ag_gemm_expert_sort(ids, 8, off, place),            # on the host
                 lambda: agg.ag_gemm_expert_dispatch(x, place, xs.float()),
                 lambda: agg.ag_gemm_expert_dispatch(x.double(), place, xs),
                 lambda: agg.ag_gemm_expert_dispatch(x, place, xs),
                 lambda: agg.ag_gemm_expert_combine(xs, place, w.double(), x),
                 lambda: agg.ag_gemm_expert_combine(xs, place, w, x.half()),
                 lambda: agg.ag_gemm_expert_combine_grad(x, xs, place, w),
                 lambda: agg.ag_gemm_expert_combine_grad(x, xs, place, w, xs.float()),
                 lambda: agg.ag_gemm_rmsnorm(x),
                 lambda: agg.ag_gemm_rmsnorm(x, q=x.to(torch.float8_e4m3fn)),
                 lambda: agg.ag_gemm_rmsnorm(x, torch.ones(64), x),
                 lambda: agg.ag_gemm_rmsnorm(x, None, x),
                 lambda: agg.ag_gemm_rmsnorm_grad(x, x.float(), None, torch.ones(4), x),
                 lambda: agg.ag_gemm_quant_mxfp4(x[:, :63], q, s),
                 lambda: agg.ag_gemm_quant_mxfp4(x, q.short(), s),
                 lambda: agg.ag_gemm_quant_mxfp4(x, q, s),
                 lambda: agg.ag_gemm_dequant_mxfp4(q, s.float(), x),
                 lambda: agg.ag_gemm_mxfp4(q, s, q[None], s, x),
                 lambda: agg.ag_gemm_grouped_mxfp4(q, s, q, s, off, x),
                 lambda: agg.ag_gemm_mxfp4(q, s, q, s, torch.empty(4, 4))):
        with pytest.raises(ValueError):
            call()
