"""The calls of tests/mx_kernels.py run the kernels they name, and together
every kernel of the 4-bit products; layouts that the fast kernels cannot take
go to the others: the rules are the library's, compiled for the host."""
import shutil

import pytest

from mx_kernels import PRODUCTS, VARIANTS, P, Chooser

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ needed")


@pytest.fixture(scope="module")
def chooser(tmp_path_factory):
    return Chooser(str(tmp_path_factory.mktemp("choice")))


@pytest.mark.parametrize("name", list(PRODUCTS))
def test_a_product_runs_the_kernel_it_names(chooser, name):
    c = PRODUCTS[name]
    for K in c["K"]:
        for out in ("f16", "bf16", "f32"):
            assert chooser.product(c["counts"], K, c["N"], out) == c["kernel"]


def test_every_kernel_is_run_by_a_call(chooser):
    got = {c["kernel"] for c in PRODUCTS.values()} | {chooser.product([40], 90, 70)}
    assert got == set(VARIANTS)
    slices = {-(-K // 256) % 4 for c in PRODUCTS.values() if c["kernel"] == "large" for K in c["K"]}
    assert slices == {0, 1, 2, 3}


@pytest.mark.parametrize("K,N,lda", [(90, 64, None),    # rows of codes in pieces
                                     (96, 64, 49)])     # on 16-byte boundaries
def test_products_of_other_layouts(chooser, K, N, lda):
    assert chooser.product([40], K, N, lda=lda) == "any layout"


@pytest.mark.parametrize("name", list(PRODUCTS))
def test_outputs_off_boundaries_run_the_same_kernels(chooser, name):
    c = PRODUCTS[name]
    want = "128 x 128" if c["kernel"] == "large" else c["kernel"]
    for K in c["K"]:
        assert chooser.product(c["counts"], K, c["N"] - 3) == want
        assert chooser.product(c["counts"], K, c["N"], ldc=c["N"] + 3) == want


@pytest.mark.parametrize("name", list(PRODUCTS))
def test_scales_off_dwords_run_the_same_kernels(chooser, name):
    c = PRODUCTS[name]
    for K in c["K"]:
        assert chooser.product(c["counts"], K, c["N"], lds=-(-K // 32) | 1) == c["kernel"] + ", shifted"


def test_one_row_of_scales_has_no_stride(chooser):
    """Five scales, as the binding gives a single row's stride."""
    for at, lda, ldb, want in ((P, 5, 8, "16 rows"), (P + 1, 8, 8, "16 rows, shifted"), (P, 8, 5, "16 rows, shifted")):
        v = chooser.call("ag_gemm_mxfp4", P, 80, at, lda, P, 80, P, ldb, P, 64, 2, 1, 160, 64, None)
        assert VARIANTS[v % 16] + ", shifted" * (v >= 16) == want
    v = chooser.call("ag_gemm_mxfp4", P, 80, P, 8, P, 80, P, 5, P, 16, 2, 8, 160, 1, None)
    assert VARIANTS[v % 16] == "16 rows"


def test_rows_on_boundaries_are_moved_whole(chooser):
    """16 bytes at a time where every row starts on such a boundary."""
    c = chooser.call
    for at, ld, k, unit in ((P, 64, 64, 16), (P + 2, 64, 64, 2), (P, 63, 62, 2), (P, 68, 64, 2), (P, 72, 60, 2)):
        assert c("ag_gemm_expert_dispatch", 2, at, ld, P, 2, P, 64, 32, 16, k, None) == unit
        wide = unit == 16
        assert c("ag_gemm_expert_combine", 2, at, ld, 32, P, 2, P, 2, P, 64, 2, 16, k, None) == wide
        assert c("ag_gemm_expert_combine", 2, P, 64, 32, P, 2, P, 2, at, ld, 2, 16, k, None) == wide
        assert c("ag_gemm_expert_combine_grad", 2, at, ld, P, 64, 32, P, 2, P, 2, P, 64, P, 2, 16, k, None) == wide
        assert c("ag_gemm_expert_combine_grad", 2, P, 64, at, ld, 32, P, 2, P, 2, P, 64, P, 2, 16, k, None) == wide
        assert c("ag_gemm_expert_combine_grad", 2, P, 64, P, 64, 32, P, 2, P, 2, at, ld, P, 2, 16, k, None) == wide
        for i in range(4):       # x, residual, h, y
            ptrs, lds = [P + 4096 * j for j in range(4)], [64] * 4
            ptrs[i], lds[i] = ptrs[i] + at - P, ld
            (x, res, h, y), (ldx, ldr, ldh, ldy) = ptrs, lds
            assert c("ag_gemm_rmsnorm", 2, x, ldx, res, ldr, P, h, ldh, y, ldy, None, 0, None, 0, P, 1e-6, 16, k,
                     None) == wide
        assert c("ag_gemm_rmsnorm_grad", 2, at, ld, P, 64, P, P, P, 64, P, 64, P, 2, P, 1 << 20, 16, k, None) == wide
        assert c("ag_gemm_rmsnorm_grad", 2, P, 64, P, 64, P, P, at, ld, P, 64, P, 2, P, 1 << 20, 16, k, None) == wide
        assert c("ag_gemm_quant_mxfp4", 2, at, ld, P, 32, P, 2, 16, k, None) == wide
        assert c("ag_gemm_dequant_mxfp4", P, 32, P, 2, at, ld, 2, 16, k, None) == wide
    assert c("ag_gemm_rmsnorm", 2, P, 64, None, 0, P + 2, None, 0, P, 64, None, 0, None, 0, P, 1e-6, 16, 64, None) == 0
    assert c("ag_gemm_quant_mxfp4", 2, P, 64, P + 1, 32, P, 2, 16, 64, None) == 0
    assert c("ag_gemm_expert_dispatch", 3, P, 64, P, 2, P, 64, 32, 16, 64, None) == 16
    assert c("ag_gemm_expert_dispatch", 3, P + 1, 64, P, 2, P, 64, 32, 16, 64, None) == 1
    assert c("ag_gemm_expert_dispatch", 4, P + 4, 64, P, 2, P, 64, 32, 16, 64, None) == 4
