"""The expert products' Python side where no GPU is needed: row strides,
gradients that do not exist, rows of no group, and the stream of prepared
calls."""
import pytest
import torch

from communication_gemm_amd import _native


# The last token of one sequence is a row of [tokens * width] elements' stride.
@pytest.mark.parametrize("n,step", [(64, 3 * 64), (4096, 4096 * 4096), (128, 129)])
def test_one_row_has_no_row_stride(n, step):
    row = torch.empty(n, dtype=torch.float16).as_strided((1, n), (step, 1))
    assert _native._matrix(row, 1, n, -1, "x") == n
    stack = torch.empty(2 * n, dtype=torch.float16).as_strided((2, 1, n), (n, step, 1))
    assert _native._matrices(stack, 2, 1, n, -1, "w") == (n, n)


def test_more_rows_keep_their_stride():
    t = torch.empty(6, 40)[:, :33]
    assert _native._matrix(t, 6, 33, -1, "x") == 40
    s = torch.empty(3, 6, 40)[:, :, :33]
    assert _native._matrices(s, 3, 6, 33, -1, "w") == (40, 240)
