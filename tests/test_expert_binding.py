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


# ---- gradients that do not exist ---------------------------------------------

@pytest.fixture
def experts(monkeypatch):
    """The layer functions with products that only fill their outputs."""
    from communication_gemm_amd import experts as m

    def fill(*out):
        for t in out:
            t.view(torch.uint8).fill_(0x38)      # 1 in E4M3
        return out

    monkeypatch.setattr(m.agg, "ag_gemm_quant_fp8_block", lambda x, q, s, rows: fill(q, s))
    monkeypatch.setattr(m.agg, "ag_gemm_grouped_fp8_block", lambda a, sa, b, sb, off, y: fill(y)[0])
    return m


def fp8_weights():
    return torch.zeros(2, 16, 8, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(2, 1, 1)


OFFSETS = torch.tensor([0, 2, 4], dtype=torch.int32)


def test_a_gradient_through_the_fp8_product_is_refused(experts):
    """It would be missing without a word: the rest of the loss has one."""
    x = torch.ones(4, 8, requires_grad=True)
    y = experts.grouped_linear_fp8(x, *fp8_weights(), OFFSETS)
    with pytest.raises(RuntimeError, match="no gradient"):
        (y.sum() + x.sum()).backward()


@pytest.mark.parametrize("shape", [(4, 8), (2, 4, 8)])
def test_a_gradient_through_the_quantisers_is_refused(experts, shape):
    x = torch.ones(shape, requires_grad=True)
    for quantise in [experts.quantize_weights] + [experts.quantize] * (len(shape) == 2):
        q, scale = quantise(x)
        for part in (q.float().sum(), scale.sum()):
            with pytest.raises(RuntimeError, match="no gradient"):
                (part + x.sum()).backward(retain_graph=True)


def test_serving_calls_record_nothing(experts):
    x, plain = torch.ones(4, 8, requires_grad=True), torch.ones(4, 8)
    with torch.no_grad():
        got = [experts.grouped_linear_fp8(x, *fp8_weights(), OFFSETS), *experts.quantize(x),
               *experts.quantize_weights(x)]
    for t in (plain, x.detach()):
        got += [experts.grouped_linear_fp8(t, *fp8_weights(), OFFSETS), *experts.quantize(t)]
    assert not any(t.requires_grad for t in got)


def test_rows_of_no_group_are_zeros_where_padded(experts, monkeypatch):
    """The product writes rows of groups only."""
    monkeypatch.setattr(experts.agg, "ag_gemm_grouped_fp8_block",
                        lambda a, sa, b, sb, off, y: y[int(off[0]):int(off[-1])].fill_(5) is None or y)
    off = torch.tensor([1, 2, 3], dtype=torch.int32)
    y = experts.grouped_linear_fp8(torch.ones(4, 8), *fp8_weights(), off, padded=True)
    assert y[:, 0].tolist() == [0, 5, 5, 0]


# ---- the stream of prepared calls ---------------------------------------------

def test_a_prepared_call_follows_the_current_stream(monkeypatch):
    """Unless it was prepared for a stream of its own."""
    now, seen = [11], []
    monkeypatch.setattr(_native, "_raw_stream", lambda dev: now[0])

    def fn(*args):
        seen.append(args)
        return 0

    free = _native._call(fn, (1, 2), None, 0, "fn", None, True)
    fixed = _native._call(fn, (1, 2), 77, 0, "fn", None, True)
    assert not seen
    for now[0] in (11, 12):
        free()
        fixed()
    at = [a[-1] if isinstance(a[-1], int) else a[-1].value for a in seen]
    assert at == [11, 77, 12, 77] and all(a[:2] == (1, 2) for a in seen)
    assert _native._call(fn, (1, 2), None, 0, "fn", "out", False) == "out" and seen[-1] == (1, 2, 12)
    for call in (_native._call(lambda *a: 2, (), None, 0, "fn", None, True),
                 _native._call(lambda *a: 2, (), 77, 0, "fn", None, True)):
        with pytest.raises(_native.AggError):
            call()
