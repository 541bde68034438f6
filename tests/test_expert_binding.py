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


# ---- what the layer functions make of their inputs ------------------------------

def test_scales_are_float32_whatever_the_default_type(experts, monkeypatch):
    """Models built for serving set torch's default type; the library takes
    float32 scales."""
    made = {}
    monkeypatch.setattr(experts.agg, "ag_gemm_rmsnorm", lambda *a, **kw: made.update(kw))
    x = torch.ones(4, 8, dtype=torch.bfloat16)
    torch.set_default_dtype(torch.bfloat16)
    try:
        got = [experts.quantize(x)[1], experts.quantize_weights(x)[1], experts.quantize_weights(x[None])[1],
               experts.rms_norm_fp8(x)[1]]
    finally:
        torch.set_default_dtype(torch.float32)
    assert [t.dtype for t in got + [made["scale"]]] == [torch.float32] * 5


def test_a_gradient_through_codes_and_scales_is_refused(experts):
    """As through the product that quantises its rows itself; so is one of the
    weights' codes and scales."""
    rows, w = torch.ones(4, 8, requires_grad=True), torch.ones(2, 16, 8, requires_grad=True)
    with torch.no_grad():
        plain, wq = experts.quantize(rows), experts.quantize_weights(w)
    for pair, weights in ((experts.quantize(rows), wq), (plain, experts.quantize_weights(w)),
                          ((plain[0], experts.quantize(rows)[1]), wq)):
        y = experts.grouped_linear_fp8(pair, *weights, OFFSETS, torch.float32)
        with pytest.raises(RuntimeError, match="no gradient"):
            (y.sum() + rows.sum() + w.sum()).backward()
    assert not experts.grouped_linear_fp8(plain, *wq, OFFSETS, torch.float32).requires_grad
    with pytest.raises(ValueError, match="out_dtype"):
        experts.grouped_linear_fp8(plain, *wq, OFFSETS)


def test_a_gradient_through_4_bit_codes_is_refused(experts, monkeypatch):
    """Codes and scales are integers, which autograd does not follow: the call
    itself is the last place that sees it."""
    monkeypatch.setattr(experts.agg, "ag_gemm_quant_mxfp4", lambda x, q, s: (q.fill_(0), s.fill_(127)))
    x = torch.ones(4, 32, requires_grad=True)
    for t in (x, x.view(2, 2, 32) * 2):
        with pytest.raises(RuntimeError, match="no gradient"):
            experts.quantize_mxfp4(t)
        with torch.no_grad():
            assert experts.quantize_mxfp4(t)[0].shape == (*t.shape[:-1], 16)
        assert experts.quantize_mxfp4(t.detach())[1].shape == (*t.shape[:-1], 1)


def test_rows_of_any_strides_are_taken(experts, monkeypatch):
    """Transposed, expanded and narrowed rows reach the library as matrices with unit
    column stride, weights of a norm as contiguous ones; others as they are."""
    def check(*names):
        def call(*args, **kw):
            for t in (*args, *kw.values()):
                if isinstance(t, torch.Tensor) and t.dim() == 2:
                    assert t.stride(1) == 1 and t.stride(0) >= t.shape[1]
                assert not isinstance(t, torch.Tensor) or t.dim() != 1 or t.is_contiguous()
            kept.extend(t.data_ptr() for t in args if isinstance(t, torch.Tensor))
            return args[names[0]] if len(names) == 1 else tuple(args[n] for n in names)
        return call

    kept = []
    for name, out in (("ag_gemm_expert_dispatch", (2,)), ("ag_gemm_expert_combine", (3,)),
                      ("ag_gemm_rmsnorm", (0,)), ("ag_gemm_grouped", (3,)), ("ag_gemm_quant_fp8_block", (1, 2))):
        monkeypatch.setattr(experts.agg, name, check(*out))
    place = torch.zeros(4, 2, dtype=torch.int32)
    r, vector = experts.Routing(OFFSETS, place), torch.ones(2, 8)[:, 0]
    for x in (torch.ones(8, 4).t(), torch.ones(8).expand(4, 8), torch.ones(4, 24)[:, ::3]):
        h = x.repeat(2, 1).t().contiguous().t()
        assert experts.dispatch(x, r).shape == (8, 8)
        assert experts.combine(h, torch.ones(2, 4).t(), r).shape == (4, 8)
        experts.rms_norm(x[:, :2], vector, x[:, :2])
        experts.rms_norm_fp8(x[:, :2], vector, x[:, :2], with_y=True)
        experts.quantize(x)
        experts.quantize_weights(x)
        experts.quantize_weights(x[None])
        experts.grouped_linear(x, torch.ones(2, 8, 16), OFFSETS)
        experts.grouped_linear_fp8(x, *fp8_weights(), OFFSETS)
    kept.clear()
    x = torch.ones(4, 40)[:, :8]                 # a wider matrix's rows are not copied
    experts.dispatch(x, r)
    experts.quantize(x)
    experts.grouped_linear(x, torch.ones(2, 8, 16), OFFSETS)
    assert kept.count(x.data_ptr()) == 3
    for bad in (x[0], x[None]):
        for call in (lambda t: experts.dispatch(t, r), lambda t: experts.rms_norm_fp8(t),
                     lambda t: experts.combine(t, torch.ones(4, 2), r)):
            monkeypatch.undo()
            with pytest.raises((ValueError, IndexError)):
                call(bad)


def test_no_columns_reach_the_library(experts, monkeypatch):
    """Its own check refuses them; here it only notes the sizes."""
    seen = []
    for name in ("ag_gemm_rmsnorm", "ag_gemm_quant_mxfp4", "ag_gemm_dequant_mxfp4"):
        monkeypatch.setattr(experts.agg, name, lambda x, *a, **kw: seen.append(tuple(x.shape)))
    x, codes = torch.empty(2, 3, 0), torch.empty(2, 3, 0, dtype=torch.uint8)
    experts.rms_norm(x)
    experts.quantize_mxfp4(x)
    experts.dequantize_mxfp4(codes, codes)
    assert seen == [(6, 0)] * 3
