"""Calls of the expert products as a program makes them: rows cut out of
larger tensors, gradients that do not exist, rows of no group, prepared calls
under another stream."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def agg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import communication_gemm_amd as m
    return m


def whole(seed, *shape, top=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").double()


def offsets(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("tokens", [3, 520])
def test_last_token_of_one_sequence(agg, tokens):
    """hidden[:, -1]: one row whose stride is the whole sequence's (past the
    largest row stride at 520 tokens of 4096)."""
    K, N = 4096, 264
    hidden = whole(1, 1, tokens, K).to(torch.bfloat16)
    w = whole(2, 2, K, N).to(torch.bfloat16)
    x = hidden[:, -1]
    want = (x.double() @ w[1].double()).float()
    off = offsets(0, 0, 1)
    y = torch.empty(1, tokens, N, device="cuda")[:, -1]
    agg.ag_gemm_grouped(x, w, off, y)
    assert torch.equal(y, want)
    dw = torch.empty(2, K, N, device="cuda")
    agg.ag_gemm_grouped_wgrad(x, y.to(torch.bfloat16), off, dw)
    assert torch.equal(dw[1], x.float().t() * y.to(torch.bfloat16).float()) and (dw[0] == 0).all()
    q, scale = torch.empty(1, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, 32, device="cuda")
    agg.ag_gemm_quant_fp8_block(x, q, scale)
    q2, scale2 = torch.empty_like(q), torch.empty_like(scale)
    agg.ag_gemm_quant_fp8_block(x.clone(), q2, scale2)
    assert torch.equal(scale, scale2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))


@pytest.mark.parametrize("out", [None, torch.float32])
def test_padded_fp8_batch(agg, out):
    """Rows of no group, as a batch padded to a fixed size has them, are zeros
    (and NaN in them reaches nothing); the others are as without padding."""
    from communication_gemm_amd.experts import grouped_linear_fp8, quantize_weights
    first, rows, T, K, N = 3, 40, 64, 256, 136
    x = whole(3, T, K).to(torch.bfloat16)
    x[:first] = float("nan")
    x[first + rows:] = float("nan")
    wq, ws = quantize_weights(whole(4, 2, N, K).to(torch.bfloat16))
    want = grouped_linear_fp8(x[first:first + rows].contiguous(), wq, ws, offsets(0, 15, rows), out)
    torch.full((T, N), float("nan"), dtype=want.dtype, device="cuda")   # the allocator's next block
    y = grouped_linear_fp8(x, wq, ws, offsets(first, first + 15, first + rows), out, padded=True)
    assert torch.equal(y[first:first + rows], want)
    assert (y[:first] == 0).all() and (y[first + rows:] == 0).all()


def test_prepared_calls_run_on_the_stream_that_is_current(agg):
    """A prepared call inside a graph capture becomes part of the graph, and
    under another stream it runs behind that stream's work."""
    T, K, N = 40, 256, 264
    xs = [whole(s, T, K).to(torch.bfloat16) for s in range(5)]
    w = whole(9, 2, K, N).to(torch.bfloat16)
    off = offsets(0, 17, T)
    x, y = torch.empty_like(xs[0]), torch.empty(T, N, device="cuda")
    call = agg.ag_gemm_grouped(x, w, off, y, prepare=True)
    own = torch.cuda.Stream()
    fixed = agg.ag_gemm_grouped(x, w, off, y, stream=own, prepare=True)

    def want(t):
        return torch.cat([t[:17].float() @ w[0].float(), t[17:].float() @ w[1].float()])

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in xs:
        x.copy_(t)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want(t))
        x.zero_()
        call()
        torch.cuda.synchronize()
        assert (y == 0).all()
    other = torch.cuda.Stream()
    for s, f in ((other, call), (own, fixed)):
        for t in xs:
            with torch.cuda.stream(s):
                x.copy_(t)
                f()
                got = y.clone()
            s.synchronize()
            assert torch.equal(got, want(t))


# ---- values and sizes at the ends of their ranges ------------------------------

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 70, 700])
def test_subnormal_values_count(agg, dtype, rows):
    """Small gradients: subnormal inputs are multiplied as they are, and
    fp16 results below 2^-14 keep their bits.  Whole multiples of the smallest
    step times whole numbers are exact."""
    step = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133
    K, N = 72, 264
    m = whole(20, rows, K)
    x = (m * step).to(dtype)
    assert torch.equal(x.double(), m * step)
    w = whole(21, 1, K, N).to(dtype)
    want = m @ w[0].double()
    off = offsets(0, rows)
    y = torch.empty(rows, N, device="cuda")
    agg.ag_gemm_grouped(x, w, off, y)
    assert torch.equal(y.double(), want * step)
    dw = torch.empty(1, K, N, device="cuda")
    dy = whole(22, rows, N).to(dtype)
    agg.ag_gemm_grouped_wgrad(x, dy, off, dw)
    assert torch.equal(dw[0].double(), (m.t() @ dy.double()) * step)
    y = torch.empty(rows, N, dtype=dtype, device="cuda")
    agg.ag_gemm_grouped(x, w, off, y)
    assert torch.equal(y.double(), (want * step).to(dtype).double())


def test_rows_past_32_bit_offsets(agg):
    """The last rows of matrices of more than 2^32 bytes (16-bit) and 2^31
    (fp8); the rows before them belong to no group."""
    K, N, last = 2048, 2056, 70
    T = (1 << 32) // (2 * K) + 5000
    at = T - last
    off = offsets(at, at + 30, T)
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    x[at:] = whole(23, last, K).to(torch.bfloat16)
    w = whole(24, 2, K, N).to(torch.bfloat16)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    y[at - 1] = 7
    agg.ag_gemm_grouped(x, w, off, y)
    xd, wd = x[at:].double(), w.double()
    want = torch.cat([xd[:30] @ wd[0], xd[30:] @ wd[1]])
    assert torch.equal(y[at:], want.to(torch.bfloat16)) and (y[at - 1] == 7).all()
    dw = torch.empty(2, K, N, device="cuda")
    y[at:] = whole(25, last, N).to(torch.bfloat16)
    agg.ag_gemm_grouped_wgrad(x, y, off, dw)
    yd = y[at:].double()
    assert torch.equal(dw.double(), torch.stack([xd[:30].t() @ yd[:30], xd[30:].t() @ yd[30:]]))
    x[:at] = 1
    q, s = torch.empty(T, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, K // 128, device="cuda")
    agg.ag_gemm_quant_fp8_block(x, q, s)
    q2, s2 = torch.empty(last, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(last, K // 128, device="cuda")
    agg.ag_gemm_quant_fp8_block(x[at:].contiguous(), q2, s2)
    assert torch.equal(q[at:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[at:], s2)
    b, sb = (torch.empty(2, N, K, dtype=torch.float8_e4m3fn, device="cuda"),
             torch.empty(2, -(-N // 128), K // 128, device="cuda"))
    for e in range(2):
        agg.ag_gemm_quant_fp8_block(w[e].t().contiguous(), b[e], sb[e], 128)
    agg.ag_gemm_grouped_fp8_block(q, s, b, sb, off, y)
    y2 = torch.empty(last, N, dtype=torch.bfloat16, device="cuda")
    agg.ag_gemm_grouped_fp8_block(q2, s2, b, sb, offsets(0, 30, last), y2)
    # the same rows by tiles for other sizes: 2^-7 of the value and, of sums that
    # cancel, 2^-11 of the magnitudes
    scale = (q2.double() * s2.double().repeat_interleave(128, 1)).abs()
    e = b.double() * sb.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
    mags = torch.cat([scale[:30] @ e[0].abs().t(), scale[30:] @ e[1].abs().t()])
    assert ((y[at:].double() - y2.double()).abs() <= 2.0 ** -7 * y2.double().abs() + 2.0 ** -11 * mags).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("rows", [3, 200])
def test_weights_past_32_bit_offsets(agg, trans, rows):
    """The last of so many experts that their weights take more than 2^32
    elements."""
    K, N = 8192, 8200
    E = (1 << 32) // (K * N) + 2
    w = torch.empty(E, *((N, K) if trans else (K, N)), dtype=torch.float16, device="cuda")
    w[-1] = whole(26, *w.shape[1:]).half()
    x = whole(27, rows, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = rows
    y = torch.empty(rows, N, device="cuda")
    agg.ag_gemm_grouped(x.half(), w, off, y, trans)
    m = w[-1].double()
    assert torch.equal(y.double(), x @ (m.t() if trans else m))
