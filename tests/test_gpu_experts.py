"""The expert products on the GPU against 64-bit references.

Two kinds of inputs:
  * whole numbers so small that every partial sum is exact in fp32 (at most
    2^24): the result has one correct value, and an fp32 output must equal it
    bit for bit, a 16-bit one its rounding;
  * normal draws, held to the forward error of an fp32 sum in any order,
    R * 2^-23 * sum |p q| (twice the unit roundoff for each of R terms), plus
    the output's own rounding, 2^-8 (bf16) or 2^-11 (fp16) of the value and
    half of fp16's smallest step.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
OUT_REL = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def agg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import communication_gemm_amd as m
    return m


def whole(seed, *shape, top=3):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g).double()


def normal(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).double()


def strided(t, dtype, ld=None, shift=0):
    """t on the GPU as `dtype`, its rows `ld` apart and its start `shift`
    elements into a buffer whose other elements are NaN."""
    *lead, m, n = t.shape
    ld = n if ld is None else ld
    groups = int(np.prod(lead)) if lead else 1
    size = shift + groups * m * ld + 64
    if dtype == torch.float8_e4m3fn:
        buf = torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda").view(dtype)
    else:
        buf = torch.full((size,), float("nan"), dtype=dtype, device="cuda")
    st = ([m * ld] if lead else []) + [ld, 1]
    v = buf.as_strided(t.shape, st, shift)
    if dtype == torch.float8_e4m3fn:
        v.view(torch.uint8).copy_(t.to(dtype).view(torch.uint8))
    else:
        v.copy_(t)
    return v, buf


def offsets_of(counts, first=0):
    return torch.tensor(np.cumsum([first] + list(counts)), dtype=torch.int32, device="cuda")


def grouped_reference(x, w, counts, trans):
    y = torch.zeros(x.shape[0], w.shape[1 if trans else 2], dtype=torch.float64)
    a = torch.zeros_like(y)
    lo = 0
    for e, c in enumerate(counts):
        m = w[e].t() if trans else w[e]
        y[lo:lo + c] = x[lo:lo + c] @ m
        a[lo:lo + c] = x[lo:lo + c].abs() @ m.abs()
        lo += c
    return y, a


def check(got, want, sum_abs, R, out):
    got = got.double().cpu()
    bound = R * 2.0 ** -23 * sum_abs + OUT_REL[out] * want.abs() + (2.0 ** -25 if out == "f16" else 0)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} out of bound, first {bad.nonzero()[:3].tolist()}"


COUNTS = {
    "one row": [1],
    "ones and empties": [0, 1, 0, 0, 1, 2, 0],
    "all empty but one": [0] * 70 + [37] + [0] * 9,
    "tile edges": [255, 1, 256, 0, 257, 15, 16, 17],
    "middling": [63, 64, 65, 127, 128, 129, 31, 33],
    "long": [1500, 40],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K,N", [(8, 8), (64, 72), (200, 264), (1032, 520), (13, 7), (129, 300)])
def test_grouped_whole_numbers(agg, name, trans, K, N):
    counts = COUNTS[name]
    T, E = sum(counts), len(counts)
    x, w = whole(1, T, K), whole(2, E, *((N, K) if trans else (K, N)))
    want, _ = grouped_reference(x, w, counts, trans)
    off = offsets_of(counts)
    for typ, out in (("f16", "f32"), ("bf16", "bf16")):
        y = torch.full((T, N), float("nan"), dtype=DT[out], device="cuda")
        agg.ag_gemm_grouped(x.to(DT[typ]).cuda(), w.to(DT[typ]).cuda(), off, y, trans)
        assert torch.equal(y.cpu(), want.to(DT[out])), (typ, out)


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K", [96, 2048])
def test_grouped_normal(agg, typ, trans, K):
    counts, N = [5, 0, 130, 300, 1], 136
    T, E = sum(counts), len(counts)
    x = normal(3, T, K).to(DT[typ]).double()
    w = normal(4, E, *((N, K) if trans else (K, N))).to(DT[typ]).double()
    want, sum_abs = grouped_reference(x, w, counts, trans)
    for out in (typ, "f32"):
        y = torch.empty(T, N, dtype=DT[out], device="cuda")
        agg.ag_gemm_grouped(x.to(DT[typ]).cuda(), w.to(DT[typ]).cuda(), offsets_of(counts), y, trans)
        check(y, want, sum_abs, K, out)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("shift,pad", [(0, 8), (0, 3), (1, 0), (8, 16)])
def test_grouped_strides_and_untouched_memory(agg, trans, shift, pad):
    """Padded rows, shifted starts; NaN in everything the call must not read
    (the padding, rows of no group) and values it must not overwrite."""
    counts, first, K, N = [3, 0, 70, 129, 20], 5, 72, 136
    T, E = first + sum(counts) + 9, len(counts)
    x, w = whole(5, T, K), whole(6, E, *((N, K) if trans else (K, N)))
    want, _ = grouped_reference(x[first:], w, counts, trans)
    xs, _ = strided(x, torch.bfloat16, K + pad, shift)
    xs[:first] = float("nan")
    xs[first + sum(counts):] = float("nan")
    ws, _ = strided(w, torch.bfloat16, w.shape[-1] + pad, shift)
    buf = torch.full((shift + T * (N + pad) + 64,), 7.0, device="cuda")
    y = buf.as_strided((T, N), (N + pad, 1), shift)
    agg.ag_gemm_grouped(xs, ws, offsets_of(counts, first), y, trans)
    full = torch.full((T, N), 7.0)
    full[first:first + sum(counts)] = want[:sum(counts)].float()
    assert torch.equal(y.cpu(), full)
    y.fill_(7.0)
    assert (buf == 7.0).all(), "memory outside y was written"


def test_grouped_shared_weights_and_row_views(agg):
    """One matrix for every group (stride 0), x a column slice of a wider one."""
    counts, K, N = [4, 40, 0, 200], 64, 128
    T = sum(counts)
    wide, w = whole(7, T, 3 * K), whole(8, 1, K, N)
    want = wide[:, K:2 * K] @ w[0]
    x = wide.to(torch.float16).cuda()[:, K:2 * K]
    y = torch.empty(T, N, device="cuda")
    agg.ag_gemm_grouped(x, w.to(torch.float16).cuda().expand(4, K, N), offsets_of(counts), y)
    assert torch.equal(y.cpu(), want.float())


@pytest.mark.parametrize("bad", [[-5, 10, 20], [0, 10, 10 ** 6], [0, 12, 4]])
def test_offsets_outside_the_rows_stay_in_the_buffers(agg, bad):
    """Offsets that break the rules: rows that one group alone holds keep
    their result, and nothing outside y is written."""
    T, K, N = 20, 64, 64
    x, w = whole(9, T, K), whole(10, 2, K, N)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    buf = torch.full((64 + T * N + 64,), 7.0, device="cuda")
    y = buf[64:64 + T * N].view(T, N)
    agg.ag_gemm_grouped(x.half().cuda(), w.half().cuda(), off, y)
    dw = torch.empty(2, K, N, device="cuda")
    agg.ag_gemm_grouped_wgrad(x.half().cuda(), x.half().cuda(), off, dw)
    if bad[2] != 4:
        assert torch.equal(y[:10].cpu(), (x[:10] @ w[0]).float())
        assert torch.equal(y[10:].cpu(), (x[10:] @ w[1]).float())
        assert torch.equal(dw[1].cpu(), (x[10:].t() @ x[10:]).float())
    assert (buf[:64] == 7.0).all() and (buf[64 + T * N:] == 7.0).all()


def test_no_rows(agg):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = (torch.empty(0, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.ones(3, 64, 64, dtype=torch.bfloat16, device="cuda")
    agg.ag_gemm_grouped(x, w, off, torch.empty_like(dy))
    dw = torch.full((3, 64, 64), float("nan"), device="cuda")
    agg.ag_gemm_grouped_wgrad(x, dy, off, dw)
    assert (dw == 0).all()


def test_non_finite_values_stay_in_their_rows(agg):
    counts, K, N = [100, 60, 3], 128, 256
    T = sum(counts)
    x, w = whole(11, T, K), whole(12, 3, K, N)
    want, _ = grouped_reference(x, w, counts, False)
    xg = x.to(torch.bfloat16).cuda()
    xg[7, 3] = float("nan")
    xg[99, 0] = float("inf")
    xg[160, 127] = float("nan")
    y = torch.empty(T, N, device="cuda")
    agg.ag_gemm_grouped(xg, w.to(torch.bfloat16).cuda(), offsets_of(counts), y)
    y = y.cpu()
    for r in (7, 160):
        assert y[r].isnan().all()
    assert not y[99][w[0][0] != 0].isfinite().any()
    keep = [r for r in range(T) if r not in (7, 99, 160)]
    assert torch.equal(y[keep], want[keep].float())


# ---- weight gradient ------------------------------------------------------

@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("K,N", [(8, 8), (72, 264), (300, 129), (520, 256)])
def test_wgrad_whole_numbers(agg, name, K, N):
    counts = COUNTS[name][-12:] if len(COUNTS[name]) > 12 else COUNTS[name]
    T, E = sum(counts), len(counts)
    x, dy = whole(13, T, K), whole(14, T, N)
    want = torch.stack([a.t() @ b for a, b in zip(x.split(counts), dy.split(counts))])
    for typ, out in (("f16", "f32"), ("bf16", "bf16")):
        dw = torch.full((E, K, N), float("nan"), dtype=DT[out], device="cuda")
        agg.ag_gemm_grouped_wgrad(x.to(DT[typ]).cuda(), dy.to(DT[typ]).cuda(), offsets_of(counts), dw)
        assert torch.equal(dw.cpu(), want.to(DT[out])), (typ, out)


def test_wgrad_strides_nan_neighbours_and_untouched_memory(agg):
    """Rows of no group are NaN, and so is the padding of x and dy; the
    padding of dw keeps its values.  Group ends fall inside a slice."""
    counts, first, K, N = [3, 0, 70, 129], 5, 72, 136
    T = first + sum(counts) + 9
    x, dy = whole(15, T, K), whole(16, T, N)
    lo, want = first, []
    for c in counts:
        want.append(x[lo:lo + c].t() @ dy[lo:lo + c])
        lo += c
    for pad, shift in ((8, 0), (3, 1)):
        xs, _ = strided(x, torch.bfloat16, K + pad, shift)
        ds, _ = strided(dy, torch.bfloat16, N + pad, shift)
        for t in (xs, ds):
            t[:first] = float("nan")
            t[first + sum(counts):] = float("nan")
        buf = torch.full((4 * K * (N + pad) + 64,), 7.0, device="cuda")
        dw = buf.as_strided((4, K, N), (K * (N + pad), N + pad, 1), 8)
        agg.ag_gemm_grouped_wgrad(xs, ds, offsets_of(counts, first), dw)
        assert torch.equal(dw.cpu(), torch.stack(want).float())
        dw.fill_(7.0)
        assert (buf == 7.0).all()


@pytest.mark.parametrize("typ", ["f16", "bf16"])
def test_wgrad_normal(agg, typ):
    counts, K, N = [700, 3, 0, 64], 136, 200
    T = sum(counts)
    x, dy = (normal(s, T, n).to(DT[typ]).double() for s, n in ((17, K), (18, N)))
    pairs = list(zip(x.split(counts), dy.split(counts)))
    want = torch.stack([a.t() @ b for a, b in pairs])
    sum_abs = torch.stack([a.abs().t() @ b.abs() for a, b in pairs])
    for out in (typ, "f32"):
        dw = torch.empty(4, K, N, dtype=DT[out], device="cuda")
        agg.ag_gemm_grouped_wgrad(x.to(DT[typ]).cuda(), dy.to(DT[typ]).cuda(), offsets_of(counts), dw)
        check(dw, want, sum_abs, max(counts), out)


@pytest.mark.parametrize("trans", [False, True])
def test_gradients_against_formula_and_differences(agg, trans):
    """Whole numbers make the product, its gradients and differences of the
    loss exact: L(x + d) - L(x) = <dL/dx, d> because L is linear in x and in w."""
    from communication_gemm_amd.experts import grouped_linear
    counts, K, N = [3, 0, 9, 20], 24, 40
    T = sum(counts)
    x = whole(19, T, K, top=2).half().cuda().requires_grad_()
    w = whole(20, 4, *((N, K) if trans else (K, N)), top=2).half().cuda().requires_grad_()
    g = whole(21, T, N, top=2).half().cuda()
    off = offsets_of(counts)
    grouped_linear(x, w, off, trans).backward(g)
    gd, xd, wd = (t.detach().double().cpu() for t in (g, x, w))
    dx, _ = grouped_reference(gd, wd, counts, not trans)
    assert torch.equal(x.grad.double().cpu(), dx)
    dw = [a.t() @ b for a, b in zip(xd.split(counts), gd.split(counts))]
    dw = torch.stack([m.t() if trans else m for m in dw])
    assert torch.equal(w.grad.double().cpu(), dw)

    def loss(x, w):
        return (grouped_linear(x, w, off, trans).double() * g.double()).sum().item()

    with torch.no_grad():
        for seed in range(3):
            d = whole(30 + seed, T, K, top=1).half().cuda()
            assert loss(x + d, w) - loss(x, w) == (x.grad.double() * d.double()).sum().item()
            d = whole(40 + seed, *w.shape, top=1).half().cuda()
            assert loss(x, w + d) - loss(x, w) == (w.grad.double() * d.double()).sum().item()


def test_gradient_of_padded_rows_and_of_a_broadcast_output(agg):
    """padded: rows of no group give zeros; the gradient that sum() sends back
    is a broadcast of one number."""
    from communication_gemm_amd.experts import grouped_linear
    x = whole(22, 12, 16).half().cuda().requires_grad_()
    w = whole(23, 2, 16, 8).half().cuda().requires_grad_()
    off = torch.tensor([2, 5, 9], dtype=torch.int32, device="cuda")
    y = grouped_linear(x, w, off, padded=True)
    y.sum().backward()
    assert (y[:2] == 0).all() and (y[9:] == 0).all()
    assert (x.grad[:2] == 0).all() and (x.grad[9:] == 0).all()
    assert torch.equal(x.grad[2:5], w[0].sum(1).expand(3, 16))
    assert torch.equal(w.grad[1], x[5:9].sum(0)[:, None].expand(16, 8))


def test_second_derivatives_are_refused(agg):
    """The gradients' kernels are not recorded, so a derivative of them would
    be wrong without a word."""
    from communication_gemm_amd.experts import grouped_linear
    x = whole(44, 9, 16).to(torch.bfloat16).cuda().requires_grad_()
    w = whole(45, 2, 16, 8).to(torch.bfloat16).cuda().requires_grad_()
    y = grouped_linear(x, w, offsets_of([4, 5]))
    dx, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.float().sum().backward()


# ---- fp8 ------------------------------------------------------------------

def fp8_inputs(M, N, K, groups, exact):
    """Codes and scales; `exact`: whole numbers and powers of two."""
    kb, nb = -(-K // 128), -(-N // 128)
    if exact:
        a, b = whole(50, M, K), whole(51, groups, N, K)
        sa, sb = 2.0 ** whole(52, M, kb, top=2), 2.0 ** whole(53, groups, nb, kb, top=2)
    else:
        a, b = (normal(s, *sh).clamp(-6, 6).float().to(torch.float8_e4m3fn).double()
                for s, sh in ((54, (M, K)), (55, (groups, N, K))))
        sa, sb = (normal(s, *sh).abs().add(0.1).float().double()
                  for s, sh in ((56, (M, kb)), (57, (groups, nb, kb))))
    return a, sa, b, sb


def fp8_reference(a, sa, b, sb, counts):
    K, N = a.shape[1], b.shape[1]
    da = a * sa.repeat_interleave(128, 1)[:, :K]
    y, s = (torch.zeros(a.shape[0], N, dtype=torch.float64) for _ in range(2))
    lo = 0
    for e, c in enumerate(counts):
        db = b[e] * sb[e].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        y[lo:lo + c] = da[lo:lo + c] @ db.t()
        s[lo:lo + c] = da[lo:lo + c].abs() @ db.abs().t()
        lo += c
    return y, s


def e4m3(t):
    return t.float().to(torch.float8_e4m3fn).cuda()


@pytest.mark.parametrize("M", [1, 5, 16, 33, 64, 130, 257, 600])
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (264, 144), (520, 1040), (100, 77), (136, 2048)])
def test_fp8_dense_whole_numbers(agg, M, N, K):
    a, sa, b, sb = fp8_inputs(M, N, K, 1, True)
    want, _ = fp8_reference(a, sa, b, sb, [M])
    for out in ("f32", "bf16"):
        c = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        agg.ag_gemm_fp8_block(e4m3(a), sa.float().cuda(), e4m3(b[0]), sb[0].float().cuda(), c)
        assert torch.equal(c.cpu(), want.to(DT[out])), out


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", [(136, 272), (264, 1040), (50, 130)])
def test_fp8_grouped_whole_numbers(agg, name, N, K):
    counts = COUNTS[name]
    T = sum(counts)
    a, sa, b, sb = fp8_inputs(T, N, K, len(counts), True)
    want, _ = fp8_reference(a, sa, b, sb, counts)
    c = torch.full((T, N), float("nan"), device="cuda")
    agg.ag_gemm_grouped_fp8_block(e4m3(a), sa.float().cuda(), e4m3(b), sb.float().cuda(),
                                  offsets_of(counts), c)
    assert torch.equal(c.cpu(), want.float())


@pytest.mark.parametrize("M", [3, 200, 700])
def test_fp8_normal(agg, M):
    N, K = 392, 1552
    a, sa, b, sb = fp8_inputs(M, N, K, 1, False)
    want, sum_abs = fp8_reference(a, sa, b, sb, [M])
    for out in ("f32", "f16", "bf16"):
        c = torch.empty(M, N, dtype=DT[out], device="cuda")
        agg.ag_gemm_fp8_block(e4m3(a), sa.float().cuda(), e4m3(b[0]), sb[0].float().cuda(), c)
        # two more roundings a term: the product of the scales, and its use
        check(c, want, sum_abs, K + 2, out)


@pytest.mark.parametrize("pad,shift", [(16, 0), (5, 3)])
def test_fp8_strides_and_untouched_memory(agg, pad, shift):
    counts, N, K = [3, 0, 70, 130], 136, 272
    T = sum(counts)
    a, sa, b, sb = fp8_inputs(T, N, K, 4, True)
    want, _ = fp8_reference(a, sa, b, sb, counts)
    at, _ = strided(a, torch.float8_e4m3fn, K + pad, shift)
    bt, _ = strided(b, torch.float8_e4m3fn, K + pad, shift)
    sat, _ = strided(sa, torch.float32, sa.shape[1] + 2, shift)
    sbt, _ = strided(sb, torch.float32, sb.shape[2] + 2, shift)
    buf = torch.full((shift + T * (N + pad) + 64,), 7.0, device="cuda")
    c = buf.as_strided((T, N), (N + pad, 1), shift)
    agg.ag_gemm_grouped_fp8_block(at, sat, bt, sbt, offsets_of(counts), c)
    assert torch.equal(c.cpu(), want.float())
    c.fill_(7.0)
    assert (buf == 7.0).all()


def quant_reference(x, br):
    """The stated formulas in numpy float32, each operation rounded once."""
    import synth
    x = x.float().numpy()
    M, K = x.shape
    q = np.zeros((M, K), np.uint8)
    scale = np.zeros((-(-M // br), -(-K // 128)), np.float32)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            blk = x[i * br:(i + 1) * br, j * 128:(j + 1) * 128]
            amax = np.float32(max(np.abs(blk).max(), np.float32(2.0 ** -100)))
            scale[i, j] = amax / np.float32(448)
            q[i * br:(i + 1) * br, j * 128:(j + 1) * 128] = synth.to_fp8e4m3_bits(
                blk * (np.float32(448) / amax))
    return q, scale


@pytest.mark.parametrize("typ", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 128), (17, 200), (130, 264), (129, 1000), (5, 37)])
def test_quant(agg, typ, br, M, K):
    x = normal(60, M, K) * torch.exp(2 * normal(61, 1, K))
    x[0, 0] = 0.0
    x = x.to(DT[typ])
    if M > 2:
        x[1] = 0.0                     # zero blocks
        x[2, :K // 2] = torch.tensor(2.0 ** -24).to(DT[typ])   # fp16's smallest value
    q = torch.full((M, K), 0xEE, dtype=torch.uint8, device="cuda")
    scale = torch.full((-(-M // br), -(-K // 128)), float("nan"), device="cuda")
    agg.ag_gemm_quant_fp8_block(x.cuda(), q, scale, br)
    qr, sr = quant_reference(x, br)
    assert np.array_equal(scale.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("br", [1, 128])
def test_quant_strides_and_non_finite_blocks(agg, br):
    M, K = 140, 392
    x = normal(62, M, K).to(torch.bfloat16).double()
    for pad, shift in ((8, 0), (3, 1)):
        xs, _ = strided(x, torch.bfloat16, K + pad, shift)
        buf = torch.full((M * (K + pad) + 64,), 0xEE, dtype=torch.uint8, device="cuda")
        q = buf.as_strided((M, K), (K + pad, 1), shift)
        scale = torch.empty(-(-M // br), 4, device="cuda")
        agg.ag_gemm_quant_fp8_block(xs, q, scale, br)
        qr, sr = quant_reference(x, br)
        assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(scale.cpu().numpy(), sr)
        q.fill_(0xEE)
        assert (buf == 0xEE).all()
    xg = x.to(torch.bfloat16).cuda()
    xg[4, 130] = float("nan")
    xg[5, 3] = float("-inf")
    q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    agg.ag_gemm_quant_fp8_block(xg, q, scale, br)
    d = (q.float() * scale.repeat_interleave(br, 0)[:M].repeat_interleave(128, 1)[:, :K]).cpu()
    block = slice(0, 128) if br == 128 else None
    assert d[block or 4, 128:256].isnan().all() and d[block or 5, :128].isnan().all()
    keep = d[128:] if br == 128 else d[6:]
    assert keep.isfinite().all()


# ---- every kernel the sizes can choose --------------------------------------

# (rows of each group, N): sizes that choose each tile, their groups ending
# inside, at and just past a tile's edge
KERNELS = {
    "large, a cut round": ([700, 300, 129, 1, 257, 0, 128], 4360),
    "large, whole rounds": ([512, 1280, 256, 384], 4360),
    "large, one group": ([1700], 8200),
    "128 x 128": ([300, 257, 0, 511, 132], 2056),
    "128 x 128, many": ([120, 128, 129, 90, 64, 200], 2184),
    "64 x 256": ([3, 0, 64, 65, 17] * 12, 1032),
    "64 x 64, longer groups": ([100, 64, 65, 171], 1608),
    "64 x 64": ([20, 64, 1, 0, 7, 33, 16, 65], 1608),
    "64 x 64, few tiles": ([60, 70], 520),
    "64 x 64, one group": ([200], 328),
    "16 rows": ([1, 16, 17, 0, 3], 328),
    "32 rows": ([32, 33, 20, 18], 328),
    "32 rows, one group": ([60], 328),
}


@pytest.mark.parametrize("name", list(KERNELS))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K", [8, 64, 136, 520])
def test_every_grouped_kernel(agg, name, trans, K):
    counts, N = KERNELS[name]
    T, E = sum(counts), len(counts)
    x, w = whole(80, T, K).cuda(), whole(81, E, *((N, K) if trans else (K, N))).cuda()
    want = torch.cat([a @ (m.t() if trans else m) for a, m in zip(x.split(counts), w)])
    for typ, out in (("bf16", "f32"), ("f16", "f16")):
        y = torch.full((T, N), float("nan"), dtype=DT[out], device="cuda")
        agg.ag_gemm_grouped(x.to(DT[typ]), w.to(DT[typ]), offsets_of(counts), y, trans)
        assert torch.equal(y, want.to(DT[out])), (typ, out)


@pytest.mark.parametrize("name", list(KERNELS))
@pytest.mark.parametrize("K", [16, 128, 272, 1168])
def test_every_fp8_kernel(agg, name, K):
    counts, N = KERNELS[name]
    T, E = sum(counts), len(counts)
    a, sa, b, sb = (t.cuda() for t in fp8_inputs(T, N, K, E, True))
    da = a * sa.repeat_interleave(128, 1)[:, :K]
    want = torch.cat([m @ (q * s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).t()
                      for m, q, s in zip(da.split(counts), b, sb)])
    c = torch.full((T, N), float("nan"), device="cuda")
    if E == 1:
        agg.ag_gemm_fp8_block(e4m3(a), sa.float(), e4m3(b[0]), sb[0].float(), c)
    else:
        agg.ag_gemm_grouped_fp8_block(e4m3(a), sa.float(), e4m3(b), sb.float(), offsets_of(counts), c)
    assert torch.equal(c, want.float())


@pytest.mark.parametrize("counts,K,N", [
    ([70, 0, 1, 129, 64, 65], 1544, 2056),      # 256 x 256 tiles, ragged edges
    ([300] * 20, 776, 1032),
    ([70, 0, 1, 129, 64, 65], 136, 264),        # 128 x 128 tiles
])
def test_every_wgrad_kernel(agg, counts, K, N):
    T = sum(counts)
    x, dy = whole(82, T, K).cuda(), whole(83, T, N).cuda()
    want = torch.stack([a.t() @ b for a, b in zip(x.split(counts), dy.split(counts))])
    for typ, out in (("bf16", "f32"), ("f16", "f16")):
        dw = torch.full((len(counts), K, N), float("nan"), dtype=DT[out], device="cuda")
        agg.ag_gemm_grouped_wgrad(x.to(DT[typ]), dy.to(DT[typ]), offsets_of(counts), dw)
        assert torch.equal(dw, want.to(DT[out])), (typ, out)


@pytest.mark.parametrize("M,N,K", [(5, 512, 512), (64, 256, 128), (40, 512, 128), (300, 1024, 256),
                                   (2000, 2048, 128), (64, 255, 120)])
def test_fp8_float32_output_keeps_every_bit(agg, M, N, K):
    """A float32 output is the sum of 128 exact products a block, each added
    with an error of at most 2^-23 of the magnitudes, times two scales'
    product (three roundings), and of the blocks."""
    kb, nb = -(-K // 128), -(-N // 128)
    x = (normal(90, M, K) * torch.exp(normal(91, K))).float().cuda()
    w = normal(92, N, K).float().cuda()
    a, sa = (torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"),
             torch.empty(M, kb, device="cuda"))
    b, sb = (torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda"),
             torch.empty(nb, kb, device="cuda"))
    agg.ag_gemm_quant_fp8_block(x, a, sa, 1)
    agg.ag_gemm_quant_fp8_block(w, b, sb, 128)
    y = agg.ag_gemm_fp8_block(a, sa, b, sb, torch.empty(M, N, device="cuda"))
    p = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    q = b.double() * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    bound = (p.abs() @ q.abs().t()) * (128 + 3 + kb) * 2.0 ** -23
    assert ((y.double() - p @ q.t()).abs() <= bound).all()


# ---- streams, graphs, repeated calls ----------------------------------------

def test_other_stream_graph_and_repeats(agg):
    """The same bits on another stream, from a prepared call, and from every
    replay of a captured graph (with other work between the replays)."""
    counts, K, N = [5, 0, 90, 300], 256, 264
    T = sum(counts)
    x = normal(70, T, K).to(torch.bfloat16).cuda()
    w = normal(71, 4, K, N).to(torch.bfloat16).cuda()
    off = offsets_of(counts)
    a, sa = (torch.empty(T, K, dtype=torch.float8_e4m3fn, device="cuda"),
             torch.empty(T, K // 128, device="cuda"))
    b, sb = (torch.empty(4, N, K, dtype=torch.float8_e4m3fn, device="cuda"),
             torch.empty(4, -(-N // 128), K // 128, device="cuda"))
    for e in range(4):
        agg.ag_gemm_quant_fp8_block(w[e].t().contiguous(), b[e], sb[e], 128)
    outs = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dw = torch.empty(4, K, N, device="cuda")

    def step(**kw):
        return [agg.ag_gemm_grouped(x, w, off, outs[0], **kw),
                agg.ag_gemm_quant_fp8_block(x, a, sa, 1, **kw),
                agg.ag_gemm_grouped_fp8_block(a, sa, b, sb, off, outs[1], **kw),
                agg.ag_gemm_grouped_wgrad(x, outs[0], off, dw, **kw)]

    def results():
        torch.cuda.synchronize()
        got = [t.clone() for t in (*outs, dw, sa)] + [a.view(torch.uint8).clone()]
        for t in (*outs, dw, sa):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        return got

    step()
    want = results()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    runs = [results()]
    step(stream=s)
    runs.append(results())
    for call in step(prepare=True):
        call()
    runs.append(results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        graph.replay()
        runs.append(results())
        step()
        runs.append(results())
    for k, got in enumerate(runs):
        assert all(torch.equal(g, v) for g, v in zip(got, want)), k


def test_example_layer_trains_and_serves(agg):
    """The example runs the operators together: a training run lowers the
    loss, and fp8 serving stays near bf16 (E4M3 rounds a value by up to
    2^-4, on average about 2^-5.3 of it; two products with two rounded
    operands each, and the gate's product of two of their results)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, off = mod.main(["--tokens", "300", "--hidden", "256", "--inner", "128", "--experts", "8",
                            "--steps", "12"])
    assert losses[-1] < 0.8 * losses[0]
    assert off < 0.12
