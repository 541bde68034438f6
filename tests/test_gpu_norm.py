"""The root-mean-square norm and its gradient against 64-bit forms.

Tolerances: u = 2^-24.  A lane adds its columns one after the other (k / 64 at
most), then come the lanes, waves and a few single roundings, so with n = k / 64
+ 32 a sum of squares is off by n u of itself, rstd by (n / 2 + 4) u, y before
its rounding by (n / 2 + 8) u; the output's rounding is half a step."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float16, torch.bfloat16, torch.float32]
# each kernel's lengths, their ends, and lengths and strides it cannot take
SHAPES = [(1, 1, 0), (3, 7, 1), (2, 8, 0), (5, 128, 0), (70, 512, 8), (9, 520, 0), (3, 2048, 0), (4, 2056, 8),
          (6, 4096, 0), (3, 4104, 0), (5, 7168, 0), (2, 8192, 0), (3, 8200, 0), (2, 16384, 0), (2, 16392, 0),
          (3, 4099, 0), (2, 20001, 3), (600, 136, 0), (1100, 33, 0), (1030, 264, 0)]


@pytest.fixture(scope="module")
def agg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import communication_gemm_amd as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(seed, T, K, pad, dtype, scale=1.0):
    """Rows of a wider matrix."""
    return (torch.randn(T, K + pad, generator=gen(seed), device="cuda") * scale).to(dtype)[:, :K]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the smallest subnormal step."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def near(got, want, rel, extra=0.0):
    err = (got.double() - want).abs()
    tol = rel * want.abs() + extra + tiny(got.dtype)
    assert (err <= tol).all(), float((err / tol).max())


def inputs(T, K, pad, dtype):
    x, res = rows(1, T, K, pad, dtype), rows(2, T, K, pad, dtype, 3.0)
    weight = (1 + torch.randn(K, generator=gen(3), device="cuda") / 4).to(dtype)
    return x, res, weight


def norm64(x, res, weight, eps):
    """h as it is stored, and y and rstd from it in 64 bits."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hd = h.double()
    r = (hd.square().mean(1, keepdim=True) + eps).rsqrt()
    return h, hd * r * (1 if weight is None else weight.double()), r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,pad", SHAPES)
def test_norm(agg, dtype, T, K, pad):
    n = K / 64 + 32
    x, res, weight = inputs(T, K, pad, dtype)
    for use_res, use_w, keep in ((True, True, True), (False, True, False), (True, False, False), (False, False, True)):
        r, w = (res if use_res else None), (weight if use_w else None)
        want_h, want, rstd64 = norm64(x, r, w, 1e-5)
        y = torch.full((T, K + pad), 9., device="cuda").to(dtype)
        h = torch.full((T, K + pad), 9., device="cuda").to(dtype) if keep else None
        rstd = torch.empty(T, device="cuda") if keep else None
        agg.ag_gemm_rmsnorm(x, w, y=y[:, :K], residual=r, h=None if h is None else h[:, :K], rstd=rstd, eps=1e-5)
        near(y[:, :K], want, half_step(dtype) + (n / 2 + 8) * U)
        assert (y[:, K:] == 9).all()
        if keep:
            assert torch.equal(h[:, :K], want_h) and (h[:, K:] == 9).all()
            near(rstd, rstd64[:, 0], (n / 2 + 4) * U)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,pad", SHAPES)
def test_norm_to_codes(agg, dtype, T, K, pad):
    """Codes are the nearest of y / scale: half a step (2^-4 of the value, or
    2^-10 of the scale below the normal ones), y itself being off as above; the
    scale is amax / 448.  y and h are those of a call without codes."""
    n = K / 64 + 32
    rel = (n / 2 + 12) * U
    x, res, weight = inputs(T, K, pad, dtype)
    kb = -(-K // 128)
    q = torch.zeros(T, K + pad, dtype=torch.uint8, device="cuda")
    scale = torch.full((T, kb + 1), 9., device="cuda")
    h, y = torch.empty(T, K, dtype=dtype, device="cuda"), torch.empty(T, K, dtype=dtype, device="cuda")
    agg.ag_gemm_rmsnorm(x, weight, y=y, q=q[:, :K], scale=scale[:, :kb], residual=res, h=h)
    want_h, want, _ = norm64(x, res, weight, 1e-6)
    assert torch.equal(h, want_h) and (scale[:, kb:] == 9).all() and (q[:, K:] == 0).all()
    y2, h2 = torch.empty_like(y), torch.empty_like(h)
    agg.ag_gemm_rmsnorm(x, weight, y=y2, residual=res, h=h2)
    assert torch.equal(y, y2)
    pad64 = torch.nn.functional.pad(want, (0, kb * 128 - K)).view(T, kb, 128)
    near(scale[:, :kb], pad64.abs().amax(2).clamp_min(2.0 ** -100) / 448, rel + 2 * U)
    each = scale[:, :kb].double().repeat_interleave(128, 1)[:, :K]
    codes = q[:, :K].contiguous().view(torch.float8_e4m3fn).double()
    err = (codes * each - want).abs()
    assert (err <= (2.0 ** -4 + 2 * rel) * want.abs() + 2.0 ** -10 * each * (1 + rel)).all()


def test_codes_are_the_exact_values(agg):
    """Of 16-bit rows, whose products u with the weight float32 holds: 448 u /
    amax(u) is off by 2^-24 at most, so a code differs from the exact value's only
    where that lies so near a tie (ties lie 2^-4 of the value apart or more: 2^-20 of
    the codes, 8 of 2^23).  Compared as 448 u against tie * amax(u), both exact."""
    levels = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                           for c in range(0x7F)], dtype=torch.float64, device="cuda")
    T, K = 2048, 4096
    for dtype in (torch.float16, torch.bfloat16):
        x, res, weight = inputs(T, K, 0, dtype)
        q, s = torch.empty(T, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, K // 128, device="cuda")
        h = torch.empty_like(x)
        agg.ag_gemm_rmsnorm(x, weight, q=q, scale=s, residual=res, h=h)
        u = (h.double() * weight.double()).view(T, K // 128, 128)
        amax = u.abs().amax(2, keepdim=True).expand_as(u).reshape(T, K)
        u = u.view(T, K)
        hi = torch.searchsorted(levels, (u.abs() / amax * 448).contiguous()).clamp(1, 126)
        lo = hi - 1
        tie = (levels[hi] + levels[lo]) / 2 * amax
        a = u.abs() * 448
        want = torch.copysign(torch.where((a > tie) | ((a == tie) & (hi % 2 == 0)), levels[hi], levels[lo]), u)
        wrong = q.double() != want
        assert int(wrong.sum()) <= 8
        assert ((a - tie).abs() <= 2.0 ** -23 * tie)[wrong].all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,pad", SHAPES)
def test_norm_grad(agg, dtype, T, K, pad):
    """dx's two terms are each off by their roundings and the mean's: (n + 16) u
    of their magnitudes; dw's sum over rows by T / 512 + 96 additions and rstd."""
    n = K / 64 + 32
    x, _, weight = inputs(T, K, pad, dtype)
    h, dy, dh = x, rows(4, T, K, pad, dtype), rows(5, T, K, pad, dtype)
    hd, gd = h.double(), dy.double()
    r = (hd.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    rstd = r[:, 0].float()
    r = rstd.double()[:, None]          # the gradient's own input
    ws = torch.full((agg.rmsnorm_grad_workspace_bytes(T, K),), 0x7f, dtype=torch.uint8, device="cuda")
    for use_w, use_dh, want_dw in ((True, True, True), (True, False, True), (False, True, False), (False, False, True)):
        w64 = weight.double() if use_w else torch.ones_like(weight).double()
        g = gd * w64
        mean, mean_abs = (g * hd).mean(1, keepdim=True), (g * hd).abs().mean(1, keepdim=True)
        want = r * (g - hd * r * r * mean) + (dh.double() if use_dh else 0)
        mags = r * (g.abs() + hd.abs() * r * r * mean_abs) + (dh.double().abs() if use_dh else 0)
        want_w, mags_w = (gd * hd * r).sum(0), (gd * hd * r).abs().sum(0)
        for dw_type in {dtype, torch.float32} if want_dw else {None}:
            dx = torch.full((T, K + pad), 9., device="cuda").to(dtype)
            dw = None if dw_type is None else torch.empty(K, dtype=dw_type, device="cuda")
            agg.ag_gemm_rmsnorm_grad(dy, h, weight if use_w else None, rstd, dx[:, :K], dw, ws,
                                     dh=dh if use_dh else None)
            near(dx[:, :K], want, half_step(dtype), (n + 16) * U * mags)
            assert (dx[:, K:] == 9).all()
            if dw is not None:
                near(dw, want_w, half_step(dw_type), (T / 512 + 96) * U * mags_w)


def test_gradient_against_differences(agg):
    """float32 rows: (f(v + e d) - f(v - e d)) / 2e along random directions.  e
    = 2^-7 leaves e^2 of third derivatives (1e-4 of order one values) and
    rounding of 1e-6 / e."""
    from communication_gemm_amd.experts import rms_norm
    T, K = 7, 264
    x, res, w = (t.clone().requires_grad_() for t in inputs(T, K, 0, torch.float32))
    cy, ch = rows(6, T, K, 0, torch.float32), rows(7, T, K, 0, torch.float32)

    def loss(x, res, w):
        y, h = rms_norm(x, w, res)
        return (y.double() * cy).sum() + (h.double() * ch).sum()

    loss(x, res, w).backward()
    for i, t in enumerate((x, res, w)):
        d = torch.randn(t.shape, generator=gen(8 + i), device="cuda")
        e = 2.0 ** -7
        with torch.no_grad():
            args = [x, res, w]
            args[i] = t + e * d
            up = loss(*args)
            args[i] = t - e * d
            slope = (up - loss(*args)) / (2 * e)
        want = (t.grad.double() * d).sum()
        scale = (t.grad.double() * d).abs().sum() + T * K * 1e-2
        assert abs(float(slope - want)) <= 3e-3 * float(scale), (i, float(slope), float(want))


@pytest.mark.parametrize("dtype", TYPES)
def test_rms_norm_has_its_gradients(agg, dtype):
    """Leading dimensions, an unused output, no residual, no weight."""
    from communication_gemm_amd.experts import rms_norm
    x0, r0, w0 = inputs(12, 72, 0, dtype)
    x0, r0 = x0.view(3, 4, 72), r0.view(3, 4, 72)

    def leaf(t):
        return t.clone().requires_grad_()

    def plain(x, w, h_grad, dy):
        xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
        y = xd * (xd.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wd
        ((y * dy).sum() + (xd * h_grad).sum()).backward()
        return xd.grad, wd.grad

    rel = 4 * half_step(dtype) + 200 * U
    dy, dh = rows(6, 12, 72, 0, dtype).view(3, 4, 72), rows(7, 12, 72, 0, dtype).view(3, 4, 72)
    x, r, w = leaf(x0), leaf(r0), leaf(w0)
    y, h = rms_norm(x, w, r)
    torch.autograd.backward([y, h], [dy, dh])
    gx, gw = plain(h, w, dh.double(), dy.double())
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    near(x.grad, gx, rel, rel * 3)
    near(w.grad, gw, rel, rel * 12)
    x, r, w = leaf(x0), leaf(r0), leaf(w0)
    y, h = rms_norm(x, w, r)
    h.backward(dh)                                   # the norm itself unused
    assert torch.equal(x.grad, dh) and torch.equal(r.grad, dh) and (w.grad is None or (w.grad == 0).all())
    x, w = leaf(x0), leaf(w0)
    rms_norm(x, w).backward(dy)
    gx, gw = plain(x, w, torch.zeros_like(dy).double(), dy.double())
    near(x.grad, gx, rel, rel * 3)
    near(w.grad, gw, rel, rel * 12)
    x = leaf(x0)
    rms_norm(x).backward(dy)
    gx, _ = plain(x, torch.ones_like(w0), torch.zeros_like(dy).double(), dy.double())
    near(x.grad, gx, rel, rel * 3)


def test_rms_norm_of_other_strides(agg):
    """Transposed and expanded tensors, one row, no rows."""
    from communication_gemm_amd.experts import rms_norm
    x, res, w = (t.float() for t in inputs(72, 40, 0, torch.float32))
    w = w.new_ones(72)
    for a in (x.t(), x.t()[None].expand(3, -1, -1), x.t()[5], x.t()[:0]):
        a = a.detach().requires_grad_()
        y = rms_norm(a, w)
        y.backward(torch.ones_like(y))
        b = a.detach().double().contiguous().requires_grad_()
        z = b * (b.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        z.backward(torch.ones_like(z))
        near(y, z, 40 * U)
        near(a.grad, b.grad, 40 * U, 200 * U)


@pytest.mark.parametrize("K", [264, 4099])
@pytest.mark.parametrize("place", ["x", "residual"])
def test_h_in_the_place_of_an_input(agg, K, place):
    x, res, weight = inputs(5, K, 0, torch.bfloat16)
    want_h, want_y = torch.empty_like(x), torch.empty_like(x)
    agg.ag_gemm_rmsnorm(x, weight, y=want_y, residual=res, h=want_h)
    y = torch.empty_like(x)
    h = x if place == "x" else res
    agg.ag_gemm_rmsnorm(x, weight, y=y, residual=res, h=h)
    assert torch.equal(h, want_h) and torch.equal(y, want_y)


@pytest.mark.parametrize("K", [64, 4096, 4099])
def test_rows_of_zeros_infinities_and_nan(agg, K):
    """Zeros stay zeros (eps keeps rstd finite); a row with a value that is not
    finite becomes NaN where the formula is, and touches no other row."""
    x = rows(9, 4, K, 0, torch.float32)
    x[0] = 0
    x[1, K // 2] = float("inf")
    x[2, 0] = float("nan")
    y, rstd = torch.empty_like(x), torch.empty(4, device="cuda")
    kb = -(-K // 128)
    q, scale = torch.empty(4, K, dtype=torch.uint8, device="cuda"), torch.empty(4, kb, device="cuda")
    agg.ag_gemm_rmsnorm(x, None, y=y, q=q, scale=scale, rstd=rstd, eps=2.0 ** -20)
    assert (y[0] == 0).all() and rstd[0] == 2.0 ** 10 and (q[0] & 0x7f == 0).all()
    assert rstd[1] == 0 and y[1, K // 2].isnan() and (y[1, :K // 2] == 0).all()
    assert y[2].isnan().all() and not scale[2].isfinite().any()
    assert not scale[1, K // 2 // 128].isfinite()
    near(y[3], norm64(x[3:], None, None, 2.0 ** -20)[1][0], (K / 128 + 24) * U)


def test_no_rows(agg):
    """Nothing to write but the weight's gradient, which is zeros."""
    x = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    agg.ag_gemm_rmsnorm(x, None, y=torch.empty_like(x))
    dw = torch.full((264,), 9., device="cuda")
    agg.ag_gemm_rmsnorm_grad(x, x, None, torch.empty(0, device="cuda"), torch.empty_like(x), dw)
    assert (dw == 0).all()


def test_rows_past_32_bit_offsets(agg):
    K = 8192
    T = (1 << 32) // (2 * K) + 3
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-2:] = rows(10, 2, K, 0, torch.bfloat16)
    y = torch.empty_like(x)
    rstd = torch.empty(T, device="cuda")
    agg.ag_gemm_rmsnorm(x, None, y=y, rstd=rstd)
    few = torch.empty(2, K, dtype=torch.bfloat16, device="cuda")
    agg.ag_gemm_rmsnorm(x[-2:], None, y=few)
    assert torch.equal(y[-2:], few) and (y[-3] == 0).all()
    dw = torch.empty(K, device="cuda")
    ws = torch.empty(agg.rmsnorm_grad_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    dx = y
    agg.ag_gemm_rmsnorm_grad(x, x, None, rstd, dx, dw, ws)
    xd, r = x[-2:].double(), rstd[-2:].double()[:, None]
    near(dw, (xd * xd * r).sum(0), 1024 * U)
    near(dx[-2:], r * (xd - xd * r * r * (xd * xd).mean(1, keepdim=True)), half_step(torch.bfloat16),
         200 * U * r * xd.abs())


def test_captured_training_step(agg):
    """Forward and backward in one graph, replayed with eager work in between."""
    T, K = 300, 520
    x, res, w = inputs(T, K, 0, torch.bfloat16)
    dy, dh = rows(11, T, K, 0, torch.bfloat16), rows(12, T, K, 0, torch.bfloat16)
    h, y, dx = (torch.empty_like(x) for _ in range(3))
    rstd, dw = torch.empty(T, device="cuda"), torch.empty(K, device="cuda")
    ws = torch.empty(agg.rmsnorm_grad_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")

    def work():
        agg.ag_gemm_rmsnorm(x, w, y=y, residual=res, h=h, rstd=rstd)
        agg.ag_gemm_rmsnorm_grad(dy, h, w, rstd, dx, dw, ws, dh=dh)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in range(4):
        x.copy_(rows(20 + seed, T, K, 0, torch.bfloat16))
        for t in (y, dx, dw):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, h, dx, dw)]
        ws.fill_(0x7f)
        work()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, h, dx, dw)))


def test_codes_refuse_a_gradient(agg):
    from communication_gemm_amd.experts import rms_norm_fp8
    x, res, w = inputs(4, 256, 0, torch.bfloat16)
    for a in ((x.clone().requires_grad_(), w, None), (x, w.clone().requires_grad_(), res)):
        got = rms_norm_fp8(*a)
        with pytest.raises(RuntimeError, match="no gradient"):
            got[1].sum().backward()
    q, scale, h = rms_norm_fp8(x, w, res)
    assert not scale.requires_grad and torch.equal(h, (x.float() + res.float()).bfloat16())
