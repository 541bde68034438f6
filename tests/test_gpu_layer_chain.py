"""The operators around the expert products together, as a layer uses them:
norm with the residual, router, sort, dispatch, products, combine; in training
with all gradients, and in serving with 8 and 4 bits, captured and padded."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_gemm_amd import experts
    return experts


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


T, TOP, E, K, N = 150, 3, 7, 256, 136


def inputs(dtype=torch.bfloat16):
    return dict(x=normal(1, T, K, dtype=dtype), res=normal(2, T, K, dtype=dtype),
                norm=(1 + normal(3, K, scale=0.1).float()).to(dtype),
                w_in=normal(4, E, K, N, scale=K ** -0.5, dtype=dtype),
                w_out=normal(5, E, N, K, scale=N ** -0.5, dtype=dtype),
                weight=torch.softmax(normal(6, T, TOP, dtype=torch.float32), 1),
                ids=torch.randint(0, E, (T, TOP), generator=gen(7), device="cuda"))


def test_training_step(ex):
    """float16 rows against the same layer in 64 bits: each of the six roundings
    on the way of a value is half a step (2^-11) of what it rounds, and a sum of n
    values of size s that are each off by e s is off by e s sqrt(n) typically, so
    outputs and gradients are within 6 * 2^-11 times a few of their norm."""
    p = inputs(torch.float16)
    ids = p.pop("ids")
    ids[5:9] = -1                                     # tokens that go nowhere
    leaf = {k: v.clone().requires_grad_() for k, v in p.items()}
    r = ex.sort_by_expert(ids, E)
    n, h = ex.rms_norm(leaf["x"], leaf["norm"], leaf["res"])
    a = ex.grouped_linear(ex.dispatch(n, r, True), leaf["w_in"], r.offsets, padded=True)
    y = ex.combine(ex.grouped_linear(torch.nn.functional.silu(a), leaf["w_out"], r.offsets, padded=True),
                   leaf["weight"], r, True)
    out = h + y
    dy = normal(8, T, K, scale=0.1, dtype=torch.float16)
    out.backward(dy)

    d = {k: v.double().requires_grad_() for k, v in p.items()}
    hd = d["x"] + d["res"]
    nd = hd * (hd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * d["norm"]
    yd = torch.zeros_like(hd)
    for j in range(TOP):
        has = ids[:, j] >= 0
        e = ids[:, j].clamp_min(0)
        mid = torch.nn.functional.silu((nd[:, None] @ d["w_in"][e])[:, 0])
        yd = yd + torch.where(has, d["weight"][:, j], 0.0)[:, None] * (mid[:, None] @ d["w_out"][e])[:, 0]
    (hd + yd).backward(dy.double())
    for got, want in [(out, hd + yd)] + [(leaf[k].grad, d[k].grad) for k in p]:
        off = (got.detach().double() - want).norm() / want.norm()
        assert off <= 4 * 6 * 2.0 ** -11, float(off)
    assert (leaf["weight"].grad[5:9] == 0).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_serving(ex, bits):
    """Against products of the values that the codes stand for, in 64 bits:
    grouped outputs of few hundred values a sum are off by a bf16 rounding (2^-8)
    and the fp8 instruction's 2^-11 of the magnitudes, the combined ones by
    another 2^-8.  Values below half of the outputs' mean size stand for those."""
    p = inputs()
    r = ex.sort_by_expert(p["ids"], E)
    w = p["w_in"].transpose(1, 2).contiguous()
    if bits == 8:
        q, s, y16, h = ex.rms_norm_fp8(p["x"], p["norm"], p["res"], with_y=True)
        wq, ws = ex.quantize_weights(w)
        rows = ex.dispatch(q, r), ex.dispatch(s, r)
        got = ex.grouped_linear_fp8(rows, wq, ws, r.offsets, torch.bfloat16)
        xv = q.double() * s.double().repeat_interleave(128, 1)
        wv = wq.double() * ws.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
        n2, h2 = ex.rms_norm(p["x"], p["norm"], p["res"])
        assert torch.equal(n2, y16) and torch.equal(h2, h)
    else:
        n, h = ex.rms_norm(p["x"], p["norm"], p["res"])
        wq, ws = ex.quantize_mxfp4(w)
        got = ex.grouped_linear_mxfp4(ex.dispatch(n, r), wq, ws, r.offsets)
        xv = ex.dequantize_mxfp4(*ex.quantize_mxfp4(n), torch.float32).double()
        wv = ex.dequantize_mxfp4(wq, ws, torch.float32).double()
    y = ex.combine(got, p["weight"], r)
    each = (xv[:, None, None] @ wv[p["ids"]].transpose(2, 3).contiguous())[:, :, 0]       # [T, top, N]
    mags = (xv.abs()[:, None, None] @ wv.abs()[p["ids"]].transpose(2, 3).contiguous())[:, :, 0]
    back = got.double()[r.place.long()]
    assert ((back - each).abs() <= 2.0 ** -8 * each.abs() + 2.0 ** -11 * mags).all()
    weight = p["weight"].double()[:, :, None]
    tol = 2.0 ** -8 * (each.abs() * weight).sum(1) + 2.0 ** -11 * (mags * weight).sum(1)
    want = (each * weight).sum(1)
    assert ((y.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()


def test_serving_under_another_default_type(ex):
    """The default type of a model that is built for serving changes nothing."""
    p = inputs()
    off = torch.tensor([0, 20, 20, 55, 70, 111, 140, T], dtype=torch.int32, device="cuda")

    def serve():
        wq, ws = ex.quantize_weights(p["w_in"].transpose(1, 2).contiguous())
        q, s, y, h = ex.rms_norm_fp8(p["x"], p["norm"], p["res"], with_y=True)
        return [t.view(torch.uint8) for t in (wq, q)] + [
            ws, s, y, h, ex.grouped_linear_fp8(p["x"], wq, ws, off), ex.rms_norm(p["x"], p["norm"]),
            ex.combine(p["x"], p["weight"][:T // TOP], ex.sort_by_expert(p["ids"][:T // TOP], E))]

    want = serve()
    torch.set_default_dtype(torch.bfloat16)
    try:
        got = serve()
    finally:
        torch.set_default_dtype(torch.float32)
    assert all(a.dtype == b.dtype and torch.equal(a, b) for a, b in zip(got, want))


def test_captured_serving_of_a_padded_batch(ex):
    """A graph of the whole chain on a fixed batch, of which a varying part is
    padding (ids of -1, rows of NaN): the others are as in an eager call on them
    alone, the padding's results zeros."""
    p = inputs()
    wq, ws = ex.quantize_mxfp4(p["w_in"].transpose(1, 2).contiguous())
    x, ids, weight = p["x"].clone(), p["ids"].clone(), p["weight"].clone()

    def serve(x, ids, weight, padded):
        r = ex.sort_by_expert(ids, E)
        n = ex.rms_norm(x, p["norm"])
        return ex.combine(ex.grouped_linear_mxfp4(ex.dispatch(n, r, padded), wq, ws, r.offsets, padded=padded),
                          weight, r)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.no_grad():
        serve(x, ids, weight, True)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        y = serve(x, ids, weight, True)
    for keep in (T, 1, 97, 40):
        x.copy_(normal(20 + keep, T, K))
        ids.copy_(torch.randint(0, E, (T, TOP), generator=gen(keep), device="cuda"))
        ids[keep:] = -1
        x[keep:] = float("nan")
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        with torch.no_grad():
            alone = serve(x[:keep], ids[:keep], weight[:keep], False)
        # kernels of other sizes add in another order: K u of sums that are some
        # tens, and a rounding that then goes the other way
        assert ((got[:keep].float() - alone.float()).abs() <= 2.0 ** -7 * alone.float().abs() + 2.0 ** -8).all()
        assert (got[keep:] == 0).all()


def test_rows_of_other_strides(ex):
    """Transposed and expanded rows give what their copies do, gradients too."""
    p = inputs()
    r = ex.sort_by_expert(p["ids"], E)
    turn = {k: p[k].t().contiguous().t() for k in ("x", "res", "weight")}
    wide = torch.stack([p["norm"], p["norm"]], 1)[:, 0]

    def run(x, res, weight, norm):
        x, res, weight, norm = (t.detach().requires_grad_() for t in (x, res, weight, norm))
        y, h = ex.rms_norm(x, norm, res)
        a = ex.grouped_linear(ex.dispatch(h.t().contiguous().t(), r).t().contiguous().t(), p["w_in"], r.offsets)
        out = ex.combine(a.t().contiguous().t(), weight, r)
        (out.float().sum() + y.float().sum()).backward()
        with torch.no_grad():
            codes = [t.view(torch.uint8) for t in (*ex.rms_norm_fp8(x, norm, res, with_y=True), *ex.quantize(x))]
        return [out, y, h, x.grad, res.grad, weight.grad, norm.grad, *codes]

    plain = run(p["x"], p["res"], p["weight"], p["norm"])
    for got, want in zip(run(turn["x"], turn["res"], turn["weight"], wide), plain):
        assert torch.equal(got, want)
    one = p["x"][:1].expand(T, K)
    for got, want in zip(run(one, one, p["weight"][:1].expand(T, TOP), p["norm"]),
                         run(one.contiguous(), one.contiguous(), p["weight"][:1].repeat(T, 1), p["norm"])):
        assert torch.equal(got, want)


def test_no_columns_are_refused(ex):
    """By the library's own error, whichever function."""
    from communication_gemm_amd import AggError
    x, codes = (torch.empty(4, 0, dtype=t, device="cuda") for t in (torch.bfloat16, torch.uint8))
    for call in (lambda: ex.rms_norm(x), lambda: ex.rms_norm_fp8(x), lambda: ex.quantize_mxfp4(x),
                 lambda: ex.dequantize_mxfp4(codes, codes), lambda: ex.quantize(x)):
        with pytest.raises(AggError):
            call()
