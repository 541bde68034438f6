"""The operators around the expert products on more rows than one launch has
workgroups for, and on rows that stand 2^32 bytes and more apart."""
import pytest

from test_gpu_mxfp4 import quantised, same, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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


# 8192 workgroups take 524288 blocks of 32 in a pass, and 2097152 eights of columns
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,pad", [(2500, 7168, 0), (2500, 7170, 1), (530000, 32, 0), (2100000, 8, 8)])
def test_quantiser_and_back_in_several_passes(agg, dtype, M, K, pad):
    x = (torch.randn(M, K + pad, generator=gen(M), device="cuda") *
         torch.exp(2 * torch.randn(K + pad, generator=gen(1), device="cuda"))).to(dtype)[:, :K]
    q = torch.full((M, K // 2 + pad), 0x77, dtype=torch.uint8, device="cuda")
    s = torch.full((M, -(-K // 32) + pad), 9, dtype=torch.uint8, device="cuda")
    q_, s_ = q[:, :K // 2], s[:, :-(-K // 32)]
    agg.ag_gemm_quant_mxfp4(x, q_, s_)
    want = quantised(x)
    assert torch.equal(q_, want[0]) and torch.equal(s_, want[1])
    assert (q[:, K // 2:] == 0x77).all() and (s[:, -(-K // 32):] == 9).all()
    y = torch.full((M, K + pad), 9., dtype=dtype, device="cuda")
    agg.ag_gemm_dequant_mxfp4(q_, s_, y[:, :K])
    assert same(y[:, :K], values(q_, s_).to(dtype)) and (y[:, K:] == 9).all()


@pytest.mark.parametrize("K", [64, 62])
def test_quantiser_and_back_past_32_bit_offsets(agg, K):
    """Every row of x, codes, scales and y 2^21 elements behind the last."""
    M, ld = (1 << 32) // (1 << 21) + 3, 1 << 21
    x, y = (torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")[:, :K] for _ in range(2))
    q = torch.empty(M, ld, dtype=torch.uint8, device="cuda")[:, :K // 2]
    s = torch.empty(M, ld, dtype=torch.uint8, device="cuda")[:, :2]
    x.copy_(torch.randn(M, K, generator=gen(2), device="cuda"))
    agg.ag_gemm_quant_mxfp4(x, q, s)
    want = quantised(x)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
    agg.ag_gemm_dequant_mxfp4(q, s, y)
    assert same(y, values(q, s).bfloat16())


# a launch has 2^21 workgroups at most, a row each
@pytest.mark.parametrize("K", [8, 7])
def test_norm_of_many_rows(agg, K):
    """All rows, the second pass' too; the sums are of K values: (K / 2 + 8) u
    before the rounding."""
    T = (1 << 21) + 300
    x = torch.randn(T, K, generator=gen(3), device="cuda").bfloat16()
    res = torch.randn(T, K, generator=gen(4), device="cuda").bfloat16()
    w = (1 + torch.randn(K, generator=gen(5), device="cuda") / 4).bfloat16()
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    q, scale = torch.empty(T, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, 1, device="cuda")
    agg.ag_gemm_rmsnorm(x, w, y=y, q=q, scale=scale, residual=res, h=h, rstd=rstd, eps=1e-5)
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    hd = h.double()
    r = (hd.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    want = hd * r * w.double()
    rel = (K / 2 + 8) * U
    assert ((rstd.double() - r[:, 0]).abs() <= rel * r[:, 0]).all()
    assert ((y.double() - want).abs() <= (2.0 ** -8 + rel) * want.abs()).all()
    amax = want.abs().amax(1, keepdim=True)
    assert ((scale.double() - amax / 448).abs() <= (rel + 4 * U) * amax / 448).all()
    codes = q.double() * scale.double()
    assert ((codes - want).abs() <= (2.0 ** -4 + 2 * rel) * want.abs() + 2.0 ** -10 * scale.double() * (1 + rel)).all()


# 2^23 workgroups at most, a token each
@pytest.mark.parametrize("K", [8, 3])
def test_tokens_in_two_passes(agg, K):
    """Values of few bits, so that all of it is exact."""
    T = (1 << 23) + 300
    x = torch.randint(-8, 9, (T, K), generator=gen(6), device="cuda").float()
    place = torch.randperm(T, generator=gen(7), device="cuda").to(torch.int32).view(T, 1)
    place[::1001] = -1
    has = place[:, 0] >= 0
    at = place[has, 0].long()
    xs = torch.full((T, K), 99., device="cuda")
    agg.ag_gemm_expert_dispatch(x, place, xs)
    want = torch.full_like(xs, 99)
    want[at] = x[has]
    assert torch.equal(xs, want)
    w = torch.randint(-4, 5, (T, 1), generator=gen(8), device="cuda") / 4
    y = agg.ag_gemm_expert_combine(xs, place, w, torch.empty_like(x))
    assert torch.equal(y, torch.where(has[:, None], x * w, 0.0))
    dh, dw = torch.full_like(xs, 99), torch.empty_like(w)
    agg.ag_gemm_expert_combine_grad(x, xs, place, w, dh, dw)
    want[at] = (x * w)[has]
    assert torch.equal(dh, want) and torch.equal(dw[:, 0], torch.where(has, x.square().sum(1), 0.0))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_of_many(agg, dtype):
    """Chunks of several passes a workgroup."""
    T, top, E = 4000003, 3, 100
    ids = torch.randint(-1, E + 1, (T, top), generator=gen(9), device="cuda").to(dtype)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    place = torch.empty(T, top, dtype=torch.int32, device="cuda")
    ws = torch.empty(agg.expert_sort_workspace_bytes(T, top, E), dtype=torch.uint8, device="cuda")
    agg.ag_gemm_expert_sort(ids, E, off, place, ws)
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    want = torch.empty_like(order)
    want[order] = torch.arange(len(order), device="cuda")
    assert torch.equal(place.flatten().long(), torch.where(key < E, want, -1))
    assert torch.equal(off.long(), torch.bincount(key, minlength=E + 1).cumsum(0).roll(1) * (
        torch.arange(E + 1, device="cuda") > 0))
