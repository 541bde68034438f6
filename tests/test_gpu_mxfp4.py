"""Microscaled 4-bit values: codes bit by bit against the format's definition,
products of few-bit values exactly, and ordinary ones against 64-bit sums."""
import pytest

from mx_kernels import PRODUCTS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


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


def values(q, scale):
    """64-bit values of packed codes and scales."""
    t = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=q.device)
    v = torch.stack([t[(q & 15).long()], t[(q >> 4).long()]], -1).flatten(-2)
    s = torch.exp2(scale.double() - 127)
    s[scale == 255] = float("nan")
    return v * s.repeat_interleave(32, -1)[..., :v.shape[-1]]


def quantised(x):
    """Codes and scales by the definition, in 64 bits."""
    m, k = x.shape
    kb = -(-k // 32)
    p = torch.nn.functional.pad(x.double(), (0, kb * 32 - k)).view(m, kb, 32)
    amax = p.abs().amax(2)
    e = torch.frexp(amax).exponent.double() - 3          # floor(log2) - 2
    e = torch.where(amax == 0, -127.0, e.clamp_min(-127.0))
    bad = ~p.isfinite().all(2)
    v = torch.where(bad[:, :, None], 0.0, p / torch.exp2(torch.where(bad, 0.0, e))[:, :, None])
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    a = v.abs().clamp_max(6.0).contiguous()
    hi = torch.searchsorted(levels, a).clamp_max(7)
    lo = (hi - 1).clamp_min(0)
    up, down = levels[hi] - a, a - levels[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(bad[:, :, None], 0, code + 8 * torch.signbit(v)).view(m, -1)[:, :k].to(torch.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, torch.where(bad, 255.0, e + 127).to(torch.uint8)


def same(a, b):
    """Equal values, NaN in the same places (fp16 draws past 65504 make blocks of NaN)."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def library_quant(agg, x, pad=0):
    m, k = x.shape
    q = torch.zeros(m, k // 2 + pad, dtype=torch.uint8, device="cuda")[:, :k // 2]
    s = torch.zeros(m, -(-k // 32) + pad, dtype=torch.uint8, device="cuda")[:, :-(-k // 32)]
    agg.ag_gemm_quant_mxfp4(x, q, s)
    return q, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,pad", [(1, 2, 0), (1, 32, 0), (3, 30, 1), (5, 64, 8), (33, 1544, 0), (70, 4096, 4),
                                     (2, 34, 3), (700, 520, 0), (9, 7168, 0)])
def test_codes(agg, dtype, M, K, pad):
    x = torch.randn(M, K + pad, generator=gen(M), device="cuda")
    x = (x * torch.exp(3 * torch.randn(M, K + pad, generator=gen(1), device="cuda"))).to(dtype)[:, :K]
    q, s = library_quant(agg, x, pad)
    want_q, want_s = quantised(x)
    assert torch.equal(s, want_s) and torch.equal(q, want_q)
    for out in TYPES:
        y = torch.full((M, K + pad), 9., device="cuda").to(out)
        agg.ag_gemm_dequant_mxfp4(q, s, y[:, :K])
        assert same(y[:, :K], values(q, s).to(out)) and (y[:, K:] == 9).all()


def test_every_tie_and_sign(agg):
    """All multiples of 1/8 up to 8 and their neighbours, both signs, beside a 4
    that fixes the scale at 1; then the same 2^-100 and 2^100 times."""
    v = torch.arange(0, 64, device="cuda") / 8.0
    v = torch.cat([v, torch.nextafter(v, v + 1), torch.nextafter(v, v - 1)])
    v = torch.cat([v, -v])
    x = torch.zeros(len(v), 32, device="cuda")
    x[:, 0], x[:, 1], x[:, 31] = 4, v, -v
    for f in (1.0, 2.0 ** -100, 2.0 ** 100):
        q, s = library_quant(agg, x * f)
        want_q, want_s = quantised(x * f)
        assert torch.equal(q, want_q) and torch.equal(s, want_s)


def test_ends_of_the_scales(agg):
    """Subnormal blocks (scale 2^-127), the largest values, zeros, infinities, NaN."""
    x = torch.zeros(9, 64, device="cuda")
    x[0, 3] = 2.0 ** -149
    x[1, 3] = 2.0 ** -126
    x[2, :32] = torch.arange(32, device="cuda") * 2.0 ** -128
    x[3, 3] = 3.4e38
    x[4, 40] = float("inf")
    x[5, 0] = -float("inf")
    x[6, 33] = float("nan")
    x[7] = -0.0
    x[8, :32], x[8, 32:] = 2.0 ** -125, -(2.0 ** -124)
    q, s = library_quant(agg, x)
    want_q, want_s = quantised(x)
    assert torch.equal(s, want_s) and torch.equal(q, want_q)
    assert s[4].tolist() == [0, 255] and s[5].tolist() == [255, 0] and s[6].tolist() == [0, 255]
    y = torch.empty_like(x)
    agg.ag_gemm_dequant_mxfp4(q, s, y)
    assert same(y, values(q, s).float())


# ---- products ----------------------------------------------------------------


def codes(seed, *shape, lo=126, hi=128, pad=0, scale_pad=0, scale_at=0):
    """Random codes [..., K] with scales in [lo, hi] as rows of wider matrices, the
    scales from column scale_at on."""
    *lead, k = shape
    kb = -(-k // 32)
    q = torch.randint(0, 256, (*lead, k // 2 + pad), generator=gen(seed), device="cuda").to(torch.uint8)
    s = torch.randint(lo, hi + 1, (*lead, scale_at + kb + scale_pad), generator=gen(seed + 1),
                      device="cuda").to(torch.uint8)
    return q[..., :k // 2], s[..., scale_at:scale_at + kb]


def groups(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def product(a, b, counts):
    """64-bit products by group (b [E, N, K])."""
    parts, at = [], 0
    for e, c in enumerate(counts):
        parts.append(a[at:at + c] @ b[e].t().contiguous())
        at += c
    return torch.cat(parts)


CALLS = [(name, K) for name, c in PRODUCTS.items() for K in c["K"]]


@pytest.mark.parametrize("name,K", CALLS)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("tidy", [True, False, "but for the scales", "but for c"])
def test_products_of_few_bits_are_exact(agg, name, K, out, tidy):
    """Products are multiples of 2^-2, at most 36, times scales of 2^-2 .. 2^2: sums
    of up to 7168 are below 2^24 of their step of 2^-4, so every sum is exact in
    float32 and rounds once.  tidy: the kernel that the call names, with rows of
    scales on dwords or at odd strides from an odd start, and rows of c in pieces of 16
    bytes or of any number of columns (large: 128 x 128); otherwise the one for every
    layout."""
    counts, N = PRODUCTS[name]["counts"], PRODUCTS[name]["N"]
    if tidy is False:
        if sum(counts) * N * K > 2 ** 31:
            counts = counts[:1]
        K = max(K - 6, 2)
    if tidy in (False, "but for c"):
        N -= 3
    T, E = sum(counts), len(counts)
    kb = -(-K // 32)
    pad = 32 if tidy else 5
    if tidy in (True, "but for c"):     # strides: multiples of 4
        pa = pb = dict(scale_pad=-kb % 4)
    elif tidy:                          # 1 and 3 more
        pa, pb = dict(scale_pad=(-kb - 2) % 4, scale_at=3), dict(scale_pad=(-kb + 2) % 4, scale_at=1)
    else:
        pa = pb = dict(scale_pad=1)
    a, sa = codes(1, T, K, pad=pad, **pa)
    b, sb = codes(3, E, N, K, pad=pad, **pb)
    want = product(values(a, sa), values(b, sb), counts)
    c = torch.full((T + 2, N + (8 if tidy not in (False, "but for c") else 1)), 9., device="cuda").to(out)
    if E == 1:
        agg.ag_gemm_mxfp4(a, sa, b[0], sb[0], c[:T, :N])
    else:
        agg.ag_gemm_grouped_mxfp4(a, sa, b, sb, groups(counts), c[:T, :N])
    assert torch.equal(c[:T, :N].double(), want.to(out).double())
    assert (c[T:] == 9).all() and (c[:, N:] == 9).all()


@pytest.mark.parametrize("counts", [[1], [40], [3, 0, 90]])
@pytest.mark.parametrize("N", [1, 2, 5, 61])
@pytest.mark.parametrize("out", TYPES)
def test_few_columns(agg, counts, N, out):
    T, E, K = sum(counts), len(counts), 1056
    a, sa = codes(39, T, K)
    b, sb = codes(41, E, N, K)
    c = torch.full((T + 1, N), 9., device="cuda").to(out)
    agg.ag_gemm_grouped_mxfp4(a, sa, b, sb, groups(counts), c[:T])
    want = product(values(a, sa), values(b, sb), counts)
    assert torch.equal(c[:T].double(), want.to(out).double()) and (c[T:] == 9).all()


@pytest.mark.parametrize("counts,K,N", [([5], 7168, 264), ([300], 4096, 520), ([100, 0, 171], 1056, 328),
                                        ([1024, 700], 2048, 1288), ([64], 7168, 4088), ([200], 4096, 2056),
                                        ([300], 4096, 2568), ([500], 4096, 2056)])
def test_scales_far_apart(agg, counts, K, N):
    """Scales of 2^-20 .. 2^20 each: against 64 bits within the roundings of a
    float32 sum of K products, K u of the sum of magnitudes."""
    T, E = sum(counts), len(counts)
    a, sa = codes(5, T, K, lo=107, hi=147)
    b, sb = codes(7, E, N, K, lo=107, hi=147)
    va, vb = values(a, sa), values(b, sb)
    want, mags = product(va, vb, counts), product(va.abs(), vb.abs(), counts)
    c = torch.empty(T, N, device="cuda")
    agg.ag_gemm_grouped_mxfp4(a, sa, b, sb, groups(counts), c)
    assert ((c.double() - want).abs() <= K * 2.0 ** -24 * mags).all()


FAR = [(name, min(k for k in c["K"] if k >= 256)) for name, c in PRODUCTS.items() if max(c["K"]) >= 256]


def multiply(agg, a, sa, b, sb, counts):
    c = torch.empty(sum(counts), b.shape[1], device="cuda")
    if len(counts) == 1:
        return agg.ag_gemm_mxfp4(a, sa, b[0], sb[0], c)
    return agg.ag_gemm_grouped_mxfp4(a, sa, b, sb, groups(counts), c)


@pytest.mark.parametrize("name,K", FAR)
def test_single_products_far_apart_are_joined_exactly(agg, name, K):
    """1, and a power of two 2^-1 .. 2^-22 of either sign in another block of the
    same 256 (one instruction joins two or four of those), at every distance and
    pair of blocks in turn: float32 holds their sum, so the result equals it.  An
    instruction that cut at 13 bits, as E4M3's does, would lose the second."""
    counts, N = PRODUCTS[name]["counts"], PRODUCTS[name]["N"]
    T, E, kb = sum(counts), len(counts), K // 32
    t = torch.arange(T, device="cuda")
    base = torch.randint(0, kb // 8, (T,), generator=gen(51), device="cuda") * 8
    first = torch.randint(0, 8, (T,), generator=gen(52), device="cuda")
    second = (first + 1 + torch.randint(0, 7, (T,), generator=gen(53), device="cuda")) % 8
    at = torch.randint(0, 32, (2, T), generator=gen(54), device="cuda")
    code = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    code[t, (base + first) * 32 + at[0]] = 2
    code[t, (base + second) * 32 + at[1]] = (2 + 8 * (t % 2)).to(torch.uint8)
    sa = torch.full((T, kb), 127, dtype=torch.uint8, device="cuda")
    d = 1 + (t + 5 * (t // 22)) % 22
    sa[t, base + second] = (127 - d).to(torch.uint8)
    a = code[:, 0::2] | code[:, 1::2] << 4
    b = torch.full((E, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    sb = torch.full((E, N, kb), 127, dtype=torch.uint8, device="cuda")
    c = multiply(agg, a, sa, b, sb, counts)
    want = 1 + torch.where(t % 2 == 0, 1.0, -1.0).double() * torch.exp2(-d.double())
    assert torch.equal(c.double(), want[:, None].expand(T, N))


@pytest.mark.parametrize("name,K", FAR)
def test_blocks_far_apart_are_joined_exactly(agg, name, K):
    """Rows of two blocks of random codes among zeros, one's scales 2^-8 of the
    other's, b's 2^-1 .. 2^1: products are multiples of 2^-2, blocks at most 32 * 36,
    so a sum is below 2^12 and a multiple of 2^-11: 23 bits."""
    counts, N = PRODUCTS[name]["counts"], PRODUCTS[name]["N"]
    T, E, kb = sum(counts), len(counts), K // 32
    t = torch.arange(T, device="cuda")
    first = torch.randint(0, kb // 8 * 8, (T,), generator=gen(55), device="cuda")
    second = first ^ (1 + t % 7)
    a, sa = codes(56, T, K, lo=120, hi=134)
    keep = torch.zeros(T, kb, dtype=torch.bool, device="cuda")
    keep[t, first] = keep[t, second] = True
    a = torch.where(keep.repeat_interleave(16, 1), a, 0)
    sa[t, first] = 127
    sa[t, second] = 119
    b, sb = codes(57, E, N, K, lo=126, hi=128)
    c = multiply(agg, a, sa, b, sb, counts)
    assert torch.equal(c.double(), product(values(a, sa), values(b, sb), counts))


@pytest.mark.parametrize("counts,N", [([3], 72), ([200], 328), ([700, 400], 1288), ([200], 2056), ([300], 2568),
                                      ([500], 2056)])
@pytest.mark.parametrize("K", [64, 160, 288, 4128])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_what_stands_behind_a_row_is_not_read(agg, counts, N, K, at):
    """Scales of 255 (NaN) and codes behind each row's end, rows of no group
    with NaN scales, and rows of c outside the groups: none of it matters."""
    T, E, kb = sum(counts), len(counts), K // 32
    a, sa = codes(9, T + 5, K, pad=64, scale_pad=8, scale_at=at)
    b, sb = codes(11, E, N, K, pad=64, scale_pad=8, scale_at=3 * at)
    for s in (sa, sb):
        kept = s.clone()
        s._base.fill_(255)
        s.copy_(kept)
    sa[:2] = 255
    sa[T + 2:] = 255
    off = groups(counts) + 2
    c = torch.full((T + 5, N), 9., device="cuda")
    agg.ag_gemm_grouped_mxfp4(a, sa, b, sb, off, c)
    want = product(values(a, sa)[2:T + 2], values(b, sb), counts)
    assert torch.equal(c[2:T + 2].double(), want) and (c[:2] == 9).all() and (c[T + 2:] == 9).all()


@pytest.mark.parametrize("K", [544, 4128])
def test_a_scale_of_nan_reaches_its_row_only(agg, K):
    for counts, N in (([5], 264), ([300], 520), ([1000], 2056), ([200], 2056), ([300], 2568), ([500], 2056)):
        T = sum(counts)
        a, sa = codes(13, T, K)
        b, sb = codes(15, 1, N, K)
        sa[1, 3] = 255
        sb[0, 7, 16] = 255
        c = torch.empty(T, N, device="cuda")
        agg.ag_gemm_mxfp4(a, sa, b[0], sb[0], c)
        bad = c.isnan()
        assert bad[1].all() and bad[:, 7].all()
        bad[1] = bad[:, 7] = False
        assert not bad.any()


def test_float4_and_e8m0_types(agg):
    if not hasattr(torch, "float4_e2m1fn_x2"):
        pytest.skip("no such types")
    a, sa = codes(17, 9, 64)
    b, sb = codes(19, 24, 64)
    c, d = torch.empty(9, 24, device="cuda"), torch.empty(9, 24, device="cuda")
    agg.ag_gemm_mxfp4(a, sa, b, sb, c)
    agg.ag_gemm_mxfp4(a.view(torch.float4_e2m1fn_x2), sa.view(torch.float8_e8m0fnu),
                      b.view(torch.float4_e2m1fn_x2), sb.view(torch.float8_e8m0fnu), d)
    assert torch.equal(c, d)


def test_equal_calls_give_equal_bits(agg):
    a, sa = codes(21, 1000, 2048, lo=100, hi=150)
    b, sb = codes(23, 1544, 2048, lo=100, hi=150)
    c = [torch.empty(1000, 1544, device="cuda") for _ in range(3)]
    for t in c:
        agg.ag_gemm_mxfp4(a, sa, b, sb, t)
    assert torch.equal(c[0], c[1]) and torch.equal(c[0], c[2])


@pytest.mark.parametrize("rows", [3, 300])
def test_operands_past_32_bit_offsets(agg, rows):
    """The last expert of more than 2^32 bytes of codes; the last rows of as many."""
    K, N = 8192, 4104
    E = (1 << 32) // (K // 2 * N) + 2
    b = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    sb = torch.zeros(E, N, K // 32, dtype=torch.uint8, device="cuda")
    b[-1:], sb[-1:] = codes(25, 1, N, K)
    T = (1 << 32) // (K // 2) + 9
    a = torch.zeros(T, K // 2, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(T, K // 32, dtype=torch.uint8, device="cuda")
    a[T - rows:], sa[T - rows:] = codes(27, rows, K)
    off = torch.full((E + 1,), T - rows, dtype=torch.int32, device="cuda")
    off[-1] = T
    c = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    agg.ag_gemm_grouped_mxfp4(a, sa, b, sb, off, c)
    want = values(a[T - rows:], sa[T - rows:]) @ values(b[-1], sb[-1]).t().contiguous()
    assert torch.equal(c[T - rows:].double(), want.to(torch.bfloat16).double())


def test_layer_functions(agg):
    """quantize_mxfp4 of stacks, the products on them, zeros in rows of no group,
    and a gradient that is refused."""
    from communication_gemm_amd import experts as ex
    w = torch.randn(3, 40, 160, generator=gen(29), device="cuda").bfloat16()
    wq, ws = ex.quantize_mxfp4(w)
    assert wq.shape == (3, 40, 80) and ws.shape == (3, 40, 5) and ws.stride(-2) % 4 == 0
    for e in range(3):
        want = quantised(w[e])
        assert torch.equal(wq[e], want[0]) and torch.equal(ws[e], want[1])
    assert torch.equal(ex.dequantize_mxfp4(wq, ws, torch.float32).double(), values(wq, ws))
    x = torch.randn(20, 160, generator=gen(30), device="cuda").bfloat16()
    xq, xs = ex.quantize_mxfp4(x)
    off = torch.tensor([1, 5, 5, 18], dtype=torch.int32, device="cuda")
    torch.full((20, 40), float("nan"), device="cuda")        # the allocator's next block
    y = ex.grouped_linear_mxfp4(x, wq, ws, off, torch.float32, padded=True)
    va, vb = values(xq, xs), values(wq, ws)
    want = torch.zeros(20, 40, dtype=torch.float64, device="cuda")
    want[1:5], want[5:18] = va[1:5] @ vb[0].t().contiguous(), va[5:18] @ vb[2].t().contiguous()
    mags = va.abs().sum(1, keepdim=True) * vb.abs().amax()
    assert ((y.double() - want).abs() <= 160 * 2.0 ** -24 * mags).all() and (y[0] == 0).all() and (y[18:] == 0).all()
    y = ex.linear_mxfp4(x, wq[1], ws[1])
    want = va @ vb[1].t().contiguous()
    # bf16 keeps 8 bits: half a step is up to 2^-8 of the value
    assert y.dtype == x.dtype and ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 160 * 2.0 ** -24 * mags).all()
    for call in (lambda t: ex.linear_mxfp4(t, wq[0], ws[0]), lambda t: ex.grouped_linear_mxfp4(t, wq, ws, off)):
        with pytest.raises(RuntimeError, match="no gradient"):
            call(x.clone().requires_grad_()).sum().backward()


@pytest.mark.parametrize("K", [160, 4128])
def test_one_row_of_odd_many_scales(agg, K):
    """A single row's scales need no stride, and what stands behind them is not used."""
    kb = K // 32
    a, sa = codes(33, 1, K)
    b, sb = codes(35, 72, K, scale_pad=-kb % 4)
    behind = torch.full((kb + 8,), 255, dtype=torch.uint8, device="cuda")
    behind[:kb] = sa[0]
    c = torch.empty(1, 72, device="cuda")
    agg.ag_gemm_mxfp4(a, behind[None, :kb], b, sb, c)
    assert torch.equal(c.double(), values(a, sa) @ values(b, sb).t().contiguous())


def test_no_rows_and_transposed_rows(agg):
    from communication_gemm_amd import experts as ex
    x = torch.randn(160, 24, generator=gen(37), device="cuda")
    q, s = ex.quantize_mxfp4(x.t())
    want = quantised(x.t().contiguous())
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
    for lead in ((0,), (2, 0)):
        q, s = ex.quantize_mxfp4(torch.empty(*lead, 160, device="cuda"))
        assert q.shape == (*lead, 80) and s.shape == (*lead, 5)
        assert ex.dequantize_mxfp4(q, s).shape == (*lead, 160)
    wq, ws = ex.quantize_mxfp4(torch.randn(40, 160, device="cuda"))
    assert ex.linear_mxfp4(torch.empty(0, 160, device="cuda"), wq, ws).shape == (0, 40)


def test_captured_chain(agg):
    """Quantise, multiply and dequantise in a graph, replayed with other inputs."""
    x = torch.zeros(40, 320, dtype=torch.bfloat16, device="cuda")
    b, sb = codes(31, 136, 320)
    q, s = torch.empty(40, 160, dtype=torch.uint8, device="cuda"), torch.empty(40, 12, dtype=torch.uint8, device="cuda")[:, :10]
    c, y = torch.empty(40, 136, device="cuda"), torch.empty_like(x)

    def work():
        agg.ag_gemm_quant_mxfp4(x, q, s)
        agg.ag_gemm_mxfp4(q, s, b, sb, c)
        agg.ag_gemm_dequant_mxfp4(q, s, y)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in range(4):
        x.copy_(torch.randn(40, 320, generator=gen(40 + seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, s, c, y)]
        for t in (q, s, c, y):
            t.fill_(1)
        work()
        assert all(torch.equal(a, b_) for a, b_ in zip(got, (q, s, c, y)))
