"""Every kernel of the expert products on the GPU, at sizes that choose it
(tests/expert_kernels.py; tests/test_expert_choice.py checks the choice): group
ends inside, at and just past tiles, cut and half tiles, several rounds, wide
and narrow strips, and each output type.

Inputs are whole numbers so small that every partial sum is exact in fp32 and
no fp8 product is cut off, so each output has one right value.
"""
import pytest

from expert_kernels import CUS, GROUPED, WGRAD

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


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


def offsets_of(counts):
    return torch.tensor([0] + list(counts), device="cuda").cumsum(0).to(torch.int32)


def filled(shape, out):
    """An output that holds NaN, inside a buffer whose ends must stay as they are."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 512,), float("nan"), dtype=DT[out], device="cuda")
    buf[:256] = 7.0
    buf[-256:] = 7.0
    return buf[256:-256].view(shape), buf


def check(got, want, out, buf, *what):
    assert torch.equal(got, want.to(DT[out])), what
    assert (buf[:256] == 7.0).all() and (buf[-256:] == 7.0).all(), what


CASES = [(n, K) for n, c in GROUPED.items() for K in c["K"]]


def test_the_device_has_the_compute_units_the_cases_are_made_for():
    assert torch.cuda.get_device_properties(0).multi_processor_count == CUS


@pytest.mark.parametrize("name,K", CASES)
@pytest.mark.parametrize("trans", [False, True])
def test_grouped_16_bit(agg, name, K, trans):
    counts, N = GROUPED[name]["counts"], GROUPED[name]["N"]
    T, E = sum(counts), len(counts)
    x, w = whole(1, T, K), whole(2, E, *((N, K) if trans else (K, N)))
    want = torch.cat([a @ (m.t() if trans else m) for a, m in zip(x.split(counts), w)])
    off = offsets_of(counts)
    for typ in ("f16", "bf16"):
        for out in (typ, "f32"):
            y, buf = filled((T, N), out)
            agg.ag_gemm_grouped(x.to(DT[typ]), w.to(DT[typ]), off, y, trans)
            check(y, want, out, buf, typ, out)


@pytest.mark.parametrize("name,K", CASES)
def test_fp8(agg, name, K):
    counts, N = GROUPED[name]["counts"], GROUPED[name]["N"]
    T, E, kb, nb = sum(counts), len(counts), -(-K // 128), -(-N // 128)
    a, b = whole(3, T, K), whole(4, E, N, K)
    sa, sb = 2.0 ** whole(5, T, kb, top=2), 2.0 ** whole(6, E, nb, kb, top=2)
    da = a * sa.repeat_interleave(128, 1)[:, :K]
    want = torch.cat([m @ (q * s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).t()
                      for m, q, s in zip(da.split(counts), b, sb)])
    a8, b8 = (t.float().to(torch.float8_e4m3fn) for t in (a, b))
    off = offsets_of(counts)
    for out in ("bf16", "f16", "f32"):
        c, buf = filled((T, N), out)
        if E == 1:
            agg.ag_gemm_fp8_block(a8, sa.float(), b8[0], sb[0].float(), c)
        else:
            agg.ag_gemm_grouped_fp8_block(a8, sa.float(), b8, sb.float(), off, c)
        check(c, want, out, buf, out)


@pytest.mark.parametrize("name", list(WGRAD))
def test_wgrad(agg, name):
    counts, K, N = (WGRAD[name][k] for k in ("counts", "K", "N"))
    T, E = sum(counts), len(counts)
    x, dy = whole(7, T, K), whole(8, T, N)
    want = torch.stack([a.t() @ b for a, b in zip(x.split(counts), dy.split(counts))])
    for typ in ("f16", "bf16"):
        for out in (typ, "f32"):
            dw, buf = filled((E, K, N), out)
            agg.ag_gemm_grouped_wgrad(x.to(DT[typ]), dy.to(DT[typ]), offsets_of(counts), dw)
            check(dw, want, out, buf, typ, out)
