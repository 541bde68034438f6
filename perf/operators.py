"""What the expert-product operators are measured on: their cases, inputs,
plain forms and 64-bit definitions.

Four operators, used together by a layer of experts whose tokens are sorted
by expert (``offsets[e] .. offsets[e + 1]`` are the rows of expert e):

``grouped``   y[r] = x[r] @ w[e(r)]            16-bit in; also the input gradient
``wgrad``     dw[e] = x[rows of e]^T @ dy[rows of e]
``fp8``       y = (a * sa) @ (b * sb)^T        E4M3 with a float32 scale for each 128
                                               of k (a: for each row; b: for each 128
                                               rows), dense (experts = 0) or by expert
``quant``     q, scale of a 16-bit matrix      the fp8 form's inputs

Where ``own`` is false, ``run`` computes the plain form in 32 bits with
elementary torch operations; where it is true, it calls the library.
"""
import math
import random

import torch

own = False

BLOCK = 128           # k (and, for weights, rows) that one fp8 scale covers
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of two sequences, eight experts each, out of 64: latency
        {"name": "decode, 16 rows", "op": "grouped", "rows": 16, "experts": 64, "k": 2048,
         "n": 1024, "type": "bf16", "out": "bf16", "trans": False, "route": 1, "skew": 0.0},
        # a decoding batch over 32 experts, weights stored output channel by output channel
        {"name": "decode, 100 rows, trans", "op": "grouped", "rows": 100, "experts": 32, "k": 4096,
         "n": 2048, "type": "f16", "out": "f16", "trans": True, "route": 2, "skew": 0.5},
        # a short prompt: ragged groups of some tens of rows, some empty
        {"name": "prompt, 1001 rows", "op": "grouped", "rows": 1001, "experts": 24, "k": 2056,
         "n": 1544, "type": "bf16", "out": "bf16", "trans": False, "route": 3, "skew": 1.0},
        # a training step's forward product
        {"name": "train forward", "op": "grouped", "rows": 16384, "experts": 8, "k": 4096,
         "n": 4096, "type": "bf16", "out": "bf16", "trans": False, "route": 4, "skew": 0.3},
        # its input gradient: dy @ w^T, weights as the forward pass stores them
        {"name": "train input gradient", "op": "grouped", "rows": 8191, "experts": 16, "k": 2048,
         "n": 4096, "type": "bf16", "out": "bf16", "trans": True, "route": 5, "skew": 0.5},
        # its weight gradient, kept in 32 bits for accumulation over steps
        {"name": "train weight gradient", "op": "wgrad", "rows": 16384, "experts": 8, "k": 4096,
         "n": 2048, "type": "bf16", "out": "f32", "route": 6, "skew": 0.3},
        # a small step: short ragged reductions, some of them empty
        {"name": "weight gradient, 777 rows", "op": "wgrad", "rows": 777, "experts": 20, "k": 1024,
         "n": 1544, "type": "f16", "out": "f16", "route": 7, "skew": 1.0},
        # a dense fp8 layer for a few decoding rows: bound by the weights' bytes
        {"name": "fp8 decode, 5 rows", "op": "fp8", "rows": 5, "experts": 0, "k": 7168,
         "n": 4096, "out": "bf16", "route": 8, "skew": 0.0},
        # the same kind of layer on a long prompt: bound by the matrix cores
        {"name": "fp8 prompt, 8192 rows", "op": "fp8", "rows": 8192, "experts": 0, "k": 4096,
         "n": 4096, "out": "bf16", "route": 9, "skew": 0.0},
        # experts in fp8 on a middling batch
        {"name": "fp8 experts, 3001 rows", "op": "fp8", "rows": 3001, "experts": 32, "k": 2048,
         "n": 2816, "out": "bf16", "route": 10, "skew": 0.7},
        # activations before an fp8 product: a decoding batch, and a long prompt
        {"name": "quantise, 33 rows", "op": "quant", "rows": 33, "k": 4096, "type": "bf16",
         "block_rows": 1},
        {"name": "quantise, 8192 rows", "op": "quant", "rows": 8192, "k": 7168, "type": "bf16",
         "block_rows": 1},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, step * round(v / step)))


def _drawn(rng):
    op = rng.choice(["grouped", "grouped", "wgrad", "fp8", "fp8", "quant"])
    typ = rng.choice(["bf16", "f16"])
    route = rng.randrange(1, 1 << 30)
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 16384), "k": _log(rng, 512, 8192, 8), "type": typ,
                "block_rows": rng.choice([1, 1, 128])}
    if op == "wgrad":
        return {"op": op, "rows": _log(rng, 256, 16384), "experts": _log(rng, 4, 32),
                "k": _log(rng, 512, 4096, 8), "n": _log(rng, 512, 4096, 8), "type": typ,
                "out": rng.choice([typ, "f32"]), "route": route, "skew": rng.choice([0.0, 0.5, 1.0])}
    if op == "fp8":
        return {"op": op, "rows": _log(rng, 1, 16384), "experts": rng.choice([0, _log(rng, 4, 64)]),
                "k": _log(rng, 512, 7168, 16), "n": _log(rng, 512, 4096, 8),
                "out": rng.choice(["bf16", "f16", "f32"]), "route": route,
                "skew": rng.choice([0.0, 0.5, 1.0])}
    return {"op": op, "rows": _log(rng, 1, 16384), "experts": _log(rng, 4, 64),
            "k": _log(rng, 512, 4096, 8), "n": _log(rng, 512, 4096, 8), "type": typ, "out": typ,
            "trans": rng.random() < 0.5, "route": route, "skew": rng.choice([0.0, 0.5, 1.0])}


def draw(rng):
    """A case of the same ranges that moves and computes no more than the largest listed one."""
    top = [work(c) for c in listed()]
    while True:
        c = _drawn(rng)
        w = work(c)
        if w["flops"] <= max(t["flops"] for t in top) and w["bytes"] <= max(t["bytes"] for t in top):
            return c


def sizes(case):
    """Rows of each expert: every row picks one, with weights exp(skew * normal)."""
    if not case.get("experts"):
        return [case["rows"]]
    rng = random.Random(case["route"])
    weights = [math.exp(case["skew"] * rng.gauss(0.0, 1.0)) for _ in range(case["experts"])]
    got = [0] * case["experts"]
    for e in rng.choices(range(case["experts"]), weights, k=case["rows"]):
        got[e] += 1
    return got


def _starts(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _quantised(x, block_rows):
    """E4M3 codes of x and their float32 scales, one for each block_rows x 128 block
    (the last ones along each axis may be partial)."""
    x = x.float()
    m, k = x.shape
    mb, kb = -(-m // block_rows), -(-k // BLOCK)
    p = torch.nn.functional.pad(x, (0, kb * BLOCK - k, 0, mb * block_rows - m))
    amax = p.abs().view(mb, block_rows, kb, BLOCK).amax(dim=(1, 3)).clamp_min(AMAX_FLOOR)
    inverse = torch.full_like(amax, E4M3_MAX) / amax
    each = inverse.repeat_interleave(block_rows, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return (x * each).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _dequantised(q, scale, block_rows, dtype):
    each = scale.to(dtype).repeat_interleave(block_rows, 0)[:q.shape[0]]
    return q.to(dtype) * each.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    op, rows, k = case["op"], case["rows"], case["k"]
    s = {"case": case}
    if op == "quant":
        # activations: a few channels carry much larger values than the others
        channel = torch.exp(normal(k))
        s["x"] = (normal(rows, k) * channel).to(DTYPES[case["type"]])
        s["q"] = torch.empty(rows, k, dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty(-(-rows // case["block_rows"]), -(-k // BLOCK), device="cuda")
        return s
    n, experts = case["n"], case["experts"]
    s["counts"] = sizes(case)
    s["starts"] = _starts(s["counts"])
    s["offsets"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
    if op == "wgrad":
        dtype = DTYPES[case["type"]]
        s["x"] = normal(rows, k, dtype=dtype)
        s["dy"] = normal(rows, n, scale=0.05, dtype=dtype)
        s["dw"] = torch.empty(experts, k, n, dtype=DTYPES[case["out"]], device="cuda")
        return s
    s["y"] = torch.empty(rows, n, dtype=DTYPES[case["out"]], device="cuda")
    if op == "grouped":
        dtype = DTYPES[case["type"]]
        s["x"] = normal(rows, k, dtype=dtype)
        shape = (n, k) if case["trans"] else (k, n)
        s["w"] = torch.empty(experts, *shape, dtype=dtype, device="cuda")
        for e in range(experts):
            s["w"][e] = normal(*shape, scale=k ** -0.5)
    else:
        s["a"], s["sa"] = _quantised(normal(rows, k), 1)
        e1 = max(experts, 1)
        s["b"] = torch.empty(e1, n, k, dtype=torch.float8_e4m3fn, device="cuda")
        s["sb"] = torch.empty(e1, -(-n // BLOCK), -(-k // BLOCK), device="cuda")
        for e in range(e1):
            q, sc = _quantised(normal(n, k, scale=k ** -0.5), BLOCK)
            s["b"].view(torch.uint8)[e] = q.view(torch.uint8)
            s["sb"][e] = sc
        if not experts:
            s["b"], s["sb"] = s["b"][0], s["sb"][0]
    if own and rows <= 512:
        # a decoding loop keeps its buffers and marshals its calls once
        s["call"] = _library(s, prepare=True)
    return s


def _library(s, **kw):
    """The library's call for this state."""
    import communication_gemm_amd as agg
    op = s["case"]["op"]
    if op == "quant":
        return agg.ag_gemm_quant_fp8_block(s["x"], s["q"], s["scale"], s["case"]["block_rows"], **kw)
    if op == "wgrad":
        return agg.ag_gemm_grouped_wgrad(s["x"], s["dy"], s["offsets"], s["dw"], **kw)
    if op == "grouped":
        return agg.ag_gemm_grouped(s["x"], s["w"], s["offsets"], s["y"], s["case"]["trans"], **kw)
    if s["case"]["experts"]:
        return agg.ag_gemm_grouped_fp8_block(s["a"], s["sa"], s["b"], s["sb"], s["offsets"],
                                             s["y"], **kw)
    return agg.ag_gemm_fp8_block(s["a"], s["sa"], s["b"], s["sb"], s["y"], **kw)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if "call" in s:
            s["call"]()
        else:
            _library(s)
        return [s["q"], s["scale"]] if op == "quant" else s["dw"] if op == "wgrad" else s["y"]
    return _formula(s, torch.float32)


def _formula(s, dtype):
    """The operator with elementary operations in `dtype`, rounded once at the end."""
    case = s["case"]
    op = case["op"]
    if op == "quant":
        return list(_quantised(s["x"], case["block_rows"]))
    out = DTYPES[case["out"]]
    if op == "wgrad":
        dw = torch.empty_like(s["dw"])
        for e, lo in enumerate(s["starts"][:-1]):
            hi = s["starts"][e + 1]
            dw[e] = (s["x"][lo:hi].to(dtype).t() @ s["dy"][lo:hi].to(dtype)).to(out)
        return dw
    y = torch.empty_like(s["y"])
    if op == "fp8" and not case["experts"]:
        a = _dequantised(s["a"], s["sa"], 1, dtype)
        return (a @ _dequantised(s["b"], s["sb"], BLOCK, dtype).t()).to(out)
    for e, lo in enumerate(s["starts"][:-1]):
        hi = s["starts"][e + 1]
        if lo == hi:
            continue
        if op == "grouped":
            w = s["w"][e].to(dtype)
            x = s["x"][lo:hi].to(dtype)
            y[lo:hi] = (x @ (w.t() if case["trans"] else w)).to(out)
        else:
            a = _dequantised(s["a"][lo:hi], s["sa"][lo:hi], 1, dtype)
            y[lo:hi] = (a @ _dequantised(s["b"][e], s["sb"][e], BLOCK, dtype).t()).to(out)
    return y


def _e4m3_values():
    """The non-negative finite E4M3 values in increasing order, from the format's definition."""
    got = []
    for code in range(0x7F):
        e, f = code >> 3, code & 7
        got.append(f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def exact(case, seed):
    """The definition in 64 bits, unrounded but for the values that are codes."""
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    f8 = torch.float64
    op = case["op"]
    if op == "quant":
        x, br = s["x"].to(f8), case["block_rows"]
        m, k = x.shape
        values = _e4m3_values()
        scale = torch.empty(-(-m // br), -(-k // BLOCK), dtype=f8, device="cuda")
        q = torch.empty_like(x)
        for j in range(scale.shape[1]):
            cols = x[:, j * BLOCK:(j + 1) * BLOCK]
            top = cols.abs().amax(1)
            if br > 1:
                top = torch.stack([t.max() for t in top.split(br)])
            scale[:, j] = top.clamp_min(AMAX_FLOOR) / E4M3_MAX
            v = cols / scale[:, j].repeat_interleave(br)[:m, None]
            a = v.abs().clamp_max(E4M3_MAX)
            hi = torch.searchsorted(values, a.contiguous()).clamp_max(len(values) - 1)
            lo = (hi - 1).clamp_min(0)
            up, down = values[hi] - a, a - values[lo]
            code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            q[:, j * BLOCK:(j + 1) * BLOCK] = values[code] * torch.sign(v)
        return [q, scale]
    if op == "wgrad":
        out = torch.zeros(case["experts"], case["k"], case["n"], dtype=f8, device="cuda")
        for e, (lo, c) in enumerate(zip(s["starts"], s["counts"])):
            if c:
                out[e] = torch.mm(s["x"][lo:lo + c].to(f8).t().contiguous(), s["dy"][lo:lo + c].to(f8))
        return out
    out = torch.zeros(case["rows"], case["n"], dtype=f8, device="cuda")
    for e, (lo, c) in enumerate(zip(s["starts"], s["counts"])):
        if op == "grouped":
            w = s["w"][e].to(f8)
            out[lo:lo + c] = s["x"][lo:lo + c].to(f8) @ (w if not case["trans"] else w.t().contiguous())
            continue
        # block by block of k: the sum of products, then the two scales
        b = s["b"][e] if case["experts"] else s["b"]
        sb = (s["sb"][e] if case["experts"] else s["sb"]).to(f8)
        for j in range(sb.shape[1]):
            ks = slice(j * BLOCK, (j + 1) * BLOCK)
            part = s["a"][lo:lo + c, ks].to(f8) @ b[:, ks].to(f8).t().contiguous()
            part *= s["sa"][lo:lo + c, j, None].to(f8)
            part *= sb[:, j].repeat_interleave(BLOCK)[None, :case["n"]]
            out[lo:lo + c] += part
    return out


def work(case):
    """Bytes read and written once, and the products' operations."""
    op, rows, k = case["op"], case["rows"], case["k"]
    kb = -(-k // BLOCK)
    if op == "quant":
        return {"bytes": rows * k * 3 + 4 * -(-rows // case["block_rows"]) * kb, "flops": 0}
    n, experts = case["n"], case["experts"]
    counts = sizes(case)
    used = sum(c > 0 for c in counts)
    out = 4 if case["out"] == "f32" else 2
    index = 4 * (experts + 1) if experts else 0
    flops = 2 * rows * k * n
    if op == "wgrad":
        return {"bytes": rows * (k + n) * 2 + experts * k * n * out + index, "flops": flops}
    if op == "grouped":
        return {"bytes": rows * k * 2 + used * k * n * 2 + rows * n * out + index, "flops": flops}
    nb = -(-n // BLOCK)
    return {"bytes": rows * k + used * n * k + 4 * (rows + used * nb) * kb + rows * n * out + index,
            "flops": flops}
