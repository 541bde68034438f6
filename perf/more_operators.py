"""What the operators around the expert products are measured on: their
cases, inputs, plain forms and 64-bit definitions.

``route``    ids [T, top] of experts to offsets and places (a stable sort by expert;
             an id outside the experts has no place, -1), and xs[place[t, j]] = x[t]
``combine``  y[t] = sum_j w[t, j] h[place[t, j]]; with ``train`` also, from dy,
             dh[place[t, j]] = w[t, j] dy[t] and dw[t, j] = <dy[t], h[place[t, j]]>
``norm``     h = x + residual, rounded to its type; y = h / sqrt(mean(h^2) + eps) * weight,
             also as E4M3 codes with a float32 scale for each 128 columns; with ``train``
             y alone, and from dy and the gradient dh of h: dx (= the residual's) and dweight
``mxquant``  x to E2M1 codes with an E8M0 scale for each 32 columns, and back to values
``mxfp4``    c = (a * sa) @ (b * sb)^T of such codes, dense (experts = 0) or by expert

Where ``own`` is false, ``run`` computes the plain form in 32 bits with
elementary torch operations; where it is true, it calls the library.
"""
import math
import random

import torch

own = False

BLOCK = 128           # columns that one E4M3 scale covers
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
MX = 32               # columns that one E8M0 scale covers
EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of 16 sequences, eight experts each, out of 64: latency
        {"name": "route, decode", "op": "route", "tokens": 16, "top": 8, "experts": 64, "k": 2048,
         "type": "bf16", "ids": "int64", "skew": 0.0, "drop": 0.0},
        # a training step: two experts a token, out of eight
        {"name": "route, train", "op": "route", "tokens": 8192, "top": 2, "experts": 8, "k": 4096,
         "type": "bf16", "ids": "int64", "skew": 0.3, "drop": 0.0},
        # a decoding batch's way back
        {"name": "combine, decode", "op": "combine", "tokens": 25, "top": 4, "experts": 32, "k": 2048,
         "type": "f16", "skew": 0.5, "drop": 0.0, "train": False},
        # a training step's way back and both gradients; some tokens are padding
        {"name": "combine, train", "op": "combine", "tokens": 8191, "top": 2, "experts": 16, "k": 4096,
         "type": "bf16", "skew": 0.5, "drop": 0.02, "train": True},
        # the input of an fp8 layer: a few decoding rows, and a long prompt
        {"name": "norm, decode", "op": "norm", "rows": 5, "k": 7168, "type": "f16", "train": False},
        {"name": "norm, prompt", "op": "norm", "rows": 8192, "k": 4096, "type": "bf16", "train": False},
        # a training step's norm, forward and backward
        {"name": "norm, train", "op": "norm", "rows": 8191, "k": 4096, "type": "bf16", "train": True},
        # activations before a 4-bit product: a ragged batch, and a long prompt
        {"name": "mxfp4 quantise, 777 rows", "op": "mxquant", "rows": 777, "k": 1544, "type": "f16"},
        {"name": "mxfp4 quantise, 8192 rows", "op": "mxquant", "rows": 8192, "k": 7168, "type": "bf16"},
        # a dense 4-bit layer for a few decoding rows: bound by the weights' bytes
        {"name": "mxfp4 decode, 5 rows", "op": "mxfp4", "rows": 5, "experts": 0, "k": 7168, "n": 4096,
         "out": "bf16", "route": 8, "skew": 0.0},
        # the same kind of layer on a long prompt: bound by the matrix cores
        {"name": "mxfp4 prompt, 8192 rows", "op": "mxfp4", "rows": 8192, "experts": 0, "k": 4096,
         "n": 4096, "out": "bf16", "route": 9, "skew": 0.0},
        # experts in 4 bits on a middling batch
        {"name": "mxfp4 experts, 3001 rows", "op": "mxfp4", "rows": 3001, "experts": 32, "k": 2048,
         "n": 2816, "out": "bf16", "route": 10, "skew": 0.7},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, step * round(v / step)))


def _drawn(rng):
    op = rng.choice(["route", "combine", "norm", "norm", "mxquant", "mxfp4", "mxfp4", "mxfp4"])
    typ = rng.choice(["bf16", "f16"])
    skew = rng.choice([0.0, 0.5, 1.0])
    if op in ("route", "combine"):
        c = {"op": op, "tokens": _log(rng, 1, 16384), "top": rng.choice([1, 2, 4, 6, 8]),
             "experts": _log(rng, 8, 128), "k": _log(rng, 512, 8192, 8), "type": typ, "skew": skew,
             "drop": rng.choice([0.0, 0.0, 0.1])}
        c.update({"ids": rng.choice(["int32", "int64"])} if op == "route"
                 else {"train": rng.random() < 0.5})
        return c
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 16384), "k": _log(rng, 512, 8192, 8), "type": typ,
                "train": rng.random() < 0.5}
    if op == "mxquant":
        return {"op": op, "rows": _log(rng, 1, 16384), "k": _log(rng, 512, 8192, 8), "type": typ}
    return {"op": op, "rows": _log(rng, 1, 16384), "experts": rng.choice([0, _log(rng, 4, 64)]),
            "k": _log(rng, 512, 7168, 32), "n": _log(rng, 512, 4096, 8),
            "out": rng.choice(["bf16", "f16", "f32"]), "route": rng.randrange(1, 1 << 30),
            "skew": skew}


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
    if not case["experts"]:
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


# ---- plain pieces ----------------------------------------------------------


def _sorted(ids, experts):
    """Offsets and places of ids [T, top] by a stable sort; ids outside the experts sort last."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=order.device)
    place = torch.where(key < experts, place, -1).to(torch.int32).view(ids.shape)
    offsets = (key[None, :] < torch.arange(experts + 1, device=key.device)[:, None]).sum(1)
    return offsets.to(torch.int32), place


def _e4m3(y):
    """E4M3 codes of y (float32) and their scales, one for each 1 x 128 block."""
    m, k = y.shape
    kb = -(-k // BLOCK)
    p = torch.nn.functional.pad(y, (0, kb * BLOCK - k)).view(m, kb, BLOCK)
    amax = p.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = p * (torch.full_like(amax, E4M3_MAX) / amax)[:, :, None]
    return q.view(m, -1)[:, :k].to(torch.float8_e4m3fn), amax / E4M3_MAX


def _mx_blocks(x):
    """x in float32 as [rows, blocks, 32], zeros behind a partial last block."""
    m, k = x.shape
    kb = -(-k // MX)
    return torch.nn.functional.pad(x.float(), (0, kb * MX - k)).view(m, kb, MX)


def _mx_exponents(p):
    """E8M0 codes of blocks: floor(log2(amax)) - 2 (E2M1's largest power of two), 255 where
    a value is not finite."""
    bits = p.abs().amax(2).contiguous().view(torch.int32) >> 23
    return torch.where(p.isfinite().all(2), (bits - 2).clamp_min(0), 255)


def _mx_scales(codes):
    """The values of E8M0 codes, exactly (2^-127 is a subnormal float32)."""
    s = torch.where(codes == 0, 1 << 22, codes << 23).view(torch.float32)
    return torch.where(codes == 255, math.nan, s)


def _mx_round(v):
    """Nearest E2M1 values, ties to the even code, saturating at 6 (steps of 0.5, 1 and 2)."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp_max(6.0), v)


def _mx_codes(x):
    """Packed E2M1 codes (the even column in the low half of a byte) and E8M0 codes of x."""
    p = _mx_blocks(x)
    e = _mx_exponents(p)
    v = _mx_round(p / _mx_scales(e)[:, :, None])
    levels = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    code = torch.bucketize(v.abs(), levels, right=True) + 8 * torch.signbit(v)
    code = code.view(x.shape[0], -1)[:, :x.shape[1]].to(torch.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, e.to(torch.uint8)


def _mx_values(q, scale):
    """The float32 values of packed codes and their scales."""
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    levels = torch.cat([levels, -levels])
    v = torch.stack([levels[(q & 15).int()], levels[(q >> 4).int()]], -1).flatten(-2)
    each = _mx_scales(scale.int()).repeat_interleave(MX, -1)[..., :v.shape[-1]]
    return v * each


# ---- inputs ----------------------------------------------------------------


def _chosen(case, g):
    """Each token's experts: the top of a common preference and the token's own; a dropped
    token's are -1."""
    t, e = case["tokens"], case["experts"]
    like = case["skew"] * torch.randn(e, generator=g, device="cuda")
    gumbel = -torch.log(-torch.log(torch.rand(t, e, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    ids = (gumbel + like).topk(case["top"], 1).indices
    keep = torch.rand(t, 1, generator=g, device="cuda") >= case["drop"]
    return torch.where(keep, ids, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    op, k = case["op"], case["k"]
    s = {"case": case}
    dtype = DTYPES[case.get("type", "f32")]
    if op in ("route", "combine"):
        t, top = case["tokens"], case["top"]
        ids = _chosen(case, g)
    if op == "route":
        s["x"] = normal(t, k, dtype=dtype)
        s["ids"] = ids.to(getattr(torch, case["ids"]))
        s["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device="cuda")
        s["place"] = torch.empty(t, top, dtype=torch.int32, device="cuda")
        s["xs"] = torch.zeros(t * top, k, dtype=dtype, device="cuda")
    elif op == "combine":
        s["place"] = _sorted(ids, case["experts"])[1]
        s["h"] = normal(t * top, k, dtype=dtype)
        s["w"] = torch.softmax(normal(t, top), 1)
        s["y"] = torch.empty(t, k, dtype=dtype, device="cuda")
        if case["train"]:
            s["dy"] = normal(t, k, scale=0.05, dtype=dtype)
            s["dh"] = torch.zeros_like(s["h"])
            s["dw"] = torch.empty_like(s["w"])
    elif op == "norm":
        m = case["rows"]
        # a few channels carry much larger values than the others
        s["x"] = normal(m, k, scale=0.5, dtype=dtype)
        s["res"] = (normal(m, k) * torch.exp(normal(k))).to(dtype)
        s["weight"] = (1 + normal(k, scale=0.1)).to(dtype)
        s["h"], s["y"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        if case["train"]:
            s["rstd"] = torch.empty(m, device="cuda")
            s["dy"], s["dh"] = normal(m, k, scale=0.05, dtype=dtype), normal(m, k, scale=0.05, dtype=dtype)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty(k, device="cuda")
        else:
            s["q"] = torch.empty(m, k, dtype=torch.float8_e4m3fn, device="cuda")
            s["scale"] = torch.empty(m, -(-k // BLOCK), device="cuda")
    elif op == "mxquant":
        m = case["rows"]
        s["x"] = (normal(m, k) * torch.exp(normal(k))).to(dtype)
        s["q"] = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(m, -(-k // MX), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty_like(s["x"])
    else:
        m, n, experts = case["rows"], case["n"], case["experts"]
        s["starts"] = _starts(sizes(case))
        s["offsets"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
        s["a"], s["sa"] = _mx_codes(normal(m, k))
        e1 = max(experts, 1)
        s["b"] = torch.empty(e1, n, k // 2, dtype=torch.uint8, device="cuda")
        s["sb"] = torch.empty(e1, n, -(-k // MX), dtype=torch.uint8, device="cuda")
        for e in range(e1):
            s["b"][e], s["sb"][e] = _mx_codes(normal(n, k, scale=k ** -0.5))
        if not experts:
            s["b"], s["sb"] = s["b"][0], s["sb"][0]
        s["c"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device="cuda")
    return s


# ---- one pass --------------------------------------------------------------


def _calls(s, **kw):
    """The library's calls of one pass."""
    import communication_gemm_amd as agg
    case = s["case"]
    op = case["op"]
    if op == "route":
        if "workspace" not in s:
            n = agg.expert_sort_workspace_bytes(case["tokens"], case["top"], case["experts"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return [agg.ag_gemm_expert_sort(s["ids"], case["experts"], s["offsets"], s["place"],
                                        s["workspace"], **kw),
                agg.ag_gemm_expert_dispatch(s["x"], s["place"], s["xs"], **kw)]
    if op == "combine":
        calls = [agg.ag_gemm_expert_combine(s["h"], s["place"], s["w"], s["y"], **kw)]
        if case["train"]:
            calls.append(agg.ag_gemm_expert_combine_grad(s["dy"], s["h"], s["place"], s["w"], s["dh"],
                                                         s["dw"], **kw))
        return calls
    if op == "norm":
        if not case["train"]:
            return [agg.ag_gemm_rmsnorm(s["x"], s["weight"], q=s["q"], scale=s["scale"],
                                        residual=s["res"], h=s["h"], eps=EPS, **kw)]
        if "workspace" not in s:
            n = agg.rmsnorm_grad_workspace_bytes(case["rows"], case["k"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return [agg.ag_gemm_rmsnorm(s["x"], s["weight"], y=s["y"], residual=s["res"], h=s["h"],
                                    rstd=s["rstd"], eps=EPS, **kw),
                agg.ag_gemm_rmsnorm_grad(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"],
                                         s["workspace"], dh=s["dh"], **kw)]
    if op == "mxquant":
        return [agg.ag_gemm_quant_mxfp4(s["x"], s["q"], s["scale"], **kw),
                agg.ag_gemm_dequant_mxfp4(s["q"], s["scale"], s["y"], **kw)]
    if case["experts"]:
        return [agg.ag_gemm_grouped_mxfp4(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["c"], **kw)]
    return [agg.ag_gemm_mxfp4(s["a"], s["sa"], s["b"], s["sb"], s["c"], **kw)]


def _outputs(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return [s[n] for n in (("h", "y", "dx", "dweight") if case["train"] else ("h", "q", "scale"))]
    if op == "mxquant":
        return [s["y"], s["scale"].view(torch.float8_e8m0fnu)]
    if op == "combine":
        return [s[n] for n in (("y", "dh", "dw") if case["train"] else ("y",))]
    return [s[n] for n in (("offsets", "place", "xs") if op == "route" else ("c",))]


def run(s):
    case = s["case"]
    if own:
        if case.get("rows", case.get("tokens")) > 512:
            _calls(s)
            return _outputs(s)
        # a decoding loop keeps its buffers and marshals its calls once
        if "calls" not in s:
            s["calls"] = _calls(s, prepare=True)
        for call in s["calls"]:
            call()
        return _outputs(s)
    op = case["op"]
    if op == "route":
        offsets, place = _sorted(s["ids"], case["experts"])
        rows = torch.where(place >= 0, place, len(s["xs"])).long()      # no place: a row of its own
        xs = torch.zeros(len(s["xs"]) + 1, case["k"], dtype=s["xs"].dtype, device="cuda")
        xs[rows.flatten()] = s["x"].repeat_interleave(case["top"], 0)
        return [offsets, place, xs[:-1]]
    if op == "combine":
        dtype, has = s["h"].dtype, s["place"] >= 0
        at = s["place"].clamp_min(0).long()
        w = torch.where(has, s["w"], 0.0)
        rows = s["h"][at].float()                                       # [T, top, K]
        y = (rows * w[:, :, None]).sum(1).to(dtype)
        if not case["train"]:
            return [y]
        dy = s["dy"].float()
        dh = torch.zeros(len(s["h"]) + 1, case["k"], dtype=dtype, device="cuda")
        dh[torch.where(has, at, len(s["h"])).flatten()] = (dy[:, None] * w[:, :, None]).to(dtype).flatten(0, 1)
        dw = torch.where(has, (rows * dy[:, None]).sum(2), 0.0)
        return [y, dh[:-1], dw]
    if op == "norm":
        dtype, weight = s["x"].dtype, s["weight"].float()
        h = (s["x"].float() + s["res"].float()).to(dtype)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
        y = hf * rstd * weight
        if not case["train"]:
            return [h, *_e4m3(y)]
        dy = s["dy"].float()
        g, n = dy * weight, hf * rstd
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True)) + s["dh"].float()
        return [h, y.to(dtype), dx.to(dtype), (dy * n).sum(0)]
    if op == "mxquant":
        p = _mx_blocks(s["x"])
        e = _mx_exponents(p)
        scale = _mx_scales(e)[:, :, None]
        y = (_mx_round(p / scale) * scale).view(len(p), -1)[:, :case["k"]]
        return [y.to(s["x"].dtype), e.to(torch.uint8).view(torch.float8_e8m0fnu)]
    a, out = _mx_values(s["a"], s["sa"]), DTYPES[case["out"]]
    if not case["experts"]:
        return [(a @ _mx_values(s["b"], s["sb"]).t()).to(out)]
    c = torch.empty_like(s["c"])
    # a product for each expert that has rows: one of padded groups would do more work
    for e, (lo, hi) in enumerate(zip(s["starts"], s["starts"][1:])):
        if hi > lo:
            c[lo:hi] = (a[lo:hi] @ _mx_values(s["b"][e], s["sb"][e]).t()).to(out)
    return [c]


# ---- definitions in 64 bits ------------------------------------------------


def _nearest(v, grid):
    """The values of grid (from 0 up) nearest to |v|, ties to the even index, with v's sign."""
    a = v.abs().clamp_max(float(grid[-1])).contiguous()
    hi = torch.searchsorted(grid, a).clamp_max(len(grid) - 1)
    lo = (hi - 1).clamp_min(0)
    up, down = grid[hi] - a, a - grid[lo]
    return torch.copysign(grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)], v)


def _exact_e4m3(y):
    grid = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                         for c in range(0x7F)], dtype=torch.float64, device="cuda")
    q = torch.empty_like(y)
    scale = torch.empty(y.shape[0], -(-y.shape[1] // BLOCK), dtype=torch.float64, device="cuda")
    for j in range(scale.shape[1]):
        cols = slice(j * BLOCK, (j + 1) * BLOCK)
        scale[:, j] = y[:, cols].abs().amax(1).clamp_min(AMAX_FLOOR) / E4M3_MAX
        q[:, cols] = _nearest(y[:, cols] / scale[:, j, None], grid)
    return q, scale


def _exact_mx(x):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    y = torch.empty_like(x)
    scale = torch.empty(x.shape[0], -(-x.shape[1] // MX), dtype=torch.float64, device="cuda")
    for j in range(scale.shape[1]):
        cols = slice(j * MX, (j + 1) * MX)
        exponent = torch.frexp(x[:, cols].abs().amax(1)).exponent.double() - 1
        zero = (x[:, cols] == 0).all(1)
        scale[:, j] = torch.exp2(torch.where(zero, -127.0, (exponent - 2).clamp_min(-127.0)))
        y[:, cols] = _nearest(x[:, cols] / scale[:, j, None], grid) * scale[:, j, None]
    return y, scale


def _exact_codes(q):
    """E2M1 values of packed codes from the format's fields."""
    code = torch.stack([q % 16, q // 16], -1).flatten(-2).double()
    sign = 1 - 2 * (code >= 8).double()
    mag = code % 8
    exponent, fraction = mag // 2, mag % 2
    return sign * torch.where(exponent == 0, fraction / 2, (1 + fraction / 2) * torch.exp2(exponent - 1))


def exact(case, seed):
    """The definition in 64 bits, unrounded but for codes and for h, which the norm is taken of
    as it is stored."""
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    f8 = torch.float64
    op, k = case["op"], case["k"]
    if op == "route":
        flat = s["ids"].flatten().long()
        mine = flat[None, :] == torch.arange(case["experts"], device="cuda")[:, None]   # [E, n]
        counts = mine.sum(1)
        ends = counts.cumsum(0)
        rank = (mine.cumsum(1) * mine).sum(0) - 1
        kept_ = mine.any(0)
        place = torch.where(kept_, rank + (ends - counts)[flat.clamp_min(0)], -1)
        xs = torch.zeros(len(flat), k, dtype=f8, device="cuda")
        token = torch.arange(len(flat), device="cuda") // case["top"]
        xs[place[kept_]] = s["x"].to(f8)[token[kept_]]
        offsets = torch.cat([ends.new_zeros(1), ends])
        return [offsets.to(torch.int32), place.to(torch.int32).view(s["ids"].shape), xs]
    if op == "combine":
        h = s["h"].to(f8)
        y = torch.zeros(case["tokens"], k, dtype=f8, device="cuda")
        dh, dw = torch.zeros_like(h), torch.zeros(s["w"].shape, dtype=f8, device="cuda")
        for j in range(case["top"]):
            t = (s["place"][:, j] >= 0).nonzero().flatten()
            at, w = s["place"][t, j].long(), s["w"][t, j, None].to(f8)
            y[t] += w * h[at]
            if case["train"]:
                dy = s["dy"][t].to(f8)
                dh[at] = w * dy
                dw[t, j] = (h[at] * dy).sum(1)
        return [y, dh, dw] if case["train"] else [y]
    if op == "norm":
        total = s["x"].to(f8) + s["res"].to(f8)
        h, weight = total.to(s["x"].dtype).to(f8), s["weight"].to(f8)
        root = torch.sqrt((h * h).sum(1, keepdim=True) / k + EPS)
        y = h * weight / root
        if not case["train"]:
            return [total, *_exact_e4m3(y)]
        dy = s["dy"].to(f8)
        inner = (dy * weight * h).sum(1, keepdim=True) / (k * root ** 3)
        return [total, y, dy * weight / root - h * inner + s["dh"].to(f8), (dy * h / root).sum(0)]
    if op == "mxquant":
        return list(_exact_mx(s["x"].to(f8)))
    c = torch.zeros(case["rows"], case["n"], dtype=f8, device="cuda")
    for e, (lo, hi) in enumerate(zip(s["starts"], s["starts"][1:])):
        if hi == lo:
            continue
        b, sb = (s["b"][e], s["sb"][e]) if case["experts"] else (s["b"], s["sb"])
        # block by block of 32: the sum of products, then the two scales
        for j in range(sb.shape[1]):
            cols = slice(j * MX // 2, (j + 1) * MX // 2)
            part = _exact_codes(s["a"][lo:hi, cols]) @ _exact_codes(b[:, cols]).t().contiguous()
            part *= torch.exp2(s["sa"][lo:hi, j, None].to(f8) - 127)
            part *= torch.exp2(sb[None, :, j].to(f8) - 127)
            c[lo:hi] += part
    return [c]


def work(case):
    """Bytes read and written once, and the products' operations."""
    op, k = case["op"], case["k"]
    elt = 4 if case.get("type") == "f32" else 2
    if op in ("route", "combine"):
        t, top = case["tokens"], case["top"]
        row = k * elt
        if op == "route":
            return {"bytes": t * row * (1 + top) + t * top * (4 + (8 if case["ids"] == "int64" else 4)) +
                    4 * (case["experts"] + 1), "flops": 0}
        n = t * row * (1 + top) + 8 * t * top
        if case["train"]:      # h, place and w once more are not needed: dy and dh, and dw
            n += t * row * (1 + top) + 4 * t * top
        return {"bytes": n, "flops": 2 * t * top * k * (3 if case["train"] else 1)}
    m = case["rows"]
    if op == "norm":
        if case["train"]:      # x, residual, dy, dh in; h, y, dx out; the weight and its gradient
            return {"bytes": 7 * m * k * elt + 6 * k, "flops": 14 * m * k}
        return {"bytes": m * k * (3 * elt + 1) + 4 * m * -(-k // BLOCK) + 2 * k, "flops": 8 * m * k}
    kb = -(-k // MX)
    if op == "mxquant":        # x in; codes, scales and values out
        return {"bytes": m * k * 2 * elt + m * (k // 2 + kb), "flops": 0}
    n, experts = case["n"], case["experts"]
    used = sum(c > 0 for c in sizes(case))
    out = 4 if case["out"] == "f32" else 2
    return {"bytes": (m + used * n) * (k // 2 + kb) + m * n * out + (4 * (experts + 1) if experts else 0),
            "flops": 2 * m * k * n}
