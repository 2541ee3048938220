"""Operators of a layer in microscaled 4 bits as cases that can be timed and compared.

The quantizer to 4-bit codes (both ways round from one read), the product of
4-bit weights with 4- or 8-bit activations, the same product of experts over
ragged rows, and the norm in front of them, whose output leaves as the
product's operand, with its backward pass.  `run` computes a case in
elementary torch operations, or, with `own` true, through the library's entry
points.
"""
import math

import torch

own = False

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
FMAX = {E4M3: 448.0, E5M2: 57344.0}
WIDE = {"f32": torch.float32, "bf16": torch.bfloat16}
FP8 = {"e4m3": E4M3, "e5m2": E5M2}


def listed():
    return [
        # one token's activations on their way into a 4-bit product: latency
        dict(name="quantise one token", op="quant", B=1, R=1, C=4096, dtype="bf16", format="mx", rows=True, cols=False),
        # float32 values of odd extent to nvfp4, under a tensor's own factor
        dict(name="quantise odd rows to nvfp4", op="quant", B=1, R=4133, C=1072, dtype="f32", format="nv", rows=True,
             cols=False),
        # eight experts' weights after an update: one read, the operand of the
        # product and the transposed one that the input's gradient needs
        dict(name="quantise weights both ways", op="quant", B=8, R=4096, C=4096, dtype="bf16", format="mx", rows=True,
             cols=True),
        # one token through a linear layer: the weights' bytes are all there is
        dict(name="product of one token", op="product", B=1, M=1, N=8192, K=4096, a="e2m1", out="bf16"),
        # a short prompt of odd length, a contraction of 90 blocks, activations in 8 bits
        dict(name="product of a prompt", op="product", B=1, M=1021, N=1792, K=2880, a="e4m3", out="bf16"),
        # a weight's gradient from transposed 4-bit operands: long contraction, few tiles, float32 out
        dict(name="product of a weight's gradient", op="product", B=1, M=1024, N=1024, K=16384, a="e2m1", out="f32"),
        # a training batch forward, 4 bits on both sides
        dict(name="product of a training batch", op="product", B=1, M=16384, N=8192, K=4096, a="e2m1", out="bf16"),
        # 8 tokens, 4 of 32 experts with 4-bit weights
        dict(name="experts for 8 tokens", op="experts", T=8, E=32, k=4, N=4096, K=2048, a="e4m3", align=1),
        # a training batch over 32 experts, tokens gathered by the product
        dict(name="experts for a batch", op="experts", T=16384, E=32, k=4, N=4096, K=2048, a="e2m1", align=128),
        # rms norm of one token, in bfloat16 for the residual path and as an 8-bit operand
        dict(name="norm of one token", op="norm", R=1, C=4096, dtype="bf16", kind="rms", code="e4m3", y=True,
             train=False),
        # layer norm of float32 rows of odd length, forward and backward
        dict(name="norm of odd rows, training", op="norm", R=4133, C=1001, dtype="f32", kind="layer", code="none",
             y=True, train=True),
        # layer norm of a training batch: bfloat16 out and the 8-bit operand,
        # then the gradients of the input, the weight and the bias
        dict(name="norm of a training batch", op="norm", R=16384, C=4096, dtype="bf16", kind="layer", code="e4m3",
             y=True, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "quant", "product", "product", "product", "experts", "experts", "norm", "norm"))
    if op == "quant":
        fmt = rng.choice(("mx", "mx", "nv"))
        rows, cols = rng.choice(((True, False), (True, True), (False, True)))
        R = _log(rng, 1, 8192)
        # blocks run along the columns, for the transposed codes along the rows
        return dict(op=op, B=rng.randint(1, 3), R=32 * -(-R // 32) if cols else R, C=32 * _log(rng, 2, 128),
                    dtype=rng.choice(("f32", "bf16")), format=fmt, rows=rows, cols=cols)
    if op == "product":
        B, a = rng.choice((1, 1, 1, 2, 3)), rng.choice(("e2m1", "e2m1", "e4m3", "e5m2"))
        # float32 where the matrix core's sums are as good as that: fp8 values
        # next to each other are cut to 13 bits below the largest product
        return dict(op=op, B=B, M=_log(rng, 1, 8192), N=16 * _log(rng, 8, 256), K=32 * _log(rng, 4, 128), a=a,
                    out=rng.choice(("f32", "bf16")) if a == "e2m1" else "bf16")
    if op == "experts":
        return dict(op=op, T=_log(rng, 1, 8192), E=rng.choice((4, 8, 16, 32, 48)), k=rng.randint(1, 4),
                    N=16 * rng.randint(16, 180), K=32 * rng.randint(8, 64),
                    a=rng.choice(("e2m1", "e4m3", "e5m2")), align=rng.choice((1, 1, 128)))
    code = rng.choice(("none", "e4m3", "e5m2"))
    C = _log(rng, 16, 8192)
    return dict(op=op, R=_log(rng, 1, 8192), C=C if code == "none" else 32 * -(-C // 32),
                dtype=rng.choice(("f32", "bf16")), kind=rng.choice(("layer", "rms")), code=code,
                y=code == "none" or rng.random() < 0.5, train=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs --

# where e2m1's magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 change
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _fp4(g, shape):
    """Packed codes (lower index in the low nibble) and block exponents as the
    quantizer makes them of normal values."""
    v = torch.randn(shape, generator=g, device="cuda") * 2.0
    c = torch.bucketize(v.abs(), torch.tensor(MIDS, device="cuda"), out_int32=True).to(torch.uint8)
    c |= torch.signbit(v).to(torch.uint8) << 3
    e = torch.randint(-8, -4, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.int32)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e + 127).to(torch.uint8).view(E8M0)


def _fp8(g, shape, dtype):
    x = torch.randn(shape, generator=g, device="cuda")
    codes = (x * (FMAX[dtype] / 5.0)).clamp_(-FMAX[dtype], FMAX[dtype]).to(dtype)
    e = torch.randint(-12, -8, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.int32)
    return codes, (e + 127).to(torch.uint8).view(E8M0)


def _operand(g, shape, kind):
    return _fp4(g, shape) if kind == "e2m1" else _fp8(g, shape, FP8[kind])


def _capacity(T, k, E, align):
    n = T * k
    return -(-(n + min(E, n) * (align - 1)) // align) * align


def _order(ids, E, align, cap):
    """First rows of the experts' segments (multiples of `align`) and the choice at each row (-1: none)."""
    flat = ids.reshape(-1).long()
    by, at = flat.sort(stable=True)
    counts = torch.zeros(E, dtype=torch.long, device=ids.device).scatter_add_(0, flat, torch.ones_like(flat))
    held = (counts + align - 1) // align * align
    offsets = torch.cat([held.new_zeros(1), held.cumsum(0)])
    before = counts.cumsum(0) - counts
    row = offsets[by] + torch.arange(flat.numel(), device=ids.device) - before[by]
    rows = torch.full((cap,), -1, dtype=torch.int32, device=ids.device)
    rows[row] = at.to(torch.int32)
    return offsets.to(torch.int32), rows


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    s = dict(case)
    op = case["op"]
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "quant":
        B, R, C = case["B"], case["R"], case["C"]
        # weights and activations: normal, rows of different size
        size = torch.exp2(torch.randn(B, R, 1, generator=g, device="cuda") * 0.5 - 5.0)
        s["x"] = (torch.randn(B, R, C, generator=g, device="cuda") * size).to(WIDE[case["dtype"]])
        block, kind = (32, E8M0) if case["format"] == "mx" else (16, E4M3)
        # a program keeps a tensor's factor from its last largest magnitude
        s["factor"] = 6.0 * 448.0 / s["x"].float().abs().amax().reshape(1) if case["format"] == "nv" else None
        s["codes"], s["scales"] = ((new((B, R, C // 2), torch.uint8), new((B, R, C // block), kind))
                                   if case["rows"] else (None, None))
        s["codes_t"], s["scales_t"] = ((new((B, C, R // 2), torch.uint8), new((B, C, R // block), kind))
                                       if case["cols"] else (None, None))
    elif op == "product":
        B, M, N, K = (case[n] for n in ("B", "M", "N", "K"))
        s["lhs"], s["lhs_scales"] = _operand(g, (B, M, K), case["a"])
        s["rhs"], s["rhs_scales"] = _fp4(g, (B, N, K))
        s["y"] = new((B, M, N), WIDE[case["out"]])
    elif op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        score = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda") * 0.5
        s["cap"] = _capacity(T, k, E, case["align"])
        s["offsets"], s["rows"] = _order(score.topk(k, dim=1).indices, E, case["align"], s["cap"])
        # the program knows the longest segment it plans for
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
        s["x"], s["x_scales"] = _operand(g, (T, K), case["a"])
        s["w"], s["w_scales"] = _fp4(g, (E, N, K))
        s["y"] = new((s["cap"], N), torch.bfloat16)
    else:
        R, C, dt = case["R"], case["C"], WIDE[case["dtype"]]
        # a residual stream: rows of different size, some columns far from zero
        shift = torch.randn(C, generator=g, device="cuda") * 0.5
        size = torch.exp2(torch.randn(R, 1, generator=g, device="cuda") * 0.5)
        s["x"] = ((torch.randn(R, C, generator=g, device="cuda") + shift) * size + 0.2).to(dt)
        s["gamma"] = 1.0 + 0.2 * torch.randn(C, generator=g, device="cuda")
        s["beta"] = 0.1 * torch.randn(C, generator=g, device="cuda") if case["kind"] == "layer" else None
        s["out"] = new((R, C), dt) if case["y"] else None
        coded = case["code"] != "none"
        s["codes"] = new((R, C), FP8[case["code"]]) if coded else None
        s["scales"] = new((R, C // 32), E8M0) if coded else None
        s["mean"] = new((R,), torch.float32) if case["kind"] == "layer" and case["train"] else None
        s["rstd"] = new((R,), torch.float32) if case["train"] else None
        if case["train"]:
            s["dy"] = torch.randn(R, C, generator=g, device="cuda").to(dt)
            s["dx"] = new((R, C), dt)
            s["dgamma"] = new((C,), torch.float32)
            s["dbeta"] = new((C,), torch.float32) if case["kind"] == "layer" else None
            s["space"] = new(max(16, 8 * C * min(R, 1024)), torch.uint8)
    return s


# ------------------------------------------------------------ plain forms --

def _power(e):
    """2^e in 32 bits, made of its bits: torch.ldexp rounds its powers."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _exponent(amax, fmax):
    """The least E with max(amax, 1e-10) <= fmax 2^E, in 64 bits (amax next to fmax 2^E)."""
    m, e = torch.frexp(amax.clamp_min(1e-10).double() / fmax)
    return torch.where(m == 0.5, e - 1, e).clamp(-127, 127).to(torch.int32)


def _e2m1(v):
    """Codes of values in [-6, 6], nearest, ties to the even code; two to a byte."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c |= torch.signbit(v).to(torch.uint8) << 3
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _quantize4(x, factor):
    """Blocks along the last axis: mxfp4 of 32 (factor None), else nvfp4 of 16."""
    if factor is None:
        b = x.float().reshape(*x.shape[:-1], -1, 32)
        E = _exponent(b.abs().amax(-1), 6.0)
        return _e2m1((b * _power(-E)[..., None]).view(x.shape)), (E + 127).to(torch.uint8).view(E8M0)
    b = (x.float() * factor).reshape(*x.shape[:-1], -1, 16)
    # a sixth in 64 bits: torch divides by a number through its reciprocal
    scale = (b.abs().amax(-1).double() / 6.0).float().clamp(2.0 ** -9, 448.0).to(E4M3)
    return _e2m1((b / scale.float()[..., None]).view(x.shape)), scale


def _plain_quant(s):
    out = {}
    if s["rows"]:
        out["codes"], out["scales"] = _quantize4(s["x"], s["factor"])
    if s["cols"]:
        out["codes_t"], out["scales_t"] = _quantize4(s["x"].transpose(1, 2).contiguous(), s["factor"])
    return out


def _values(codes, scales):
    """What codes (packed e2m1 where they are bytes, else fp8) under scales of 32 stand for, in 32 bits (exact)."""
    if codes.dtype == torch.uint8:
        v = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), device=codes.device)
        v = torch.cat([v, -v])
        # both values of a byte at once
        pairs = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)
        x = pairs[codes.int()].view(*codes.shape[:-1], -1)
    else:
        x = codes.float()
    b = x.reshape(*scales.shape, 32) * _power(scales.view(torch.uint8).int() - 127)[..., None]
    return b.view(x.shape)


def _plain_product(s):
    a, b = _values(s["lhs"], s["lhs_scales"]), _values(s["rhs"], s["rhs_scales"])
    return {"out": torch.bmm(a, b.transpose(1, 2).contiguous()).to(s["y"].dtype)}


def _plain_experts(s):
    a, b = _values(s["x"], s["x_scales"]), _values(s["w"], s["w_scales"])
    first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = first[:, None] + torch.arange(s["most"], device=first.device)
    there = at < last[:, None]
    row = s["rows"][at.clamp_max(s["cap"] - 1)]
    there = there & (row >= 0)
    x = torch.where(there[:, :, None], a[row.clamp_min(0).long() // s["k"]], 0.0)  # [E, most, K]
    y = torch.bmm(x, b.transpose(1, 2).contiguous())
    r = torch.arange(s["cap"], device=at.device)
    e = torch.searchsorted(last.contiguous(), r, right=True)
    held = e < s["E"]
    e = e.clamp_max(s["E"] - 1)
    i = (r - first[e]).clamp(0, s["most"] - 1)
    return {"out": torch.where(held[:, None], y[e, i], 0.0).bfloat16()}


EPS = 1e-5


def _plain_norm(s):
    x = s["x"].float()
    layer = s["kind"] == "layer"
    out = {}
    if layer:
        mean = x.sum(1, keepdim=True) / s["C"]
        x = x - mean
    rstd = 1.0 / torch.sqrt(x.square().sum(1, keepdim=True) / s["C"] + EPS)
    xn = x * rstd
    y = xn * s["gamma"] + s["beta"] if layer else xn * s["gamma"]
    if s["y"]:
        out["y"] = y.to(s["x"].dtype)
    if s["codes"] is not None:
        dt = s["codes"].dtype
        b = y.reshape(s["R"], -1, 32)
        E = _exponent(b.abs().amax(-1), FMAX[dt])
        out["codes"] = (b * _power(-E)[..., None]).clamp(-FMAX[dt], FMAX[dt]).view(y.shape).to(dt)
        out["scales"] = (E + 127).to(torch.uint8).view(E8M0)
    if s["train"]:
        if layer:
            out["mean"] = mean[:, 0]
        out["rstd"] = rstd[:, 0]
        dy = s["dy"].float()
        d = dy * s["gamma"]
        dx = d - xn * (d * xn).sum(1, keepdim=True) / s["C"]
        if layer:
            dx = dx - d.sum(1, keepdim=True) / s["C"]
            out["dbeta"] = dy.sum(0)
        out["dx"] = (dx * rstd).to(s["x"].dtype)
        out["dgamma"] = (dy * xn).sum(0)
    return out


# --------------------------------------------------------- the library's --

def _own(s):
    import block_scaled_precision_blockwise_amd as bsq

    op = s["op"]
    if op == "quant":
        bsq.bsq_quant_fp4(s["x"], s["codes"], s["scales"], s["codes_t"], s["scales_t"],
                          format=bsq.BSQ_MXFP4 if s["format"] == "mx" else bsq.BSQ_NVFP4, factor=s["factor"])
        return {n: s[n] for n in ("codes", "scales", "codes_t", "scales_t") if s[n] is not None}
    if op == "product":
        bsq.bsq_scaled_matmul_mxfp4(s["lhs"], s["rhs"], s["lhs_scales"], s["rhs_scales"], s["y"])
        return {"out": s["y"]}
    if op == "experts":
        bsq.bsq_moe_matmul_mxfp4(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"], s["y"], rows=s["rows"],
                                 k=s["k"])
        return {"out": s["y"]}
    kind = bsq.BSQ_LAYER_NORM if s["kind"] == "layer" else bsq.BSQ_RMS_NORM
    bsq.bsq_norm_mx(s["x"], y=s["out"], codes=s["codes"], scales=s["scales"], gamma=s["gamma"], beta=s["beta"],
                    mean=s["mean"], rstd=s["rstd"], eps=EPS, kind=kind)
    out = {"y": s["out"], "codes": s["codes"], "scales": s["scales"]}
    if s["train"]:
        bsq.bsq_norm_backward(s["x"], s["dy"], s["rstd"], s["dx"], mean=s["mean"], gamma=s["gamma"],
                              dgamma=s["dgamma"], dbeta=s["dbeta"], workspace=s["space"], kind=kind)
        out.update({n: s[n] for n in ("mean", "rstd", "dx", "dgamma", "dbeta")})
    return {n: v for n, v in out.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "product": _plain_product, "experts": _plain_experts,
            "norm": _plain_norm}[state["op"]](state)


def _bytes(kind):
    """Bytes of a value with its share of a block's scale."""
    return (0.5 if kind == "e2m1" else 1.0) + 1 / 32


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["B"] * case["R"] * case["C"]
        code = 0.5 + (1 / 32 if case["format"] == "mx" else 1 / 16)
        return {"bytes": n * ((4 if case["dtype"] == "f32" else 2) + code * (case["rows"] + case["cols"])),
                "flops": 0}
    if op == "product":
        B, M, N, K = (case[n] for n in ("B", "M", "N", "K"))
        return {"bytes": B * (M * K * _bytes(case["a"]) + N * K * _bytes("e2m1") +
                              M * N * (4 if case["out"] == "f32" else 2)), "flops": 2 * B * M * N * K}
    if op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        asked = E * (1.0 - (1.0 - 1.0 / E) ** (T * k))  # experts that some token chose
        return {"bytes": T * K * _bytes(case["a"]) + asked * N * K * _bytes("e2m1") + 2 * T * k * N,
                "flops": 2 * T * k * N * K}
    n, e = case["R"] * case["C"], 4 if case["dtype"] == "f32" else 2
    b = e + e * case["y"] + (1 + 1 / 32) * (case["code"] != "none") + 3 * e * case["train"]
    return {"bytes": n * b, "flops": n * (8 + 12 * case["train"])}


# ------------------------------------------------------- definition in 64 --

def _block64(x, size, fmax):
    """Largest magnitudes of blocks and the least power of two that brings them into the format."""
    top = x.reshape(*x.shape[:-1], -1, size).abs().amax(-1)
    E = torch.floor(torch.log2(top.clamp_min(1e-10) / fmax)) - 1
    for _ in range(3):
        E = torch.where(top.clamp_min(1e-10) > fmax * torch.exp2(E), E + 1, E)
    return top, torch.exp2(E)


def _fp64(v, mantissa, least):
    """The nearest value with `mantissa` bits behind the leading one, which is not below 2^least."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min(least).double() - mantissa)
    return torch.round(v / step) * step


def _wide64(codes, scales):
    if codes.dtype != torch.uint8:
        return codes.double() * scales.float().double().repeat_interleave(32, -1)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    return torch.where(c > 7, -v, v) * scales.float().double().repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        out = {"codes": None, "codes_t": None}  # bytes: they have to be equal
        for name, x in (("scales", s["x"]), ("scales_t", s["x"].transpose(1, 2))):
            if s[name] is None:
                continue
            x = x.double()
            if s["format"] == "mx":
                out[name] = _block64(x, 32, 6.0)[1]
            else:
                top = _block64(x * s["factor"].double(), 16, 6.0)[0]
                out[name] = _fp64((top / 6.0).clamp(2.0 ** -9, 448.0), 3, -6)
        return {n: v for n, v in out.items() if s[n] is not None}
    if op == "product":
        out = [_wide64(a, sa) @ _wide64(b, sb).t()
               for a, sa, b, sb in zip(s["lhs"], s["lhs_scales"], s["rhs"], s["rhs_scales"])]
        return {"out": torch.stack(out)}
    if op == "experts":
        out = torch.zeros(s["cap"], s["N"], dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(s["E"]):
            rows = s["rows"][ends[e]:ends[e + 1]].long()
            if rows.numel():
                at = rows.clamp_min(0) // s["k"]
                x = _wide64(s["x"][at], s["x_scales"][at]) * (rows >= 0)[:, None]
                out[ends[e]:ends[e + 1]] = x @ _wide64(s["w"][e], s["w_scales"][e]).t()
        return {"out": out}
    layer = s["kind"] == "layer"
    x = s["x"].double().requires_grad_(True)
    gamma = s["gamma"].double().requires_grad_(True)
    beta = s["beta"].double().requires_grad_(True) if layer else None
    mean = x.mean(1, keepdim=True) if layer else 0.0
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS) ** -0.5
    y = (x - mean) * rstd * gamma
    y = y + beta if layer else y
    out = {}
    if s["y"]:
        out["y"] = y.detach()
    if s["codes"] is not None:
        scale = _block64(y.detach(), 32, FMAX[s["codes"].dtype])[1]
        bits, least = (3, -6) if s["code"] == "e4m3" else (2, -14)
        out["codes"] = _fp64(y.detach() / scale.repeat_interleave(32, 1), bits, least)
        out["scales"] = scale
    if s["train"]:
        if layer:
            out["mean"] = mean.detach()[:, 0]
        out["rstd"] = rstd.detach()[:, 0]
        leaves = [x, gamma] + ([beta] if layer else [])
        for name, v in zip(("dx", "dgamma", "dbeta"), torch.autograd.grad((y * s["dy"].double()).sum(), leaves)):
            out[name] = v
    return out
