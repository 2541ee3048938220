"""The expert-layer operators as cases that can be timed and compared.

Four operators of a mixture-of-experts layer in block-scaled 8 bits: routing
(scores, choice, weights, and their gradient), the order of rows (sorting the
chosen rows by expert, gathering them into 8-bit operands, summing them back
with their weights), the experts' products over ragged rows, and the gated
activation with its 8-bit checkpoint.  `run` computes a case in elementary
torch operations, or, with `own` true, through the library's entry points.
"""
import math

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FMAX = {E4M3: 448.0, E5M2: 57344.0}


def listed():
    return [
        # one token of a serving loop: sigmoid scores, a bias for balance,
        # 4 of 8 groups, 8 of 256 experts; nothing but latency
        dict(name="route one token", op="route", T=1, E=256, k=8, groups=8, top_groups=4, group_top=2,
             score="sigmoid", bias=True, renorm=True, scale=2.5, dtype="f32", train=False, full=False),
        # a prompt of odd length in bf16: plain softmax, 8 of 128
        dict(name="route a prompt", op="route", T=4133, E=128, k=8, groups=1, top_groups=1, group_top=1,
             score="softmax", bias=False, renorm=True, scale=1.0, dtype="bf16", train=False, full=False),
        # a training step: forward, all scores for the balance loss, and the
        # gradient of the logits
        dict(name="route a training batch", op="route", T=32768, E=256, k=8, groups=8, top_groups=4, group_top=2,
             score="sigmoid", bias=True, renorm=True, scale=2.5, dtype="bf16", train=True, full=True),
        # the order of 16 tokens' rows over 256 experts, as a decoding step takes it
        dict(name="order a few tokens", op="order", T=16, E=256, k=8, align=1, H=0),
        # a training batch ordered by expert and gathered into the 8-bit
        # operand of the product and the transposed one its weight gradient reads
        dict(name="order and gather a batch", op="order", T=16384, E=32, k=4, align=128, H=2048),
        # the experts' rows summed back to their tokens, and the weights' gradient
        dict(name="combine a batch", op="combine", T=8192, E=64, k=8, H=2048, train=True),
        # 8 tokens, 4 of 32 experts: the weights' bytes are all there is
        dict(name="experts for 8 tokens", op="product", T=8, E=32, k=4, N=4096, K=2048, a="e4m3", align=1),
        # a short prompt over few experts, odd segments
        dict(name="experts for a prompt", op="product", T=1021, E=8, k=2, N=1792, K=1024, a="e4m3", align=1),
        # a training batch, forward: aligned segments, many rows per expert
        dict(name="experts for a batch", op="product", T=16384, E=32, k=4, N=4096, K=2048, a="e4m3", align=128),
        # the experts' weight gradients of a training batch from 8-bit operands
        dict(name="experts' weight gradients", op="wgrad", T=8192, E=16, k=4, N=2048, K=2048, a="e5m2"),
        # the gate of a decoding step's rows: operand of the next product only
        dict(name="gate for 32 rows", op="gate", R=32, F=2048, train=False),
        # the gate of a training batch: both operands, the 8-bit checkpoint,
        # and the backward pass that reads it
        dict(name="gate for a training batch", op="gate", R=32768, F=2048, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route", "order", "combine", "product", "product", "wgrad", "gate"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        per = rng.randint(3, 256 // groups)
        E = groups * per
        top = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(8, top * per)), groups=groups,
                    top_groups=top, group_top=rng.choice((1, 2)), score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                    dtype=rng.choice(("f32", "bf16")), train=rng.random() < 0.6, full=rng.random() < 0.3)
    E = rng.choice((8, 16, 24, 32, 48, 64))
    k = rng.randint(1, 6)
    if op == "order":
        H = rng.choice((0, 32 * rng.randint(4, 64)))
        return dict(op=op, T=_log(rng, 1, 10000), E=E, k=k, align=128 if H else rng.choice((1, 32)), H=H)
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, H=8 * rng.randint(16, 256), train=rng.random() < 0.5)
    if op == "product":
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, N=16 * rng.randint(16, 192), K=128 * rng.randint(2, 16),
                    a=rng.choice(("e4m3", "e5m2")), align=rng.choice((1, 1, 128)))
    if op == "wgrad":
        return dict(op=op, T=_log(rng, 16, 8192), E=rng.choice((4, 8, 12, 16)), k=rng.randint(1, 4),
                    N=16 * rng.randint(16, 128), K=16 * rng.randint(16, 128), a=rng.choice(("e4m3", "e5m2")))
    return dict(op=op, R=32 * _log(rng, 1, 1024), F=32 * rng.randint(8, 64), train=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs --

def _capacity(T, k, E, align):
    n = T * k
    return -(-(n + min(E, n) * (align - 1)) // align) * align


def _chosen(g, T, E, k):
    """k different experts for each token, some experts asked for more than others."""
    score = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda") * 0.5
    return score.topk(k, dim=1).indices.to(torch.int32)


def _fp8(g, shape, dtype):
    """Codes and block exponents as the quantizer makes them of normal values:
    the largest of each 32 between half the format's maximum and all of it."""
    x = torch.randn(shape, generator=g, device="cuda")
    codes = (x * (FMAX[dtype] / 5.0)).clamp_(-FMAX[dtype], FMAX[dtype]).to(dtype)
    e = torch.randint(-12, -8, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.int32)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _order(ids, E, align, cap):
    """Rows of the choices ids [T, k] sorted by expert: first rows of the
    experts' segments (multiples of `align`), how many rows each has, the
    choice at each row (-1: none), the row of each choice."""
    n = ids.numel()
    flat = ids.reshape(-1).long()
    by, at = flat.sort(stable=True)
    counts = torch.zeros(E, dtype=torch.long, device=ids.device).scatter_add_(0, flat, torch.ones_like(flat))
    held = (counts + align - 1) // align * align
    offsets = torch.cat([held.new_zeros(1), held.cumsum(0)])
    before = counts.cumsum(0) - counts
    row = offsets[by] + torch.arange(n, device=ids.device) - before[by]
    rows = torch.full((cap,), -1, dtype=torch.int32, device=ids.device)
    rows[row] = at.to(torch.int32)
    pos = torch.empty(n, dtype=torch.int32, device=ids.device)
    pos[at] = row.to(torch.int32)
    return offsets.to(torch.int32), counts.to(torch.int32), rows, pos.view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    op = case["op"]
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}[case["dtype"]]
        s["logits"] = (torch.randn(T, E, generator=g, device="cuda") * 1.5).to(dt)
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.1 if case["bias"] else None
        s["ids"], s["weights"] = new((T, k), torch.int32), new((T, k), torch.float32)
        s["scores"] = new((T, E), torch.float32) if case["full"] else None
        if case["train"]:
            s["dweights"] = torch.randn(T, k, generator=g, device="cuda")
            s["dscores"] = torch.randn(T, E, generator=g, device="cuda") * 0.01 if case["full"] else None
            s["dlogits"] = new((T, E), dt)
    elif op in ("order", "combine"):
        T, E, k, H = case["T"], case["E"], case["k"], case["H"]
        align = case.get("align", 1)
        s["choice"] = _chosen(g, T, E, k)
        s["cap"] = cap = _capacity(T, k, E, align)
        if op == "order":
            s["offsets"], s["counts"] = new(E + 1, torch.int32), new(E, torch.int32)
            s["rows"], s["pos"] = new(cap, torch.int32), new((T, k), torch.int32)
            s["space"] = new(max(16, 4 * E * (min(256, -(-T * k // 1024)) + 1)), torch.uint8)
            if H:
                s["x"] = torch.randn(T, H, generator=g, device="cuda").bfloat16()
                s["codes"], s["scales"] = new((cap, H), E4M3), new((cap, H // 32), torch.float8_e8m0fnu)
                s["codes_t"], s["scales_t"] = new((H, cap), E4M3), new((H, cap // 32), torch.float8_e8m0fnu)
        else:
            s["pos"] = _order(s["choice"], E, 1, cap)[3]
            s["y"] = torch.randn(cap, H, generator=g, device="cuda").bfloat16()
            s["weights"] = torch.rand(T, k, generator=g, device="cuda")
            s["out"] = new((T, H), torch.bfloat16)
            if case["train"]:
                s["dout"] = torch.randn(T, H, generator=g, device="cuda").bfloat16()
                s["dweights"] = new((T, k), torch.float32)
    elif op in ("product", "wgrad"):
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        align = case.get("align", 128)
        s["cap"] = cap = _capacity(T, k, E, align)
        s["offsets"], counts, s["rows"], _ = _order(_chosen(g, T, E, k), E, align, cap)
        # the program knows the longest segment it plans for
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
        a = {"e4m3": E4M3, "e5m2": E5M2}[case["a"]]
        if op == "product":
            s["a"], s["a_scales"] = _fp8(g, (T, K), a)
            s["b"], s["b_scales"] = _fp8(g, (E, N, K), E4M3)
            s["out"] = new((cap, N), torch.bfloat16)
        else:
            hole = (s["rows"] < 0)[None, :]
            for n, width, dt in (("dyt", N, a), ("xt", K, E4M3)):
                c, e = _fp8(g, (width, cap), dt)
                s[n] = torch.where(hole, torch.zeros((), dtype=torch.uint8, device="cuda"),
                                   c.view(torch.uint8)).view(dt)
                s[n + "_scales"] = e
            s["dW"] = new((E, N, K), torch.bfloat16)
    else:
        R, F = case["R"], case["F"]
        e8 = torch.float8_e8m0fnu
        s["gu"] = torch.randn(R, 2 * F, generator=g, device="cuda").bfloat16()
        s["h"], s["h_scales"] = new((R, F), E4M3), new((R, F // 32), e8)
        if case["train"]:
            s["ht"], s["ht_scales"] = new((F, R), E4M3), new((F, R // 32), e8)
            s["kept"], s["kept_scales"] = new((R, 2 * F), E4M3), new((R, 2 * F // 32), e8)
            s["dh"] = torch.randn(R, F, generator=g, device="cuda").bfloat16()
            s["dgu"] = new((R, 2 * F), torch.bfloat16)
    return s


# ------------------------------------------------------------ plain forms --

def _power(e):
    """2^e in 32 bits, made of its bits: torch.ldexp rounds its powers."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _quantize(x, dtype=E4M3):
    """Blocks of 32 along the last axis: the smallest E with max(amax, 1e-10)
    <= fmax 2^E, codes of x 2^-E.  Returns codes and E8M0 scales."""
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = b.abs().amax(-1).clamp_min(1e-10)
    m, e = torch.frexp(amax.double() / FMAX[dtype])  # in 64 bits: amax next to fmax 2^E
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127).to(torch.int32)
    codes = (b * _power(-e)[..., None]).clamp(-FMAX[dtype], FMAX[dtype]).to(dtype)
    return codes.view(x.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, scales):
    """codes 2^E of blocks of 32 along the last axis, in 32 bits (exact)."""
    b = codes.float().reshape(*scales.shape, 32)
    return (b * _power(scales.view(torch.uint8).int() - 127)[..., None]).view(codes.shape)


def _plain_route(s):
    # scores in 64 bits: a choice turns on values that lie next to each other
    x = s["logits"].double()
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    c = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        rank = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, rank, True)
        c = torch.where(keep[:, :, None], c.view(T, G, E // G), -math.inf).view(T, E)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    total = w.sum(1, keepdim=True)
    weights = (w / total if s["renorm"] else w) * s["scale"]
    out = {"ids": ids.to(torch.int32), "weights": weights.float()}
    if s["full"]:
        out["scores"] = p.float()
    if s["train"]:
        dw = s["dweights"].double() * s["scale"]
        if s["renorm"]:
            dw = (dw - (dw * (w / total)).sum(1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_(1, ids, dw)
        if s["dscores"] is not None:
            dp = dp + s["dscores"].double()
        dx = p * (dp - (p * dp).sum(1, keepdim=True)) if s["score"] == "softmax" else dp * p * (1.0 - p)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _plain_order(s):
    offsets, counts, rows, pos = _order(s["choice"], s["E"], s["align"], s["cap"])
    out = {"offsets": offsets, "counts": counts, "rows": rows, "pos": pos}
    if s["H"]:
        held = rows >= 0
        x = torch.where(held[:, None], s["x"].float()[rows.clamp_min(0).long() // s["k"]], 0.0)
        out["codes"], out["scales"] = _quantize(x)
        out["codes_t"], out["scales_t"] = _quantize(x.t().contiguous())
    return out


def _plain_combine(s):
    picked = s["y"].float()[s["pos"].long()]  # [T, k, H]
    out = {"out": (picked * s["weights"][:, :, None]).sum(1).bfloat16()}
    if s["train"]:
        out["dweights"] = (picked * s["dout"].float()[:, None, :]).sum(2)
    return out


def _segments(s):
    """For each expert the rows of its segment, padded to the longest, and which of them are there."""
    first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = first[:, None] + torch.arange(s["most"], device=first.device)
    return at.clamp_max(s["cap"] - 1), at < last[:, None]


def _plain_product(s):
    a, b = _values(s["a"], s["a_scales"]), _values(s["b"], s["b_scales"])
    at, there = _segments(s)
    row = s["rows"][at]
    there = there & (row >= 0)
    x = torch.where(there[:, :, None], a[row.clamp_min(0).long() // s["k"]], 0.0)  # [E, most, K]
    y = torch.bmm(x, b.transpose(1, 2).contiguous())
    r = torch.arange(s["cap"], device=at.device)
    e = torch.searchsorted(s["offsets"][1:].long().contiguous(), r, right=True)
    held = e < s["E"]
    e = e.clamp_max(s["E"] - 1)
    i = (r - s["offsets"].long()[e]).clamp(0, s["most"] - 1)
    return {"out": torch.where(held[:, None], y[e, i], 0.0).bfloat16()}


def _plain_wgrad(s):
    at, there = _segments(s)
    dy = torch.where(there[:, :, None], _values(s["dyt"], s["dyt_scales"]).t()[at], 0.0)  # [E, most, N]
    x = torch.where(there[:, :, None], _values(s["xt"], s["xt_scales"]).t()[at], 0.0)
    return {"dW": torch.bmm(dy.transpose(1, 2).contiguous(), x).bfloat16()}


def _plain_gate(s):
    F = s["F"]
    g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
    h = g / (1.0 + torch.exp(-g)) * u
    out = {}
    out["h"], out["h_scales"] = _quantize(h)
    if s["train"]:
        out["ht"], out["ht_scales"] = _quantize(h.t().contiguous())
        out["kept"], out["kept_scales"] = _quantize(s["gu"])
        kept = _values(out["kept"], out["kept_scales"])
        g, u, dh = kept[:, :F], kept[:, F:], s["dh"].float()
        p = 1.0 / (1.0 + torch.exp(-g))
        out["dgu"] = torch.cat([dh * u * p * (1.0 + g * (1.0 - p)), dh * g * p], 1).bfloat16()
    return out


# --------------------------------------------------------- the library's --

def _own(s):
    import block_scaled_precision_blockwise_amd as bsq

    op = s["op"]
    if op == "route":
        score = bsq.BSQ_SOFTMAX if s["score"] == "softmax" else bsq.BSQ_SIGMOID
        bsq.bsq_moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], scores=s["scores"],
                          groups=s["groups"], top_groups=s["top_groups"], group_top=s["group_top"], score=score,
                          renorm=s["renorm"], scale=s["scale"])
        out = {"ids": s["ids"], "weights": s["weights"]}
        if s["full"]:
            out["scores"] = s["scores"]
        if s["train"]:
            bsq.bsq_moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], dscores=s["dscores"],
                                       score=score, renorm=s["renorm"], scale=s["scale"])
            out["dlogits"] = s["dlogits"]
        return out
    if op == "order":
        bsq.bsq_moe_plan(s["choice"], s["offsets"], s["counts"], s["rows"], s["pos"], s["space"], align=s["align"])
        out = {n: s[n] for n in ("offsets", "counts", "rows", "pos")}
        if s["H"]:
            bsq.bsq_moe_gather_mx(s["x"], s["rows"], s["k"], s["codes"], s["scales"], s["codes_t"], s["scales_t"])
            out.update({n: s[n] for n in ("codes", "scales", "codes_t", "scales_t")})
        return out
    if op == "combine":
        bsq.bsq_moe_combine(s["y"], s["pos"], s["out"], weights=s["weights"])
        out = {"out": s["out"]}
        if s["train"]:
            bsq.bsq_moe_combine_backward(s["y"], s["pos"], s["dout"], s["dweights"])
            out["dweights"] = s["dweights"]
        return out
    if op == "product":
        bsq.bsq_moe_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"], s["offsets"], s["out"], rows=s["rows"],
                           k=s["k"])
        return {"out": s["out"]}
    if op == "wgrad":
        bsq.bsq_moe_wgrad(s["dyt"], s["dyt_scales"], s["xt"], s["xt_scales"], s["offsets"], s["dW"])
        return {"dW": s["dW"]}
    if not s["train"]:
        bsq.bsq_swiglu_mx(s["gu"], s["h"], s["h_scales"])
        return {"h": s["h"], "h_scales": s["h_scales"]}
    bsq.bsq_swiglu_mx(s["gu"], s["h"], s["h_scales"], s["ht"], s["ht_scales"], s["kept"], s["kept_scales"])
    bsq.bsq_swiglu_mx_backward(s["kept"], s["kept_scales"], s["dh"], s["dgu"])
    return {n: s[n] for n in ("h", "h_scales", "ht", "ht_scales", "kept", "kept_scales", "dgu")}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "order": _plain_order, "combine": _plain_combine, "product": _plain_product,
            "wgrad": _plain_wgrad, "gate": _plain_gate}[state["op"]](state)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * (4 if case["dtype"] == "f32" else 2)
        full = 4 * T * E * case["full"]
        n = b + 8 * T * k + full + 4 * E * case["bias"]
        if case["train"]:
            n += b + 4 * T * k + full
        return {"bytes": n, "flops": T * E * (20 if case["train"] else 10)}
    if op == "gate":
        n, train = case["R"] * case["F"], case["train"]
        mx = 1 + 1 / 32
        # gate and up in, the operand out; in training also its transposed
        # form and the checkpoint out, the checkpoint and dh in, the gradients out
        return {"bytes": n * (4 + mx + train * (mx + 2 * mx + 2 * mx + 2 + 4)), "flops": n * (12 + 20 * train)}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "order":
        n = 8 * T * k + 4 * _capacity(T, k, E, case["align"]) + 8 * E
        if case["H"]:
            n += 2 * T * case["H"] + 2 * T * k * case["H"] * (1 + 1 / 32)
        return {"bytes": n, "flops": 0}
    if op == "combine":
        H, train = case["H"], case["train"]
        return {"bytes": 2 * T * k * H + 2 * T * H + 8 * T * k + train * (2 * T * H + 4 * T * k),
                "flops": 2 * T * k * H * (1 + train)}
    N, K = case["N"], case["K"]
    mx = 1 + 1 / 32
    asked = E * (1.0 - (1.0 - 1.0 / E) ** (T * k))  # experts that some token chose
    if op == "product":
        return {"bytes": T * K * mx + asked * N * K * mx + 2 * T * k * N, "flops": 2 * T * k * N * K}
    return {"bytes": T * k * (N + K) * mx + 2 * E * N * K, "flops": 2 * T * k * N * K}


# ------------------------------------------------------- definition in 64 --

def _mx64(x, fmax, mantissa, least):
    """The 8-bit value and block scale of each number, from the format's
    definition: `mantissa` bits behind the leading one, the leading one not
    below 2^least, block scale the smallest power of two that holds the block."""
    def two_to(n):
        return ((n.long() + 1023) * 2 ** 52).view(torch.float64)

    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1).clamp_min(1e-10)
    E = torch.floor(torch.log2(top / fmax)).int() - 1
    for _ in range(3):
        E = torch.where(top > fmax * two_to(E), E + 1, E)
    v = b * two_to(-E)[..., None]
    step = two_to((torch.frexp(v)[1] - 1).clamp_min(least) - mantissa)
    return (torch.round(v / step) * step).reshape(x.shape), two_to(E)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x, k, G = s["logits"].double(), s["k"], s["groups"]
        soft = s["score"] == "softmax"
        p = torch.softmax(x, 1) if soft else torch.sigmoid(x)
        choice = p + (0.0 if s["bias"] is None else s["bias"].double())
        if G > 1:
            by_group = choice.unflatten(1, (G, -1))
            n = min(s["group_top"], by_group.shape[2])
            worth = by_group.topk(n, 2).values.sum(2)
            worst = worth.topk(s["top_groups"], 1).values[:, -1:]
            choice = by_group.masked_fill((worth < worst)[:, :, None], -math.inf).flatten(1)
        at = choice.topk(k, 1).indices
        picked = p.gather(1, at)
        weights = picked * s["scale"] / (picked.sum(1, keepdim=True) if s["renorm"] else 1.0)
        out = {"ids": None, "weights": weights}
        if s["full"]:
            out["scores"] = p
        if s["train"]:
            leaf = x.clone().requires_grad_(True)
            p = torch.softmax(leaf, 1) if soft else torch.sigmoid(leaf)
            picked = p.gather(1, at)
            w = picked * s["scale"] / (picked.sum(1, keepdim=True) if s["renorm"] else 1.0)
            loss = (w * s["dweights"].double()).sum()
            if s["dscores"] is not None:
                loss = loss + (p * s["dscores"].double()).sum()
            out["dlogits"], = torch.autograd.grad(loss, leaf)
        return out
    if op == "order":
        if not s["H"]:
            return None
        rows = _order(s["choice"], s["E"], s["align"], s["cap"])[2].long()
        x = s["x"].double()[rows.clamp_min(0) // s["k"]] * (rows >= 0)[:, None]
        codes, scales = _mx64(x, 448.0, 3, -6)
        codes_t, scales_t = _mx64(x.t().contiguous(), 448.0, 3, -6)
        return {"offsets": None, "counts": None, "rows": None, "pos": None, "codes": codes, "scales": scales,
                "codes_t": codes_t, "scales_t": scales_t}
    if op == "combine":
        out = torch.zeros(s["T"], s["H"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["T"], s["k"], dtype=torch.float64, device="cuda")
        for j in range(s["k"]):
            y = s["y"][s["pos"][:, j].long()].double()
            out += y * s["weights"][:, j:j + 1].double()
            if s["train"]:
                dw[:, j] = (y * s["dout"].double()).sum(1)
        return {"out": out, "dweights": dw} if s["train"] else {"out": out}

    def wide(codes, scales):
        return codes.double() * scales.float().double().repeat_interleave(32, -1)

    if op == "product":
        out = torch.zeros(s["cap"], s["N"], dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        a = wide(s["a"], s["a_scales"])
        for e in range(s["E"]):
            rows = s["rows"][ends[e]:ends[e + 1]].long()
            if rows.numel():
                x = a[rows.clamp_min(0) // s["k"]] * (rows >= 0)[:, None]
                out[ends[e]:ends[e + 1]] = x @ wide(s["b"][e], s["b_scales"][e]).t()
        return {"out": out}
    if op == "wgrad":
        ends = s["offsets"].tolist()
        dyt, xt = wide(s["dyt"], s["dyt_scales"]), wide(s["xt"], s["xt_scales"])
        return {"dW": torch.stack([dyt[:, ends[e]:ends[e + 1]] @ xt[:, ends[e]:ends[e + 1]].t()
                                   for e in range(s["E"])])}
    g, u = s["gu"].double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    out = dict(zip(("h", "h_scales"), _mx64(h, 448.0, 3, -6)))
    if s["train"]:
        out["ht"], out["ht_scales"] = _mx64(h.t().contiguous(), 448.0, 3, -6)
        out["kept"], out["kept_scales"] = _mx64(s["gu"].double(), 448.0, 3, -6)
        g, u = (out["kept"] * out["kept_scales"].repeat_interleave(32, 1)).chunk(2, 1)
        p, dh = torch.sigmoid(g), s["dh"].double()
        out["dgu"] = torch.cat([dh * u * (p + g * p * (1.0 - p)), dh * g * p], 1)
    return out
