"""Cases and plain forms of the microscaled 4-bit operators (MXFP4).

Four operators: rows to 4-bit floating point with a power of two for each 32 columns and back
("quantize"), the product of two such operands, float activations quantized within the call
("linear"), its input gradient ("grad"), and a whole mixture-of-experts layer with such weights for
a few tokens ("moe").
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32  # columns that share a power of two


def listed():
    return [
        # the activations of a serving batch, on their way to a product
        {"name": "quantize 64x4096 bf16", "op": "quantize", "m": 64, "k": 4096, "dtype": "bf16", "pad": 0},
        # a checkpoint's up projection, quantized once
        {"name": "quantize 11008x4096 bf16", "op": "quantize", "m": 11008, "k": 4096, "dtype": "bf16", "pad": 0},
        # one decoded token through a small square projection: launch latency
        {"name": "linear m1 2048x2048", "op": "linear", "m": 1, "n": 2048, "k": 2048, "dtype": "bf16", "out": "bf16",
         "bias": False, "pad": 0},
        # a serving batch of 32 sequences through a down projection
        {"name": "linear m32 4096x11008", "op": "linear", "m": 32, "n": 4096, "k": 11008, "dtype": "f16", "out": "f16",
         "bias": False, "pad": 0},
        # sizes that no tile divides, fp32 in and out, rows of a wider buffer
        {"name": "linear ragged f32", "op": "linear", "m": 259, "n": 1003, "k": 1555, "dtype": "f32", "out": "f32",
         "bias": True, "pad": 7},
        # a batch of long prompts through an up projection: the matrix cores
        {"name": "linear m4096 11008x4096", "op": "linear", "m": 4096, "n": 11008, "k": 4096, "dtype": "bf16",
         "out": "bf16", "bias": False, "pad": 0},
        # fine-tuning, backward through a down projection
        {"name": "grad m2048 4096x11008", "op": "grad", "m": 2048, "n": 4096, "k": 11008, "dtype": "bf16", "out": "bf16"},
        # backward with sizes that no tile divides
        {"name": "grad ragged f16", "op": "grad", "m": 131, "n": 2027, "k": 1030, "dtype": "f16", "out": "f16"},
        # one decoded token, many small experts
        {"name": "moe t1 e128 k8", "op": "moe", "t": 1, "e": 128, "top": 8, "h": 2048, "f": 768, "dtype": "bf16",
         "ldt": "f32", "masked": 0.0, "renorm": True},
        # four sequences, two of eight large experts each: the weights' bytes
        {"name": "moe t4 e8 k2", "op": "moe", "t": 4, "e": 8, "top": 2, "h": 4096, "f": 11008, "dtype": "bf16",
         "ldt": "bf16", "masked": 0.0, "renorm": True},
        # a serving batch of 32 sequences that reaches nearly all experts
        {"name": "moe t32 e128 k8", "op": "moe", "t": 32, "e": 128, "top": 8, "h": 2048, "f": 768, "dtype": "bf16",
         "ldt": "f32", "masked": 0.0, "renorm": False},
        # odd sizes in fp32, experts that a mask takes out, a padding row without any
        {"name": "moe ragged f32 masked", "op": "moe", "t": 5, "e": 20, "top": 3, "h": 1003, "f": 700, "dtype": "f32",
         "ldt": "f32", "masked": 0.3, "renorm": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    n = _log(rng, lo, hi)
    return max(lo, n // 64 * 64) if rng.random() < 0.5 else n  # model widths are multiples of 64 more often than not


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "grad", "moe", "moe"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        k = _width(rng, 64, 16384)
        return {"op": op, "m": _log(rng, 1, 11008 * 4096 // k // (2 if dt == "f32" else 1)), "k": k, "dtype": dt,
                "pad": rng.choice([0, 0, 8, 3])}
    if op in ("linear", "grad"):
        n, k = _width(rng, 512, 16384), _width(rng, 512, 16384)
        if op == "linear":
            m = _log(rng, 1, max(1, min(4096, 4096 * 11008 * 4096 // (n * k))))
            return {"op": op, "m": m, "n": n, "k": k, "dtype": dt, "out": dt, "bias": rng.random() < 0.5,
                    "pad": rng.choice([0, 0, 0, 8, 3])}
        dt = rng.choice(["bf16", "f16"])
        m = _log(rng, 16, max(16, min(4096, 2048 * 4096 * 11008 // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dt, "out": dt}
    e = rng.choice([4, 8, 16, 60, 64, 128])
    top = rng.randint(1, min(e, 8))
    h, f = _width(rng, 256, 4096), _width(rng, 128, 8192)
    f = max(128, min(f, 8 * 4096 * 11008 // (e * h)))
    t = _log(rng, 1, max(1, min(64, 32 * 8 * 2048 * 768 // (top * h * f))))
    return {"op": op, "t": t, "e": e, "top": top, "h": h, "f": f, "dtype": dt, "ldt": rng.choice(["f32", dt]),
            "masked": rng.choice([0.0, 0.0, 0.3]), "renorm": rng.random() < 0.7}


def _rand(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _wider(x, pad):
    """x as the first columns of rows that are `pad` longer."""
    if not pad:
        return x
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _pitch(k):
    return (k + 127) // 128 * 128


def _weight(g, n, k):
    """A microscaled weight as a program keeps it: codes [n][P / 2], the even column in the low four
    bits, and exponents [n][P / 32] (127 above the power of two), P = k rounded up to 128."""
    codes = torch.zeros(n, _pitch(k) // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, _pitch(k) // BLOCK, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // _pitch(k))
    for r in range(0, n, step):
        m = min(step, n - r)
        w = torch.zeros(m, _pitch(k), device="cuda")
        w[:, :k] = _rand(g, m, k) * 0.02 * torch.exp(0.3 * _rand(g, m, 1))
        mag, ex = _blocks(w)
        c = torch.bucketize(mag, torch.tensor([0.25, 1.25, 2.5, 5.0], device="cuda")).add_(
            torch.bucketize(mag, torch.tensor([0.75, 1.75, 3.5], device="cuda"), right=True)).to(torch.uint8)
        c = (c | (w < 0).to(torch.uint8) << 3).view(m, -1, 2)
        codes[r:r + m] = c[:, :, 0] | c[:, :, 1] << 4
        scales[r:r + m] = ex
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dt = DT[case["dtype"]]
    if case["op"] in ("quantize", "linear"):
        m, k = case["m"], case["k"]
        x = _rand(g, m, k) * torch.exp(0.5 * _rand(g, m, 1))
        x = x * torch.where(torch.rand(k, device="cuda", generator=g) < 0.01, 8.0, 1.0)  # outlier channels
        s["x"] = _wider(x.to(dt), case["pad"])
    if case["op"] in ("linear", "grad"):
        s["codes"], s["scales"] = _weight(g, case["n"], case["k"])
    if case["op"] == "linear":
        s["bias"] = (_rand(g, case["n"]) * 0.1).to(DT[case["out"]]) if case["bias"] else None
    if case["op"] == "grad":
        s["dy"] = (_rand(g, case["m"], case["n"]) * 0.05 * torch.exp(_rand(g, case["m"], 1))).to(dt)
    if case["op"] == "moe":
        t, e, h, f = case["t"], case["e"], case["h"], case["f"]
        s["w1"] = _weight(g, e * 2 * f, h)  # each expert's gate rows, then its up rows
        s["w2"] = _weight(g, e * h, f)
        s["x"] = _rand(g, t, h).to(dt)
        z = _rand(g, t, e) * 1.5
        if case["masked"]:
            z.masked_fill_(torch.rand(t, e, device="cuda", generator=g) < case["masked"], -math.inf)
            if t > 1:
                z[t // 2] = -math.inf  # a padding row
        s["logits"] = z.to(DT[case["ldt"]])
    return s


# ---------------------------------------------------------------- plain forms (fp32, rounded once)


def _power(ex):
    """2^(ex - 127) of exponents 0 .. 254 in fp32."""
    ex = ex.to(torch.int32)
    return torch.where(ex == 0, torch.full_like(ex, 1 << 22), ex << 23).view(torch.float32)


def _blocks(w):
    """Magnitudes of w [m][P] in fp32, as multiples of their block's power of two, and the exponents:
    the power of two takes the block's largest magnitude to [4, 8)."""
    a = w.abs().view(w.shape[0], -1, BLOCK)
    ex = ((a.amax(2).view(torch.int32) >> 23) - 2).clamp_(min=0)
    # by two factors: the inverse of the smallest power is above fp32's largest
    half = _power(127 - (ex - 127) // 2)
    rest = _power(127 - (ex - 127) + (ex - 127) // 2)
    return (a * half.unsqueeze(2) * rest.unsqueeze(2)).view(w.shape), ex.to(torch.uint8)


def _plain_round(x):
    """The fp32 values that the codes of rows x stand for."""
    m, k = x.shape
    w = torch.nn.functional.pad(x.float(), (0, _pitch(k) - k))
    mag, ex = _blocks(w)
    # steps of 1/2 below 2, 1 below 4, 2 above, ties to the even code, at most 6
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(mag / step) * step, max=6.0)
    q = torch.copysign(q, w).view(m, -1, BLOCK) * _power(ex).unsqueeze(2)
    return q.view(m, -1)[:, :k]


def _plain_values(codes, scales):
    """The fp32 values of codes [..][P / 2] with exponents [..][P / 32]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    c = torch.stack([codes & 15, codes >> 4], -1).to(torch.int32)
    v = table[c].view(*scales.shape, BLOCK) * _power(scales).unsqueeze(-1)
    return v.view(*codes.shape[:-1], -1)


def _plain_linear(s):
    y = _plain_round(s["x"]) @ _plain_values(s["codes"], s["scales"])[:, :s["k"]].t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(DT[s["out"]])


def _plain_grad(s):
    w = _plain_values(s["codes"], s["scales"])[:, :s["k"]]
    return (s["dy"].float() @ w).to(DT[s["out"]])


def _plain_moe(s):
    t, e, top, h, f = s["t"], s["e"], s["top"], s["h"], s["f"]
    z = s["logits"].float()
    # one whole number for each logit, ordered by value and then by the lower index
    b = z.view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    ids = e - 1 - ((b * 1024 + (e - 1 - torch.arange(e, device=z.device))).topk(top, dim=1).values & 1023)
    mx = z.amax(1, keepdim=True)
    p = torch.exp(z - torch.where(mx == -math.inf, torch.zeros_like(mx), mx))
    some = p.gather(1, ids)
    total = (some if s["renorm"] else p).sum(1, keepdim=True)
    g = some / torch.where(total == 0, torch.ones_like(total), total)
    sel = ids.reshape(-1)  # the experts of t * top pairs
    x = s["x"].float().repeat_interleave(top, 0).unsqueeze(2)
    w1c, w1s = s["w1"][0].view(e, 2 * f, -1)[sel], s["w1"][1].view(e, 2 * f, -1)[sel]
    u = (_plain_values(w1c, w1s)[:, :, :h] @ x).squeeze(2)
    a = u[:, :f] / (1.0 + torch.exp(-u[:, :f])) * u[:, f:]
    w2c, w2s = s["w2"][0].view(e, h, -1)[sel], s["w2"][1].view(e, h, -1)[sel]
    y = (_plain_values(w2c, w2s)[:, :, :f] @ a.unsqueeze(2)).squeeze(2)
    return (y.view(t, top, h) * g.unsqueeze(2)).sum(1).to(DT[s["dtype"]])


# ---------------------------------------------------------------- the framework's operators


def _own_run(s):
    import gemv_int4_quantize_amd as w4

    if s["op"] == "quantize":
        return w4.dequantize_mxfp4(w4.quantize_mxfp4(s["x"]), s["x"].dtype)
    if s["op"] == "linear":
        w = w4.MXFP4Rows(s["codes"], s["scales"], s["n"], s["k"])
        return w4.mm_mxfp4(s["x"], w, bias=s["bias"], out_dtype=DT[s["out"]])
    if s["op"] == "grad":
        w = w4.MXFP4Rows(s["codes"], s["scales"], s["n"], s["k"])
        return w4.mm_mxfp4_t(s["dy"], w, out_dtype=DT[s["out"]])
    w1 = w4.MXFP4Rows(*s["w1"], s["e"] * 2 * s["f"], s["h"])
    w2 = w4.MXFP4Rows(*s["w2"], s["e"] * s["h"], s["f"])
    return w4.moe_mxfp4(s["x"], s["logits"], w1, w2, s["top"], renormalize=s["renorm"])


def run(state):
    if own:
        return _own_run(state)
    if state["op"] == "quantize":
        return _plain_round(state["x"]).to(state["x"].dtype)
    if state["op"] == "linear":
        return _plain_linear(state)
    if state["op"] == "grad":
        return _plain_grad(state)
    return _plain_moe(state)


def _row_bytes(k):
    return k / 2 + (k + BLOCK - 1) // BLOCK


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "quantize":
        m, k = case["m"], case["k"]  # the codes are written, and the values that they stand for
        return {"bytes": int(2 * m * k * b + m * _row_bytes(k)), "flops": 4 * m * k}
    if case["op"] == "linear":
        m, n, k, o = case["m"], case["n"], case["k"], SIZE[case["out"]]
        return {"bytes": int(m * k * b + n * _row_bytes(k) + m * n * o + (n * o if case["bias"] else 0)),
                "flops": 2 * m * n * k}
    if case["op"] == "grad":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": int(m * n * b + n * _row_bytes(k) + m * k * SIZE[case["out"]]), "flops": 2 * m * n * k}
    t, e, top, h, f = case["t"], case["e"], case["top"], case["h"], case["f"]
    live = max(1, t - 1) if case["masked"] else t
    experts = e * (1.0 - (1.0 - top / e) ** live)  # that some token is expected to reach
    return {"bytes": int(experts * (2 * f * _row_bytes(h) + h * _row_bytes(f)) + 2 * t * h * b + t * e * SIZE[case["ldt"]]),
            "flops": live * top * 6 * h * f}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_power(n):
    """2^n of whole numbers n, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_rows(x):
    """What the codes of rows x (64 bits) stand for: each block of 32 in multiples of the power of
    two that is two below its largest magnitude's, the nearest of the eight magnitudes."""
    m, k = x.shape
    out = torch.empty_like(x)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    for c in range(0, k, BLOCK):
        v = x[:, c:c + BLOCK]
        top = v.abs().amax(dim=1, keepdim=True)
        exponent = torch.clamp(torch.frexp(top).exponent - 1 - 2, min=-127)
        exponent = torch.where(top == 0, torch.full_like(exponent, -127), exponent)
        unit = _exact_power(exponent)
        mag = v.abs() / unit
        low = torch.searchsorted(mids, mag.contiguous())  # at a midpoint: the magnitude below
        tie = (low < 7) & (mag == mids[low.clamp(max=6)]) & (low % 2 == 1)
        out[:, c:c + BLOCK] = grid[low + tie] * unit * torch.sign(v)
    return out


def _exact_values(codes, scales, k):
    """Codes one by one: sign, exponent and mantissa bits."""
    c = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    sign = 1.0 - 2.0 * (c // 8).double()
    exponent, mantissa = (c % 8) // 2, (c % 2).double()
    mag = torch.where(exponent == 0, mantissa * 0.5, (1.0 + mantissa * 0.5) * _exact_power(exponent - 1))
    unit = _exact_power(scales.to(torch.int64) - 127).repeat_interleave(BLOCK, dim=1)
    return (sign * mag * unit)[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_rows(s["x"].double())
    if case["op"] == "linear":
        y = torch.mm(_exact_rows(s["x"].double()), _exact_values(s["codes"], s["scales"], case["k"]).t())
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "grad":
        return torch.mm(s["dy"].double(), _exact_values(s["codes"], s["scales"], case["k"]))
    t, e, h, f = case["t"], case["e"], case["h"], case["f"]
    x, z = s["x"].double(), s["logits"].double()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]].cpu()
    y = torch.zeros(t, h, dtype=torch.float64, device=x.device)
    for expert in sorted(set(order.flatten().tolist())):
        rows = [r for r in range(t) if expert in order[r].tolist() and z[r, expert] > -math.inf]
        if not rows:
            continue
        (c1, e1), (c2, e2) = s["w1"], s["w2"]
        w = _exact_values(c1[expert * 2 * f:(expert + 1) * 2 * f], e1[expert * 2 * f:(expert + 1) * 2 * f], h)
        u = torch.mm(x[rows], w.t())
        a = u[:, :f] * torch.sigmoid(u[:, :f]) * u[:, f:]
        out = torch.mm(a, _exact_values(c2[expert * h:(expert + 1) * h], e2[expert * h:(expert + 1) * h], f).t())
        for i, r in enumerate(rows):
            of = z[r, order[r].to(z.device)] if case["renorm"] else z[r]
            y[r] += torch.exp(z[r, expert] - torch.logsumexp(of, 0)) * out[i]
    return y
