"""Cases and plain forms of the int8 linear operators and of the token scores.

Four operators: the int8 product with a scale for each token and channel ("linear": float activations
are quantized within the call), its input gradient ("grad"), the log probabilities of given tokens
with entropy and top alternatives ("score"), and the same with its gradient ("loss").
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
IGNORE = -100


def listed():
    return [
        # one decoded token through a small square projection: launch latency
        {"name": "linear m1 2048x2048", "op": "linear", "m": 1, "n": 2048, "k": 2048, "dtype": "bf16", "out": "bf16",
         "bias": False, "pad": 0},
        # four decoded tokens through a fused Q/K/V projection: the weight's bytes
        {"name": "linear m4 12288x4096", "op": "linear", "m": 4, "n": 12288, "k": 4096, "dtype": "bf16", "out": "bf16",
         "bias": False, "pad": 0},
        # a serving batch of 32 sequences through a down projection
        {"name": "linear m32 4096x11008", "op": "linear", "m": 32, "n": 4096, "k": 11008, "dtype": "f16", "out": "f16",
         "bias": False, "pad": 0},
        # a short prompt, with a bias
        {"name": "linear m512 8192x2048", "op": "linear", "m": 512, "n": 8192, "k": 2048, "dtype": "bf16", "out": "bf16",
         "bias": True, "pad": 0},
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
        # four decoded tokens, the alternatives that an answer shows
        {"name": "score m4 v128256 top20", "op": "score", "m": 4, "v": 128256, "dtype": "f32", "top": 20,
         "masked": 0.0, "pad": 0, "temperature": 0.7},
        # the tokens of prompts, scored
        {"name": "score m2048 v128256 top5", "op": "score", "m": 2048, "v": 128256, "dtype": "bf16", "top": 5,
         "masked": 0.0, "pad": 0, "temperature": 1.0},
        # a training loss with an entropy term
        {"name": "loss m2048 v128256", "op": "loss", "m": 2048, "v": 128256, "dtype": "bf16", "top": 0, "masked": 0.0,
         "pad": 0, "temperature": 1.0},
        # an odd vocabulary under a grammar's mask, rows of a wider buffer, a distillation term on the alternatives
        {"name": "loss ragged f32 masked", "op": "loss", "m": 331, "v": 32003, "dtype": "f32", "top": 8,
         "masked": 0.4, "pad": 5, "temperature": 1.3},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grad", "score", "loss"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("linear", "grad"):
        n, k = _log(rng, 512, 16384), _log(rng, 512, 16384)
        if rng.random() < 0.5:  # model widths are multiples of 64 more often than not
            n, k = max(512, n // 64 * 64), max(512, k // 64 * 64)
        if op == "linear":
            m = _log(rng, 1, max(1, min(4096, 4096 * 11008 * 4096 // (n * k))))
            return {"op": op, "m": m, "n": n, "k": k, "dtype": dt, "out": dt, "bias": rng.random() < 0.5,
                    "pad": rng.choice([0, 0, 0, 8, 3])}
        dt = rng.choice(["bf16", "f16"])
        m = _log(rng, 16, max(16, min(4096, 2048 * 4096 * 11008 // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dt, "out": dt}
    v = _log(rng, 8192, 131072)
    m = _log(rng, 1, max(1, 1024 * 128256 // v))
    return {"op": op, "m": m, "v": v, "dtype": dt, "top": rng.choice([0, 1, 5, 20] if op == "score" else [0, 8]),
            "masked": rng.choice([0.0, 0.0, 0.4]), "pad": rng.choice([0, 0, 5]),
            "temperature": rng.choice([1.0, 0.7, 1.3])}


def _rand(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _wider(x, pad):
    """x as the first columns of rows that are `pad` longer."""
    if not pad:
        return x
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _weight(g, n, k):
    """A channel-quantized weight as a program keeps it: int8 codes in rows padded with zeros to 64
    columns, and the channels' fp32 scales."""
    w = _rand(g, n, k) * 0.02 * torch.exp(0.3 * _rand(g, n, 1))
    scales = w.abs().amax(1).div(torch.full((n,), 127.0, device="cuda"))
    codes = torch.zeros(n, (k + 63) // 64 * 64, dtype=torch.int8, device="cuda")
    codes[:, :k] = torch.round(w * scales.reciprocal().unsqueeze(1)).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("linear", "grad"):
        m, n, k, dt = case["m"], case["n"], case["k"], DT[case["dtype"]]
        s["codes"], s["scales"] = _weight(g, n, k)
        if case["op"] == "linear":
            x = _rand(g, m, k) * torch.exp(0.5 * _rand(g, m, 1))
            x = x * torch.where(torch.rand(k, device="cuda", generator=g) < 0.01, 8.0, 1.0)  # outlier channels
            s["x"] = _wider(x.to(dt), case["pad"])
            s["bias"] = (_rand(g, n) * 0.1).to(DT[case["out"]]) if case["bias"] else None
        else:
            s["dy"] = (_rand(g, m, n) * 0.05 * torch.exp(_rand(g, m, 1))).to(dt)
        return s
    m, v = case["m"], case["v"]
    z = _rand(g, m, v) * 2.5
    z += 6.0 * (torch.rand(m, v, device="cuda", generator=g) < 12.0 / v)  # a few likely continuations
    if case["masked"]:
        z.masked_fill_(torch.rand(m, v, device="cuda", generator=g) < case["masked"], -math.inf)
        z[m // 2] = -math.inf  # a row whose mask leaves nothing
    s["logits"] = _wider(z.to(DT[case["dtype"]]), case["pad"])
    del z
    t = torch.randint(0, v, (m,), device="cuda", generator=g)
    if m > 8:
        t[torch.rand(m, device="cuda", generator=g) < 0.05] = IGNORE  # padding
    s["targets"] = t
    if case["op"] == "loss":
        s["grads"] = [-torch.rand(m, device="cuda", generator=g), 0.01 * _rand(g, m)]
        if case["top"]:
            s["grads"].append(0.1 * _rand(g, m, case["top"]))
    return s


# ---------------------------------------------------------------- plain forms (fp32, rounded once)

TINY = 2.0 ** -126  # the least scale: the smallest normal number, whose reciprocal is finite


def _plain_linear(s):
    x = s["x"].float()
    sx = torch.clamp(x.abs().amax(1).div(torch.full((x.shape[0],), 127.0, device=x.device)), min=TINY)
    q = torch.round(x * sx.reciprocal().unsqueeze(1))
    y = (q @ s["codes"][:, :s["k"]].float().t()) * sx.unsqueeze(1) * s["scales"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(DT[s["out"]])


def _plain_grad(s):
    w = s["codes"][:, :s["k"]].float() * s["scales"].unsqueeze(1)
    return (s["dy"].float() @ w).to(DT[s["out"]])


def _plain_scores(s):
    """(logprobs, entropy, top logprobs, top ids, log-sum-exp, scaled logits), all rows."""
    z = s["logits"]
    v = z.shape[1]
    u = z.float() * (1.0 / s["temperature"])
    mx = u.amax(1)
    empty = mx == -math.inf
    d = u - torch.where(empty, torch.zeros_like(mx), mx).unsqueeze(1)
    e = torch.exp(d)
    total = torch.where(empty, torch.ones_like(mx), e.sum(1))
    logs = torch.log(total)
    ent = logs - (e * torch.clamp(d, min=-1e4)).sum(1) / total
    ent = torch.where(empty, torch.zeros_like(ent), ent)
    lse = torch.where(empty, torch.zeros_like(mx), mx + logs)
    t = s["targets"]
    lp = u.gather(1, t.clamp(0, v - 1).unsqueeze(1)).squeeze(1) - lse
    lp = torch.where((t < 0) | (t >= v), torch.full_like(lp, math.nan), lp)
    lp = torch.where(t == IGNORE, torch.zeros_like(lp), lp)
    top_lp = torch.empty(z.shape[0], 0, device=z.device)
    ids = torch.empty(z.shape[0], 0, dtype=torch.int64, device=z.device)
    if s["top"]:
        # one whole number for each logit, ordered by value and then by the lower index
        b = z.float().view(torch.int32).to(torch.int64)
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        key = b * (1 << 20) + (v - 1 - torch.arange(v, device=z.device))
        ids = v - 1 - (key.topk(s["top"], dim=1).values & ((1 << 20) - 1))
        top_lp = u.gather(1, ids) - lse.unsqueeze(1)
    return lp, ent, top_lp, ids, lse, u


def _plain_loss(s):
    lp, ent, top_lp, ids, lse, u = _plain_scores(s)
    v = u.shape[1]
    t = s["targets"]
    g = torch.where(t == IGNORE, torch.zeros_like(lp), s["grads"][0])
    h = s["grads"][1]
    all_g = g + (s["grads"][2].sum(1) if s["top"] else 0.0)
    r = u - lse.unsqueeze(1)
    d = -torch.exp(r) * (all_g.unsqueeze(1) + h.unsqueeze(1) * (torch.clamp(r, min=-1e4) + ent.unsqueeze(1)))
    d.scatter_add_(1, t.clamp(0, v - 1).unsqueeze(1), g.unsqueeze(1))
    if s["top"]:
        d.scatter_add_(1, ids, s["grads"][2])
    d = d * (1.0 / s["temperature"])
    d = torch.where((u.amax(1) == -math.inf).unsqueeze(1), torch.zeros_like(d), d)
    return {"logprobs": lp, "entropy": ent, "top": top_lp, "ids": ids, "dlogits": d.to(s["logits"].dtype)}


# ---------------------------------------------------------------- the framework's operators


def _own_run(s):
    import gemv_int4_quantize_amd as w4

    if s["op"] == "linear":
        w = w4.Int8Rows(s["codes"], s["scales"], s["n"], s["k"])
        return w4.mm_int8(s["x"], w, bias=s["bias"], out_dtype=DT[s["out"]])
    if s["op"] == "grad":
        w = w4.Int8Rows(s["codes"], s["scales"], s["n"], s["k"])
        return w4.mm_int8_t(s["dy"], w, out_dtype=DT[s["out"]])
    if s["op"] == "score":
        r = w4.token_logprobs(s["logits"], s["targets"], top=s["top"], temperature=s["temperature"], ignore_index=IGNORE)
        return {"logprobs": r.logprobs, "entropy": r.entropy, "top": r.top_logprobs, "ids": r.top_ids}
    z = s["logits"].detach().requires_grad_()
    r = w4.token_logprobs(z, s["targets"], top=s["top"], temperature=s["temperature"], ignore_index=IGNORE)
    outs = [r.logprobs, r.entropy] + ([r.top_logprobs] if s["top"] else [])
    (dz,) = torch.autograd.grad(outs, z, s["grads"])
    return {"logprobs": r.logprobs.detach(), "entropy": r.entropy.detach(), "top": r.top_logprobs.detach(),
            "ids": r.top_ids, "dlogits": dz}


def run(state):
    if own:
        return _own_run(state)
    if state["op"] == "linear":
        return _plain_linear(state)
    if state["op"] == "grad":
        return _plain_grad(state)
    if state["op"] == "score":
        lp, ent, top_lp, ids, _, _ = _plain_scores(state)
        return {"logprobs": lp, "entropy": ent, "top": top_lp, "ids": ids}
    return _plain_loss(state)


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "linear":
        m, n, k, o = case["m"], case["n"], case["k"], SIZE[case["out"]]
        return {"bytes": m * k * b + n * k + 4 * n + m * n * o + (n * o if case["bias"] else 0), "flops": 2 * m * n * k}
    if case["op"] == "grad":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * n * b + n * k + 4 * n + m * k * SIZE[case["out"]], "flops": 2 * m * n * k}
    m, v, top = case["m"], case["v"], case["top"]
    rows = m * (8 + 8 + 12 * top)  # targets, logprobs and entropy, alternatives
    if case["op"] == "score":
        return {"bytes": m * v * b + rows, "flops": 6 * m * v}
    return {"bytes": 2 * m * v * b + rows + m * (8 + 4 * top), "flops": 14 * m * v}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_rows(x):
    """Codes and scales of rows of real numbers: the scale takes the largest magnitude to 127, and a
    code is the nearest whole number of scales (ties to even)."""
    top = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
    scale = torch.maximum(top / 127.0, torch.full_like(top, TINY))
    return (x / scale[:, None]).round(), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        q, sx = _exact_rows(s["x"].double())
        w = s["codes"].double()[:, :case["k"]] * s["scales"].double()[:, None]
        y = torch.mm(q * sx[:, None], w.t())
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "grad":
        return torch.mm(s["dy"].double() * s["scales"].double()[None, :], s["codes"].double()[:, :case["k"]])
    z, t = s["logits"], s["targets"]
    m, v = z.shape
    out = {"logprobs": [], "entropy": [], "top": [], "ids": []}
    if case["op"] == "loss":
        out["dlogits"] = []
    step = max(1, (1 << 27) // v)
    for r in range(0, m, step):  # some rows at a time: 64 bits of all of them would be several copies of 2 GiB
        zr, tr = z[r:r + step].double(), t[r:r + step]
        u = zr / case["temperature"]
        live = torch.isfinite(u)
        some = live.any(dim=1)
        p = torch.softmax(torch.where(some[:, None], u, torch.zeros_like(u)), dim=1)
        lse = torch.where(some, torch.logsumexp(u, dim=1), torch.zeros_like(u[:, 0]))
        logp = u - lse[:, None]
        plogp = torch.where(live, p * logp, torch.zeros_like(p))
        ent = torch.where(some, -plogp.sum(dim=1), torch.zeros_like(lse))
        inside = (tr >= 0) & (tr < v)
        lp = logp[torch.arange(len(tr), device=z.device), torch.where(inside, tr, torch.zeros_like(tr))]
        out["logprobs"].append(torch.where(inside, lp, torch.zeros_like(lp)))
        out["entropy"].append(ent)
        ids = torch.sort(zr, dim=1, descending=True, stable=True).indices[:, :case["top"]] if case["top"] else \
            torch.empty(len(tr), 0, dtype=torch.int64, device=z.device)
        out["ids"].append(ids)
        out["top"].append(logp.gather(1, ids))
        if case["op"] == "loss":
            # the chain rule through log-softmax: d = c - p * sum(c), c the gradient of the log probabilities
            c = -(s["grads"][1][r:r + step].double())[:, None] * torch.where(live, p * (1.0 + logp), torch.zeros_like(p))
            g = torch.where(inside, s["grads"][0][r:r + step].double(), torch.zeros_like(lse))
            c = c + torch.zeros_like(c).scatter_(1, torch.where(inside, tr, torch.zeros_like(tr))[:, None], g[:, None])
            if case["top"]:
                c = c + torch.zeros_like(c).scatter_(1, ids, s["grads"][2][r:r + step].double())
            d = (c - p * c.sum(dim=1, keepdim=True)) / case["temperature"]
            out["dlogits"].append(torch.where(some[:, None], d, torch.zeros_like(d)))
    return {k: torch.cat(a) for k, a in out.items()}
