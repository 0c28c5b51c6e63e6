"""The measured cases of the 8-bit linear layer and of the distillation loss.

Each case goes through one operator as a program that trains or serves a
low-precision student calls it. `run` computes the operators in elementary torch
operations in 32 bits, or, where `own` is set, calls the framework. `exact`
computes the same definitions in 64 bits."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # activations of a 4096-token batch, quantized per token
        {"name": "quantize tokens", "op": "quantize", "rows": 4096, "cols": 4096, "pad": 0, "dtype": "bf16",
         "fold": False, "transpose": False},
        # an odd gradient (a strided slice) quantized per channel for a weight gradient, levels transposed
        {"name": "quantize channels odd", "op": "quantize", "rows": 1021, "cols": 5003, "pad": 5, "dtype": "f32",
         "fold": True, "transpose": True},
        # one token of one sequence through a layer: the latency of serving
        {"name": "linear one token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16", "bias": False},
        # a few sequences decoded together, an odd width
        {"name": "linear 24 tokens odd", "op": "linear", "m": 24, "n": 5001, "k": 2048, "dtype": "f16", "bias": True},
        # a prompt through a wide layer
        {"name": "linear prompt", "op": "linear", "m": 2048, "n": 16384, "k": 4096, "dtype": "bf16", "bias": True},
        # one layer's forward and backward over a training batch
        {"name": "train layer", "op": "train", "m": 8192, "n": 4096, "k": 4096, "dtype": "bf16", "bias": False},
        # the same with sizes that no tile divides
        {"name": "train layer odd", "op": "train", "m": 1000, "n": 777, "k": 1537, "dtype": "f32", "bias": True},
        # the plain product of levels, ragged, into fp32
        {"name": "product ragged", "op": "matmul", "m": 515, "n": 4099, "k": 2064, "dtype": "f32", "bias": False},
        # the largest product
        {"name": "product 8192", "op": "matmul", "m": 8192, "n": 8192, "k": 8192, "dtype": "bf16", "bias": False},
        # the loss of a few validation positions, odd vocabulary, no gradient
        {"name": "distill loss few rows", "op": "distill", "rows": 7, "vocab": 50021, "k": 20, "pad": 0, "dtype": "f32",
         "tail": False, "tau": 1.0},
        # loss, then its gradient in a call of its own (the loss is reweighted between them)
        {"name": "distill two calls odd", "op": "distill_pair", "rows": 1531, "vocab": 32003, "k": 32, "pad": 13,
         "dtype": "bf16", "tail": False, "tau": 2.0},
        # a training step's loss and gradient over a large vocabulary, with the teacher's remaining mass
        {"name": "distill step large", "op": "distill_step", "rows": 4096, "vocab": 131072, "k": 64, "pad": 0,
         "dtype": "bf16", "tail": True, "tau": 1.0},
    ]


def _log_int(rng, lo, hi, even):
    """A size between lo and hi, uniform in its logarithm; with `even`, rounded to what layers usually have."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if even and v > 64:
        v = (v + 32) // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "linear", "train", "matmul", "distill", "distill_pair", "distill_step"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    even = rng.random() < 0.5
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 8192, even), "cols": _log_int(rng, 1, 8192, even),
                "pad": rng.choice([0, 0, 3, 64]), "dtype": dtype, "fold": rng.random() < 0.5,
                "transpose": rng.random() < 0.5}
    if op.startswith("distill"):
        vocab = _log_int(rng, 500, 131072, even)
        rows = min(_log_int(rng, 1, 4096, even), (1 << 27) // vocab)
        return {"op": op, "rows": rows, "vocab": vocab, "k": _log_int(rng, 1, 128, False),
                "pad": rng.choice([0, 0, 1, 32]), "dtype": dtype, "tail": rng.random() < 0.5,
                "tau": rng.choice([1.0, 2.0, 4.0])}
    n, k = _log_int(rng, 32, 8192, even), _log_int(rng, 32, 8192, even)
    m = min(_log_int(rng, 1, 8192, even), (1 << 36) // (n * k))
    return {"op": op, "m": m, "n": n, "k": k,
            "dtype": dtype, "bias": rng.random() < 0.5}


def _levels(gen, rows, cols):
    """Levels as a max-norm quantizer leaves them: normal, cut at 127."""
    v = torch.randn(rows, cols, generator=gen, device="cuda") * 32.0
    return v.round_().clamp_(-127, 127).to(torch.int8)


def _scales(gen, n, middle):
    return torch.exp2(torch.rand(n, generator=gen, device="cuda") * 4.0 - 2.0) * middle


def _values(gen, rows, cols, pad, dtype, middle):
    """Activations or gradients: normal, with a few channels many times as large, as trained layers have."""
    v = torch.randn(rows, cols + pad, generator=gen, device="cuda") * middle
    big = torch.rand(cols + pad, generator=gen, device="cuda") < 0.003
    v = v * torch.where(big, 12.0, 1.0)
    return v.to(dtype)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(case)}
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        s["x"] = _values(gen, case["rows"], case["cols"], case["pad"], dtype, 0.5)
        n = case["rows"] if case["transpose"] else case["cols"]
        s["fold"] = _scales(gen, n, 0.01) if case["fold"] else None
        return s
    if op in ("linear", "train", "matmul"):
        m, n, k = case["m"], case["n"], case["k"]
        s["w"], s["sw"] = _levels(gen, n, k), _scales(gen, n, 0.02 / math.sqrt(k))
        s["bias"] = torch.randn(n, generator=gen, device="cuda") * 0.1 if case["bias"] else None
        if op == "matmul":
            s["a"], s["sa"] = _levels(gen, m, k), _scales(gen, m, 0.01)
        else:
            s["x"] = _values(gen, m, k, 0, dtype, 1.0)
        if op == "train":
            s["gy"] = _values(gen, m, n, 0, dtype, 0.01)
        return s
    rows, vocab, k, tau = case["rows"], case["vocab"], min(case["k"], case["vocab"]), case["tau"]
    z = torch.randn(rows, vocab + case["pad"], generator=gen, device="cuda") * 2.5
    z[:, vocab - vocab // 500:] = -math.inf  # the columns that fill a vocabulary up are never predicted
    zt = z[:, :vocab] * 0.8 + torch.randn(rows, vocab, generator=gen, device="cuda") * 1.5
    t, idx = zt.topk(k, dim=1)
    s["teacher_lse"] = torch.logsumexp(zt / tau, dim=1) if case["tail"] else None
    del zt
    cut = torch.rand(rows, generator=gen, device="cuda")
    kept = torch.where(cut < 0.02, 0, torch.where(cut < 0.1, (cut * 10 * k).long(), k))  # positions with fewer entries, or none
    s["idx"] = torch.where(torch.arange(k, device="cuda") < kept[:, None], idx, -1).to(torch.int32)
    s["t"] = t
    s["z"] = z.to(dtype)[:, :vocab]
    weight = (torch.rand(rows, generator=gen, device="cuda") > 0.05).float() / rows  # padding positions weigh nothing
    s["grad_loss"] = weight * 1024.0 if case["dtype"] == "f16" else weight  # gradients in half precision are scaled up
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import quantized_sgd_amd as q
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        levels, scale = q.int8_quantize(s["x"], fold=s["fold"], transpose=case["transpose"])
        return levels * scale[:, None], scale
    if op == "linear":
        return q.int8_linear(s["x"], s["w"], s["sw"], bias=s["bias"])
    if op == "train":
        y, xq, sx = q.int8_linear(s["x"], s["w"], s["sw"], bias=s["bias"], keep=True)
        gx, gw = q.int8_linear_backward(s["gy"], xq, sx, s["w"], s["sw"])
        return y, gx, gw
    if op == "matmul":
        return q.int8_matmul(s["a"], s["sa"], s["w"], s["sw"], bias=s["bias"], dtype=DTYPES[case["dtype"]])
    if op == "distill":
        loss, _ = q.distill_topk(s["z"], s["idx"], s["t"], tau=case["tau"], teacher_lse=s["teacher_lse"])
        return loss
    if op == "distill_pair":
        loss, stats = q.distill_topk(s["z"], s["idx"], s["t"], tau=case["tau"], teacher_lse=s["teacher_lse"])
        dz = q.distill_topk_backward(s["z"], s["idx"], s["t"], stats, s["grad_loss"], tau=case["tau"],
                                     teacher_lse=s["teacher_lse"])
        return loss, dz
    return q.distill_topk_step(s["z"], s["idx"], s["t"], s["grad_loss"], tau=case["tau"], teacher_lse=s["teacher_lse"])


# ---- the plain forms, in 32 bits ----

def _plain_quantize(x, fold, dim):
    """Levels (in 32 bits) and scales of max-norm quantization along `dim`, in x's own layout."""
    y = x.float()
    if fold is not None:
        y = y * (fold[:, None] if dim == 0 else fold)
    amax = y.abs().amax(dim)
    scale = amax / torch.full_like(amax, 127.0)
    by = scale.unsqueeze(dim)
    levels = torch.where((by > 0) & (by < math.inf), (y / by).round().clamp(-127, 127), 0.0)
    return levels, scale


def _plain_product(a, sa, b, sb, bias):
    y = (a @ b.t()) * sa[:, None]
    if sb is not None:
        y = y * sb
    return y if bias is None else y + bias


def _plain_distill(s, gradient):
    case = s["case"]
    tau, idx = case["tau"], s["idx"].long()
    z = s["z"].float() / tau
    t = s["t"].float() / tau
    there = (idx >= 0) & (idx < z.shape[1])
    at = torch.where(there, idx, 0)
    some = there.any(1)
    m = z.amax(1, keepdim=True)
    e = (z - m).exp()
    sum_all = e.sum(1, keepdim=True)
    log_all = sum_all.log()
    log_q = z.gather(1, at) - m - log_all
    if s["teacher_lse"] is None:
        tm = torch.where(there, t, -math.inf).amax(1, keepdim=True)
        tm = torch.where(some[:, None], tm, 0.0)
        pe = torch.where(there, (t - tm).exp(), 0.0)
        norm = torch.where(some[:, None], pe.sum(1, keepdim=True), 1.0)
        p, log_p = pe / norm, t - tm - norm.log()
    else:
        log_p = t - s["teacher_lse"][:, None]
        p = torch.where(there, log_p.exp(), 0.0)
    loss = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1)
    rest = None
    if s["teacher_lse"] is not None:
        top = torch.zeros(z.shape, dtype=torch.int32, device=z.device).scatter_add_(1, at, there.int()) > 0
        zr = torch.where(top, -math.inf, z)
        mr = zr.amax(1, keepdim=True)
        mr = torch.where(mr > -math.inf, mr, 0.0)
        er = (zr - mr).exp()
        sum_rest = er.sum(1, keepdim=True)
        p_rest = (1.0 - p.sum(1, keepdim=True)).clamp_min(0.0)
        p_rest = torch.where(sum_rest > 0, p_rest, 0.0)
        log_rest = mr + sum_rest.log() - m - log_all
        loss = loss + torch.where(p_rest > 0, p_rest * (p_rest.log() - log_rest), 0.0)[:, 0]
        rest = er * torch.where(sum_rest > 0, p_rest / sum_rest, 0.0)
    loss = torch.where(some, loss, 0.0)
    if not gradient:
        return loss
    dz = e / sum_all
    if rest is not None:
        dz = dz - rest
    dz.scatter_add_(1, at, torch.where(there, -p, 0.0))
    dz = dz * (s["grad_loss"] / tau)[:, None]
    dz = torch.where(some[:, None] & (s["grad_loss"] != 0)[:, None], dz, 0.0)
    return loss, dz.to(s["z"].dtype)


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        if case["transpose"]:
            levels, scale = _plain_quantize(s["x"], s["fold"], 0)
            return (levels * scale).t().contiguous(), scale
        levels, scale = _plain_quantize(s["x"], s["fold"], 1)
        return levels * scale[:, None], scale
    if op == "matmul":
        return _plain_product(s["a"].float(), s["sa"], s["w"].float(), s["sw"], s["bias"]).to(dtype)
    if op in ("linear", "train"):
        w = s["w"].float()
        xq, sx = _plain_quantize(s["x"], None, 1)
        y = _plain_product(xq, sx, w, s["sw"], s["bias"]).to(dtype)
        if op == "linear":
            return y
        gq, sg = _plain_quantize(s["gy"], s["sw"], 1)
        gx = ((gq @ w) * sg[:, None]).to(dtype)
        hq, sh = _plain_quantize(s["gy"], sx, 0)
        gw = (hq.t() @ xq) * sh[:, None]
        return y, gx, gw
    return _plain_distill(s, op != "distill")


# ---- the definitions, in 64 bits ----

def _exact_levels(x, fold):
    """Rows of x; a folded value and a scale are held in 32 bits by definition, the quotient is not."""
    y = x.float() if fold is None else x.float() * fold
    scale = (y.abs().max(dim=1).values.double() / 127).float().double()
    ok = (scale > 0) & torch.isfinite(scale)
    r = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    r[ok] = torch.clamp(torch.round(y[ok].double() / scale[ok, None]), -127, 127)
    return r, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].t() if case["transpose"] else s["x"]
        r, scale = _exact_levels(x, s["fold"])
        return r * scale[:, None], scale
    if op in ("linear", "train", "matmul"):
        w, sw = s["w"].double(), s["sw"].double()
        a, sa = (s["a"].double(), s["sa"].double()) if op == "matmul" else _exact_levels(s["x"], None)
        y = torch.matmul(a, w.t().contiguous()) * sa[:, None] * sw[None, :]
        if s["bias"] is not None:
            y += s["bias"].double()[None, :]
        if op != "train":
            return y
        g, sg = _exact_levels(s["gy"], s["sw"])
        h, sh = _exact_levels(s["gy"].t(), sa.float())
        return y, torch.matmul(g, w) * sg[:, None], torch.matmul(h, a) * sh[:, None]
    tau, rows, vocab = case["tau"], case["rows"], case["vocab"]
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    dz = None if op == "distill" else torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for lo in range(0, rows, step):
        at = slice(lo, lo + step)
        z, idx, t = s["z"][at].double() / tau, s["idx"][at].long(), s["t"][at].double() / tau
        n = z.shape[0]
        log_q = torch.log_softmax(z, 1)
        ok = idx >= 0
        some = ok.any(1)
        # the teacher over the whole vocabulary, one column more for the entries that are none
        full = torch.full((n, vocab + 1), -math.inf, dtype=torch.float64, device="cuda")
        full.scatter_(1, torch.where(ok, idx, vocab), t)
        full = full[:, :vocab]
        listed_there = torch.zeros(n, vocab + 1, dtype=torch.bool, device="cuda")
        listed_there.scatter_(1, torch.where(ok, idx, vocab), True)
        listed_there = listed_there[:, :vocab]
        if s["teacher_lse"] is None:
            log_p = torch.log_softmax(torch.where(some[:, None], full, 0.0), 1)
        else:
            log_p = full - s["teacher_lse"][at].double()[:, None]
        p = log_p.exp() * listed_there
        row = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1)
        d = log_q.exp() - p
        if s["teacher_lse"] is not None:
            other = torch.logsumexp(torch.where(listed_there, -math.inf, log_q), 1)
            left = (1 - p.sum(1)).clamp_min(0) * (other > -math.inf)
            row = row + torch.where(left > 0, left * (left.log() - other), 0.0)
            share = torch.where(other[:, None] > -math.inf, (log_q - other[:, None]).exp(), 0.0)
            d = d - torch.where(listed_there, 0.0, share * left[:, None])
        loss[at] = torch.where(some, row, 0.0)
        if dz is not None:
            g = s["grad_loss"][at].double()
            dz[at] = torch.where((some & (g != 0))[:, None], d * (g / tau)[:, None], 0.0)
    return loss if dz is None else (loss, dz)


def work(case):
    """Inputs read once, outputs written once; two operations for each product and sum of a matrix product."""
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        other, n = (r, c) if case["transpose"] else (c, r)
        return {"bytes": r * c * (e + 4) + 4 * n + (4 * other if case["fold"] else 0), "flops": 3 * r * c}
    if op in ("linear", "train", "matmul"):
        m, n, k = case["m"], case["n"], case["k"]
        vectors = 4 * n + (4 * n if case["bias"] else 0)
        if op == "matmul":
            return {"bytes": m * k + n * k + m * n * e + 4 * m + vectors, "flops": 2 * m * n * k}
        b = m * k * e + n * k + m * n * e + vectors
        if op == "linear":
            return {"bytes": b, "flops": 2 * m * n * k}
        return {"bytes": b + m * n * e + m * k * e + 4 * n * k, "flops": 6 * m * n * k}
    rows, vocab, k = case["rows"], case["vocab"], min(case["k"], case["vocab"])
    b = rows * vocab * e + rows * k * 8 + rows * (8 if case["tail"] else 4)
    if op != "distill":
        b += rows * vocab * e + 4 * rows
    return {"bytes": b, "flops": (4 if op == "distill" else 8) * rows * vocab}
