"""The operators of the dense side of a training step, as cases to be measured: layer norm over each table's
columns of the pooled output (forward and backward), AdamW over many tensors with 32-bit or 8-bit states, and
the global norm of many gradients with its clip coefficient.

Each case runs in a plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
calls that a user makes of bwd_tbe_fwd_gb300.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

LN_EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
START_STEP = 10          # updates done before the measured one
MAX_NORM = 1.0
BLOCK = 256              # elements that share a scale of the 8-bit states


# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # The tiny two-table workload's pooled rows (32 bags, D = 64): launch latency.
        ln_case("ln_fwd_tiny", "forward", rows=32, tables=2, widths="64", x="f32", y="f32"),
        # The mixed-width workload's 64 tables (D in {32, 64, 128, 256}, 16384 bags), normalised per table
        # into the type of a 16-bit dense part.
        ln_case("ln_fwd_mixed", "forward", rows=16384, tables=64, widths="32,64,128,256", x="f32", y="bf16"),
        # Dense activations of an odd width, whose rows start at no 4-byte boundary.
        ln_case("ln_fwd_odd", "forward", rows=12345, tables=1, widths="1001", x="f16", y="f16"),
        ln_case("ln_bwd_tiny", "backward", rows=32, tables=2, widths="64", x="f32", y="f32"),
        # The mid-scale workload: 26 tables of D = 128, 8192 bags; dx is the embedding backward's grad_out.
        ln_case("ln_bwd_mid", "backward", rows=8192, tables=26, widths="128", x="f32", y="bf16"),
        # Wide dense activations of a large batch.
        ln_case("ln_bwd_wide", "backward", rows=16384, tables=1, widths="4096", x="bf16", y="bf16"),
        # A small dense network packed tightly into one bucket: launch latency.
        adam_case("adamw_small", width=128, layers=2, param="f32", grad="f32", states="f32", master=False),
        # 16-bit parameters with 32-bit masters and states.
        adam_case("adamw_large", width=1024, layers=24, param="bf16", grad="bf16", states="f32", master=True),
        # 8-bit states of an odd-sized network: every tensor ends inside a block.
        adam_case("adamw_q8_odd", width=257, layers=3, param="f32", grad="f32", states="q8", master=False),
        adam_case("adamw_q8_large", width=1024, layers=12, param="bf16", grad="bf16", states="q8", master=False),
        # The gradients of the two networks above.
        norm_case("grad_norm_small", width=128, layers=2, grad="f32"),
        norm_case("grad_norm_large", width=1024, layers=24, grad="bf16"),
    ]


def ln_case(name, direction, rows, tables, widths, x, y, pad=0):
    """`widths` repeats over the tables; `pad`: columns of the x and y buffers past the normalised ones."""
    return {"name": name, "op": "layer_norm", "direction": direction, "rows": rows, "tables": tables,
            "widths": widths, "x": x, "y": y, "pad": pad}


def adam_case(name, width, layers, param, grad, states, master):
    return {"name": name, "op": "adamw", "width": width, "layers": layers, "param": param, "grad": grad,
            "states": states, "master": master}


def norm_case(name, width, layers, grad):
    return {"name": name, "op": "grad_norm", "width": width, "layers": layers, "grad": grad}


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm", "adamw", "adamw", "grad_norm"])
    if op == "layer_norm":
        direction = rng.choice(["forward", "backward"])
        x, y = rng.choice([("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
        tables = rng.choice([1, 1, rng.randint(2, 64)])
        if tables > 1:
            widths = rng.choice(["32,64,128,256", "128", "64", "4,100,36,260", str(4 * rng.randint(1, 100))])
        else:
            widths = str(_log_uniform(rng, 4, 8192))
            if widths == "3072":
                widths = "3071"
        n = sum(case_widths({"tables": tables, "widths": widths}))
        rows = _log_uniform(rng, 1, min(131072, (1 << 26) // n))
        c = ln_case("", direction, rows, tables, widths, x, y, pad=rng.choice([0, 0, 8, rng.randint(1, 63)]))
    else:
        width, layers = _log_uniform(rng, 16, 1024), rng.randint(1, 12)
        if 4 * width == 3072:
            width += 1
        grad = rng.choice(["f32", "bf16", "f16"])
        if op == "grad_norm":
            c = norm_case("", width, layers, grad)
        else:
            param = rng.choice(["f32", grad])
            c = adam_case("", width, layers, param, grad, rng.choice(["f32", "q8"]),
                          param != "f32" and rng.random() < 0.5)
    del c["name"]
    return c


def case_widths(c):
    w = [int(v) for v in c["widths"].split(",")]
    return [w[t % len(w)] for t in range(c["tables"])]


def case_numels(c):
    """Tensor sizes of a plain network: matrices first (they decay), then biases and norm weights (they do not)."""
    w, matrices, vectors = c["width"], [], []
    for _ in range(c["layers"]):
        matrices += [w * w, 4 * w * w, 4 * w * w]
        vectors += [w, 4 * w, w, w]
    return matrices, vectors


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    return {"layer_norm": _prepare_ln, "adamw": _prepare_adamw, "grad_norm": _prepare_norm}[case["op"]](case, seed)


def _prepare_ln(c, seed):
    g = _generator(seed)
    widths, rows = case_widths(c), c["rows"]
    n = sum(widths)
    ld = n + c["pad"]
    # Pooled rows: sums of about 20 small table rows, some tables' mean off zero, one bag in 20 empty (zeros).
    x = _randn(g, rows, ld).mul_(0.03).add_(_randn(g, ld).mul_(0.02))
    x.mul_(torch.rand(rows, 1, generator=g, device="cuda") >= 0.05)
    x = x.to(DT[c["x"]])[:, :n]
    s = {"case": c, "widths": widths, "x": x,
         "weight": 1 + 0.1 * _randn(g, n), "bias": 0.1 * _randn(g, n)}
    s["segment"] = torch.repeat_interleave(torch.arange(len(widths), device="cuda"),
                                           torch.tensor(widths, device="cuda"))
    if c["direction"] == "backward":
        s["dy"] = _randn(g, rows, ld).to(DT[c["y"]])[:, :n]
        # the forward's statistics are in hand when the backward runs
        mean, var = _segment_moments(x.float(), widths, s["segment"])
        s["mean"], s["rstd"] = mean.contiguous(), (1 / torch.sqrt(var + LN_EPS)).contiguous()
    if own:  # the handle that a user's program makes once
        from bwd_tbe_fwd_gb300 import LayerNorm
        s["norm"] = LayerNorm(widths, x_dtype=DT[c["x"]], y_dtype=DT[c["y"]], weight_dtype=torch.float32, eps=LN_EPS,
                              device="cuda")
    return s


def _prepare_adamw(c, seed):
    g = _generator(seed)
    q8 = c["states"] == "q8"
    matrices, vectors = case_numels(c)
    numels = matrices + vectors
    # 32-bit states: tensors packed tightly, as in a flat bucket.  8-bit states: each tensor starts at a block.
    room = [-(-n // BLOCK) * BLOCK if q8 else n for n in numels]
    starts = np.concatenate([[0], np.cumsum(room)]).tolist()
    total = starts[-1]
    live = torch.ones(total, dtype=torch.bool, device="cuda")
    if q8:
        for n, a, b in zip(numels, starts, starts[1:]):
            live[a + n:b] = False
    s = {"case": c, "numels": numels, "starts": starts, "decayed": starts[len(matrices)], "t": START_STEP}
    master = _randn(g, total).mul_(0.02).mul_(live)
    s["param"] = master.to(DT[c["param"]])
    if c["master"]:
        s["master"] = master
    size = torch.exp(0.5 * _randn(g, total // BLOCK + 1)).mul_(1e-3).repeat_interleave(BLOCK)[:total].mul_(live)
    s["grad"] = _randn(g, total).mul_(size).to(DT[c["grad"]])
    m = _randn(g, total).mul_(size).mul_(0.3)
    v = (0.5 + torch.rand(total, generator=g, device="cuda")).mul_(size).mul_(size).mul_(1 - BETA2 ** START_STEP)
    if q8:
        s["m"], s["m_scale"] = _encode(m, signed=True)
        s["v"], s["v_scale"] = _encode(v, signed=False)
        s["m_values"], s["v_values"] = torch.zeros_like(m), torch.zeros_like(v)
        s["m_levels"], s["v_levels"] = _code_values(True), _code_values(False)
    else:
        s["m"], s["v"] = m, v
    s["step"] = torch.full((1,), START_STEP, dtype=torch.int64, device="cuda")
    s["clip"] = torch.tensor([2.0, 0.5], device="cuda")  # what the gradients' norm left there: {norm, coefficient}
    if own:  # the handle that a user's program makes once
        from bwd_tbe_fwd_gb300 import DenseAdamW

        def parts(flat, unit=1):
            return [flat[a // unit:a // unit + -(-n // unit)] for a, n in zip(starts, numels)]

        state = {"exp_avg": parts(s["m"]), "exp_avg_sq": parts(s["v"]), "step": s["step"]}
        if q8:
            state |= {"exp_avg_scale": parts(s["m_scale"], BLOCK), "exp_avg_sq_scale": parts(s["v_scale"], BLOCK)}
            s["values"] = (parts(s["m_values"]), parts(s["v_values"]))
        s["opt"] = DenseAdamW(parts(s["param"]), parts(s["grad"]), states=c["states"],
                              master=parts(s["master"]) if c["master"] else None, state=state,
                              weight_decay=[DECAY] * len(matrices) + [0.0] * len(vectors),
                              betas=(BETA1, BETA2), eps=ADAM_EPS)
    return s


def _prepare_norm(c, seed):
    g = _generator(seed)
    matrices, vectors = case_numels(c)
    numels = matrices + vectors
    starts = np.concatenate([[0], np.cumsum(numels)]).tolist()
    s = {"case": c, "grad": _randn(g, starts[-1]).mul_(1e-2).to(DT[c["grad"]])}
    if own:  # the handle that a user's program makes once
        from bwd_tbe_fwd_gb300 import GradNorm
        s["norm"] = GradNorm([s["grad"][a:a + n] for a, n in zip(starts, numels)])
    return s


# ------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if c["op"] == "layer_norm":
        if c["direction"] == "forward":
            if own:
                y, mean, rstd = s["norm"].forward(s["x"], s["weight"], s["bias"])
            else:
                y, mean, rstd = _plain_ln_forward(s)
            return {"y": y, "mean": mean, "rstd": rstd}
        if own:
            dx, dw, db = s["norm"].backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        else:
            dx, dw, db = _plain_ln_backward(s)
        return {"dx": dx, "dweight": dw, "dbias": db}
    if c["op"] == "adamw":
        if own:
            s["opt"].step(LR, clip=s["clip"])
            if c["states"] == "q8":
                s["opt"].state_values(*s["values"])
        else:
            _plain_adamw(s)
        out = {"param": s["param"], "step": s["step"]}
        if c["master"]:
            out["master"] = s["master"]
        if c["states"] == "q8":
            return out | {"exp_avg": s["m_values"], "exp_avg_sq": s["v_values"]}
        return out | {"exp_avg": s["m"], "exp_avg_sq": s["v"]}
    if own:
        return s["norm"].compute(MAX_NORM)
    norm = s["grad"].float().square().sum().sqrt()
    return torch.stack([norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)])


def _segment_mean(x, widths, segment):
    """[rows, tables]: the mean of each table's columns."""
    if len(set(widths)) == 1:
        return x.reshape(x.shape[0], len(widths), widths[0]).mean(2)
    w = torch.tensor(widths, dtype=x.dtype, device=x.device)
    member = (segment[:, None] == torch.arange(len(widths), device=x.device)).to(x.dtype)
    return (x @ member) / w


def _spread(v, widths, segment):
    """Each table's value at each of its columns."""
    if len(set(widths)) == 1:
        return v[:, :, None].expand(-1, -1, widths[0]).reshape(v.shape[0], -1)
    return v[:, segment]


def _segment_moments(x, widths, segment):
    mean = _segment_mean(x, widths, segment)
    return mean, _segment_mean((x - _spread(mean, widths, segment)).square(), widths, segment)


def _plain_ln_forward(s):
    x = s["x"].float()
    mean, var = _segment_moments(x, s["widths"], s["segment"])
    rstd = 1 / torch.sqrt(var + LN_EPS)
    xhat = (x - _spread(mean, s["widths"], s["segment"])) * _spread(rstd, s["widths"], s["segment"])
    return (xhat * s["weight"] + s["bias"]).to(DT[s["case"]["y"]]), mean, rstd


def _plain_ln_backward(s):
    widths, seg = s["widths"], s["segment"]
    x, dy = s["x"].float(), s["dy"].float()
    rstd = _spread(s["rstd"], widths, seg)
    xhat = (x - _spread(s["mean"], widths, seg)) * rstd
    h = dy * s["weight"]
    c1, c2 = _segment_mean(h, widths, seg), _segment_mean(h * xhat, widths, seg)
    dx = rstd * (h - _spread(c1, widths, seg) - xhat * _spread(c2, widths, seg))
    return dx.to(DT[s["case"]["x"]]), (dy * xhat).sum(0), dy.sum(0)


# The 8-bit code of x in [0, 1]: the number of leading zeros of the code is a power of 8, the bits below the
# leading one divide that power's interval evenly.  With k the place of the leading one, code c stands for
# (7 c + 7 - 6 * 2^k) * 2^(2 k - 3 bits), so that the largest code is 1 and the values are exact in 32 bits.
def _code_values(signed):
    """What each of the 256 codes stands for, in units of its block's scale."""
    bits = 7 if signed else 8
    c = torch.arange(1 << bits, dtype=torch.float32, device="cuda")
    k = torch.floor(torch.log2(torch.clamp(c, min=1.0) + 0.5))
    values = torch.where(c > 0, (7 * c + 7 - 6 * torch.exp2(k)) * torch.exp2(2 * k - 3 * bits), c)
    return torch.cat([values, -values]) if signed else values


def _encode(x, signed):
    """Codes (uint8; a sign bit and 7 bits of magnitude where `signed`) and the scale of each block of 256."""
    bits = 7 if signed else 8
    blocks = x.reshape(-1, BLOCK)
    a = blocks.abs().amax(1, keepdim=True)
    a = torch.where(a < 2.0 ** -120, torch.zeros_like(a), a)
    r = blocks.abs() * torch.where(a > 0, 1 / a, a)
    e = torch.where(r > 0, torch.frexp(r).exponent - 1, -126)
    z = torch.clamp((-1 - e) // 3, 0, bits - 1)           # leading zeros of the code
    low = torch.exp2((bits - 1 - z).float())              # its leading one
    # the interval's straight line, c = ((8^(z+1) r - 1) / 7) low + low - 1, with its slope and offset in 32 bits
    slope = torch.exp2((bits + 2 + 2 * z).float()) * np.float32(1 / 7).item()
    c = torch.round(r * slope + (low * np.float32(6 / 7).item() - 1))
    if signed:
        c = c + 128 * (blocks < 0)
    else:  # a positive second moment never becomes zero
        c = torch.where(r > 0, torch.clamp(c, min=1.0), c)
    return c.to(torch.uint8).reshape(-1), a.reshape(-1)


def _decode(codes, scale, levels):
    return (levels[codes.long()].reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _plain_adamw(s):
    c, n = s["case"], s["decayed"]
    q8 = c["states"] == "q8"
    s["t"] += 1
    s["step"] += 1
    g = s["grad"].float() * s["clip"][1]
    m, v = s["m"], s["v"]
    if q8:
        m, v = _decode(m, s["m_scale"], s["m_levels"]), _decode(v, s["v_scale"], s["v_levels"])
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    update = (m / (1 - BETA1 ** s["t"])) / (torch.sqrt(v / (1 - BETA2 ** s["t"])) + ADAM_EPS)
    p = s["master"] if c["master"] else s["param"].float()
    p = torch.cat([p[:n] * (1 - LR * DECAY), p[n:]]) - LR * update
    if c["master"]:
        s["master"].copy_(p)
    s["param"].copy_(p)
    if q8:
        codes, scale = _encode(m, True)
        s["m"].copy_(codes), s["m_scale"].copy_(scale)
        s["m_values"].copy_(_decode(codes, scale, s["m_levels"]))
        codes, scale = _encode(v, False)
        s["v"].copy_(codes), s["v_scale"].copy_(scale)
        s["v_values"].copy_(_decode(codes, scale, s["v_levels"]))
    else:
        s["m"].copy_(m), s["v"].copy_(v)


# ------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(c):
    if c["op"] == "layer_norm":
        rows, n = c["rows"], sum(case_widths(c))
        stats = 8 * rows * c["tables"]
        if c["direction"] == "forward":
            return {"bytes": rows * n * (SIZE[c["x"]] + SIZE[c["y"]]) + stats + 8 * n, "flops": 8 * rows * n}
        return {"bytes": rows * n * (2 * SIZE[c["x"]] + SIZE[c["y"]]) + stats + 12 * n, "flops": 14 * rows * n}
    matrices, vectors = case_numels(c)
    total = sum(matrices) + sum(vectors)
    if c["op"] == "grad_norm":
        return {"bytes": total * SIZE[c["grad"]], "flops": 2 * total}
    per = SIZE[c["grad"]] + SIZE[c["param"]] + (8 if c["master"] else SIZE[c["param"]])
    # 32-bit states are read and written; 8-bit ones too, with a scale per block, and the values they stand for are written
    per += 16 if c["states"] == "f32" else 4 + 16 / BLOCK + 8
    return {"bytes": total * per, "flops": 15 * total}


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"layer_norm": _exact_ln, "adamw": _exact_adamw, "grad_norm": _exact_norm}[case["op"]](s)


def _exact_ln(s):
    forward = s["case"]["direction"] == "forward"
    x = s["x"].double()
    outs, at = [], 0
    for t, width in enumerate(s["widths"]):
        cols = slice(at, at + width)
        at += width
        w, b = s["weight"][cols].double(), s["bias"][cols].double()
        xt = x[:, cols]
        if forward:
            mu = xt.sum(1) / width
            d = xt - mu[:, None]
            r = (d.pow(2).sum(1) / width + LN_EPS).rsqrt()
            outs.append((d * r[:, None] * w + b, mu[:, None], r[:, None]))
        else:
            dy, r = s["dy"][:, cols].double(), s["rstd"][:, t, None].double()
            hat = (xt - s["mean"][:, t, None].double()) * r
            h = dy * w
            dx = (h - h.sum(1, keepdim=True) / width - hat * (h * hat).sum(1, keepdim=True) / width) * r
            outs.append((dx, (dy * hat).sum(0), dy.sum(0)))
    if forward:
        return dict(zip(("y", "mean", "rstd"), (torch.cat(v, 1) for v in zip(*outs))))
    dx, dw, db = zip(*outs)
    return {"dx": torch.cat(dx, 1), "dweight": torch.cat(dw), "dbias": torch.cat(db)}


def _exact_levels(bits):
    levels = [0.0]
    for c in range(1, 1 << bits):
        k = c.bit_length() - 1
        levels.append(8.0 ** (k - bits) * (1 + 7 * (c - 2 ** k + 1) / 2 ** k))
    return torch.tensor(levels, dtype=torch.float64, device="cuda")


def _exact_decode(codes, scale, signed):
    c = codes.long()
    size = _exact_levels(7 if signed else 8)[c % 128 if signed else c]
    size = torch.where(c >= 128, -size, size) if signed else size
    return (size.view(-1, BLOCK) * scale.double()[:, None]).view(-1)


def _exact_requantize(x, signed):
    """The nearest code's value in the block's scale: each interval between two codes is split at its middle, but the one
    above zero, whose linear piece runs from 8^-bits."""
    levels = _exact_levels(7 if signed else 8)
    bits = 7 if signed else 8
    split = (levels[1:] + levels[:-1]) / 2
    split[0] = (levels[1] + 8.0 ** -bits) / 2 if signed else 0.0
    blocks = x.view(-1, BLOCK)
    a = blocks.abs().amax(1, keepdim=True)
    r = blocks.abs() / torch.where(a > 0, a, torch.ones_like(a))
    value = levels[torch.bucketize(r, split)] * a
    return torch.where(blocks < 0, -value, value).view(-1)


def _exact_adamw(s):
    c, t = s["case"], s["t"] + 1
    q8 = c["states"] == "q8"
    g = s["grad"].double() * 0.5
    m = _exact_decode(s["m"], s["m_scale"], True) if q8 else s["m"].double()
    v = _exact_decode(s["v"], s["v_scale"], False) if q8 else s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g.pow(2)
    p = (s["master"] if c["master"] else s["param"]).double().clone()
    p[:s["decayed"]] *= 1 - LR * DECAY
    p -= LR / (1 - BETA1 ** t) * m / (v.div(1 - BETA2 ** t).sqrt() + ADAM_EPS)
    out = {"param": p, "step": None}
    if c["master"]:
        out["master"] = p
    out["exp_avg"] = _exact_requantize(m, True) if q8 else m
    out["exp_avg_sq"] = _exact_requantize(v, False) if q8 else v
    return out


def _exact_norm(s):
    norm = torch.linalg.vector_norm(s["grad"].double())
    return torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)])
