"""The two ends of a model over tokens or items, as cases to be measured: the lookup of one table's rows with
scaling and its gradient by sorted tokens (TokenEmbedding), and the softmax cross entropy over a table's rows
without keeping the logits, with its gradient (SoftmaxLoss).

Each case runs in a plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
calls that a user makes of bwd_tbe_fwd_gb300.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IT = {"i32": torch.int32, "i64": torch.int64}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i32": 4, "i64": 8}


# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # The tiny workload's table (1000 rows, D = 64) and its 32 bags' worth of ids: launch latency.
        lookup_case("lookup_fwd_tiny", "forward", tokens=32, rows=1000, dim=64, table="f32", out="f32"),
        # A batch of the stress workload's size (131072 ids) over one of its tables (4M fp16 rows, D = 128).
        lookup_case("lookup_fwd_large", "forward", tokens=131072, rows=4_000_000, dim=128, table="f16", out="f32"),
        lookup_case("lookup_bwd_tiny", "backward", tokens=32, rows=1000, dim=64, table="f32", out="f32"),
        # Items of an odd width, whose rows start at no 4-byte boundary, with padded sequences.
        lookup_case("lookup_bwd_odd", "backward", tokens=12345, rows=50_021, dim=301, table="f16", out="f16",
                    outside=0.2, itype="i32"),
        # A training batch over a large vocabulary.
        lookup_case("lookup_bwd_large", "backward", tokens=65536, rows=131072, dim=1024, table="bf16", out="bf16"),
        # The same with the table tied to the loss, whose gradient is there already.
        lookup_case("lookup_bwd_tied", "backward", tokens=16384, rows=131072, dim=1024, table="bf16", out="bf16",
                    accumulate=True),
        # A small item table in a small batch: launch latency.
        loss_case("loss_fwd_tiny", "forward", tokens=32, rows=1000, dim=64, dtype="bf16"),
        # Scoring a few continuations: bound by the table's one pass through memory.
        loss_case("loss_fwd_few", "forward", tokens=16, rows=131072, dim=2048, dtype="bf16"),
        # A training batch over a large vocabulary, forward and backward.
        loss_case("loss_fwd_large", "forward", tokens=8192, rows=131072, dim=1024, dtype="bf16"),
        loss_case("loss_bwd_tiny", "backward", tokens=32, rows=1000, dim=64, dtype="bf16"),
        # Retrieval: normalised items of an odd width with a temperature; a third of the targets is padding.
        loss_case("loss_bwd_odd", "backward", tokens=1777, rows=50_021, dim=301, dtype="f16", scale=20.0, outside=0.33,
                  upstream="tokens"),
        loss_case("loss_bwd_large", "backward", tokens=8192, rows=131072, dim=1024, dtype="bf16"),
    ]


def lookup_case(name, direction, tokens, rows, dim, table, out, outside=0.02, scale=None, itype="i64", accumulate=False,
                pad=0):
    """`outside`: the share of ids that are padding (-1); `pad`: columns of the buffers past a row's; the scale is
    sqrt(dim) where none is given."""
    return {"name": name, "op": "lookup", "direction": direction, "tokens": tokens, "rows": rows, "dim": dim,
            "table": table, "out": out, "outside": outside, "scale": math.sqrt(dim) if scale is None else scale,
            "itype": itype, "accumulate": accumulate, "pad": pad}


def loss_case(name, direction, tokens, rows, dim, dtype, scale=1.0, outside=0.02, itype="i64", upstream="mean", pad=0):
    """`upstream`: the gradient of the mean over the tokens, or one value for each token."""
    return {"name": name, "op": "loss", "direction": direction, "tokens": tokens, "rows": rows, "dim": dim,
            "dtype": dtype, "scale": scale, "outside": outside, "itype": itype, "upstream": upstream, "pad": pad}


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    direction = rng.choice(["forward", "backward"])
    itype = rng.choice(["i32", "i64"])
    outside = rng.choice([0.0, 0.02, 0.33])
    pad = rng.choice([0, 0, 8, rng.randint(1, 15)])
    if rng.random() < 0.45:
        table, out = rng.choice([("f32", "f32"), ("f32", "bf16"), ("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                 ("bf16", "f32")])
        dim = rng.choice([_log_uniform(rng, 4, 2048), 8 * _log_uniform(rng, 1, 256)])
        rows = _log_uniform(rng, 2, min(4_000_000, (1 << 27) // dim))
        tokens = _log_uniform(rng, 1, min(131072, (1 << 26) // dim))
        c = lookup_case("", direction, tokens, rows, dim, table, out, outside, rng.choice([1.0, 0.5, None]), itype,
                        direction == "backward" and rng.random() < 0.3, pad)
    else:
        dim = rng.choice([_log_uniform(rng, 8, 2048), 8 * _log_uniform(rng, 1, 256)])
        rows = _log_uniform(rng, 16, 131072)
        tokens = _log_uniform(rng, 1, min(16384, (1 << 30) // rows, (1 << 40) // (rows * dim)))
        dtype = rng.choice(["bf16", "f16"])
        c = loss_case("", direction, tokens, rows, dim, dtype, rng.choice([1.0, 0.125, 20.0]), outside, itype,
                      rng.choice(["mean", "tokens"]) if dtype == "bf16" else "tokens", pad)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ids(g, tokens, rows, outside, dtype):
    """Ids whose frequency falls with the inverse of their rank, scattered over the table; padding is -1."""
    rank = torch.exp(torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64) * math.log(rows + 1)).long() - 1
    step = next(k for k in range(int(rows * 0.618) + 1, 2 * rows + 2) if math.gcd(k, rows) == 1)
    ids = (rank.clamp(0, rows - 1) * step + rows // 3) % rows
    drop = torch.rand(tokens, generator=g, device="cuda") < outside
    return torch.where(drop, torch.full_like(ids, -1), ids).to(IT[dtype])


def prepare(case, seed):
    return {"lookup": _prepare_lookup, "loss": _prepare_loss}[case["op"]](case, seed)


def _prepare_lookup(c, seed):
    g = _generator(seed)
    rows, dim, tokens = c["rows"], c["dim"], c["tokens"]
    s = {"case": c, "ids": _ids(g, tokens, rows, c["outside"], c["itype"])}
    if c["direction"] == "forward":
        s["table"] = _randn(g, rows, dim).mul_(dim ** -0.5).to(DT[c["table"]])
    else:
        s["dout"] = _randn(g, tokens, dim + c["pad"]).mul_(1e-3).to(DT[c["out"]])[:, :dim]
        grad = torch.zeros(rows, dim, device="cuda")
        if c["accumulate"]:
            grad = _randn(g, rows, dim).mul_(1e-3)
        s["grad"] = grad.to(DT[c["table"]])
    if own:  # the handle that a user's program makes once
        from bwd_tbe_fwd_gb300 import TokenEmbedding
        s["embedding"] = TokenEmbedding(rows, dim, tokens, table_dtype=DT[c["table"]], out_dtype=DT[c["out"]],
                                        index_dtype=IT[c["itype"]], scale=c["scale"], device="cuda")
    return s


def _prepare_loss(c, seed):
    g = _generator(seed)
    rows, dim, tokens = c["rows"], c["dim"], c["tokens"]
    # logits of a spread of about 2, the target's somewhat above the others'
    weight = _randn(g, rows, dim).mul_(2 / (c["scale"] * math.sqrt(dim))).to(DT[c["dtype"]])
    targets = _ids(g, tokens, rows, c["outside"], c["itype"])
    hidden = _randn(g, tokens, dim + c["pad"])
    hidden[:, :dim] += 0.5 * c["scale"] * weight[targets.long().clamp(min=0)].float()
    s = {"case": c, "weight": weight, "targets": targets, "hidden": hidden.to(DT[c["dtype"]])[:, :dim]}
    if c["direction"] == "backward":
        # the forward's results are in hand when the backward runs
        lse = torch.empty(tokens, device="cuda")
        for a in range(0, tokens, 1024):
            lse[a:a + 1024] = _logsumexp(c["scale"] * (s["hidden"][a:a + 1024].float() @ weight.float().T))
        counts = targets >= 0
        s["lse"] = torch.where(counts, lse, torch.zeros_like(lse))
        count = counts.sum().float()
        s["mean"] = torch.stack([torch.zeros_like(count), torch.where(count > 0, 1 / count, count)])
        if c["upstream"] == "tokens":
            s["dloss"] = torch.rand(tokens, generator=g, device="cuda") / tokens
            if c["dtype"] == "f16":  # fp16 gradients come with a loss scale
                s["dloss"] *= 8192 / max(1.0, c["scale"])
    if own:  # the handle that a user's program makes once
        from bwd_tbe_fwd_gb300 import SoftmaxLoss
        s["loss"] = SoftmaxLoss(rows, dim, tokens, dtype=DT[c["dtype"]], index_dtype=IT[c["itype"]], scale=c["scale"],
                                device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if c["op"] == "lookup":
        if c["direction"] == "forward":
            return s["embedding"].forward(s["table"], s["ids"]) if own else _plain_lookup(s)
        if own:
            return s["embedding"].backward(s["dout"], s["ids"], grad=s["grad"], accumulate=c["accumulate"])
        return _plain_lookup_gradient(s)
    if c["direction"] == "forward":
        if own:
            loss, lse, mean = s["loss"].forward(s["hidden"], s["weight"], s["targets"])
        else:
            loss, lse, mean = _plain_loss(s)
        return {"loss": loss, "lse": lse, "mean": mean}
    if own:
        one = c["upstream"] == "tokens"
        dhidden, dweight = s["loss"].backward(s["hidden"], s["weight"], s["targets"], s["lse"],
                                              dloss=s["dloss"] if one else None, mean=None if one else s["mean"])
    else:
        dhidden, dweight = _plain_loss_gradient(s)
    return {"dhidden": dhidden, "dweight": dweight}


def _plain_lookup(s):
    c, ids = s["case"], s["ids"].long()
    rows = s["table"][ids.clamp(min=0)].float() * c["scale"]
    return torch.where((ids >= 0)[:, None], rows, torch.zeros_like(rows)).to(DT[c["out"]])


def _plain_lookup_gradient(s):
    c, ids = s["case"], s["ids"].long()
    dout = s["dout"].float() * c["scale"]
    dout = torch.where((ids >= 0)[:, None], dout, torch.zeros_like(dout))
    base = s["grad"].float() if c["accumulate"] else torch.zeros(c["rows"], c["dim"], device="cuda")
    s["grad"].copy_(base.index_add(0, ids.clamp(min=0), dout))
    return s["grad"]


def _logsumexp(z):
    top = z.amax(1, keepdim=True)
    return (torch.log(torch.exp(z - top).sum(1, keepdim=True)) + top)[:, 0]


def _plain_loss(s):
    targets = s["targets"].long()
    z = (s["hidden"].float() @ s["weight"].float().T) * s["case"]["scale"]
    counts = targets >= 0
    lse = _logsumexp(z)
    loss = lse - z.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    loss, lse = torch.where(counts, loss, zero), torch.where(counts, lse, zero)
    n = counts.sum().float()
    inverse = torch.where(n > 0, 1 / n, n)
    return loss, lse, torch.stack([loss.sum() * inverse, inverse])


def _plain_loss_gradient(s):
    c, targets = s["case"], s["targets"].long()
    h, w = s["hidden"].float(), s["weight"].float()
    counts = targets >= 0
    g = s["dloss"] if c["upstream"] == "tokens" else s["mean"][1].expand(c["tokens"])
    g = torch.where(counts, g, torch.zeros_like(g)) * c["scale"]
    dz = torch.exp((h @ w.T) * c["scale"] - s["lse"][:, None])
    at = targets.clamp(min=0)[:, None]
    dz.scatter_(1, at, dz.gather(1, at) - 1)
    dz = torch.where(counts[:, None], dz * g[:, None], torch.zeros_like(dz))
    return (dz @ w).to(DT[c["dtype"]]), (dz.T @ h).to(DT[c["dtype"]])


# ------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------
def _distinct(c):
    """Expected number of distinct rows among the ids."""
    edge = np.log(np.arange(1, c["rows"] + 2, dtype=np.float64)) / math.log(c["rows"] + 1)
    return int(round(float(-np.expm1(c["tokens"] * (1 - c["outside"]) * np.log1p(-np.diff(edge).clip(0, 1 - 1e-12))).sum())))


def work(c):
    tokens, rows, dim = c["tokens"], c["rows"], c["dim"]
    live = tokens * (1 - c["outside"])
    if c["op"] == "lookup":
        distinct, ids = _distinct(c), tokens * SIZE[c["itype"]]
        if c["direction"] == "forward":
            return {"bytes": ids + distinct * dim * SIZE[c["table"]] + tokens * dim * SIZE[c["out"]], "flops": live * dim}
        touched = 2 * distinct if c["accumulate"] else rows
        return {"bytes": ids + live * dim * SIZE[c["out"]] + touched * dim * SIZE[c["table"]], "flops": live * dim}
    size = SIZE[c["dtype"]]
    read = (live + rows) * dim * size + tokens * SIZE[c["itype"]]
    if c["direction"] == "forward":
        return {"bytes": read + 8 * tokens, "flops": 2 * live * rows * dim}
    # the logits are not kept: their product again, then one for each gradient; tokens whose target is padding need none
    return {"bytes": read + 4 * tokens + (tokens + rows) * dim * size, "flops": 6 * live * rows * dim}


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"lookup": _exact_lookup, "loss": _exact_loss}[case["op"]](s)


def _exact_lookup(s):
    c, ids = s["case"], s["ids"].long()
    live = torch.nonzero(ids >= 0)[:, 0]
    if c["direction"] == "forward":
        out = torch.zeros(c["tokens"], c["dim"], dtype=torch.float64, device="cuda")
        out[live] = s["table"][ids[live]].double() * float(np.float32(c["scale"]))
        return out
    grad = s["grad"].double() if c["accumulate"] else torch.zeros(c["rows"], c["dim"], dtype=torch.float64, device="cuda")
    return grad.index_put((ids[live],), s["dout"][live].double() * float(np.float32(c["scale"])), accumulate=True)


def _exact_loss(s):
    """In pieces of the vocabulary, the tokens with a target alone."""
    c = s["case"]
    scale, rows, piece = float(np.float32(c["scale"])), c["rows"], 8192
    live = torch.nonzero(s["targets"] >= 0)[:, 0]
    h, t = s["hidden"][live].double(), s["targets"][live].long()
    everyone = lambda v, *shape: torch.zeros(c["tokens"], *shape, dtype=torch.float64, device="cuda").index_put((live,), v)  # noqa: E731
    if c["direction"] == "forward":
        at = torch.einsum("nd,nd->n", h, s["weight"][t].double()) * scale
        parts = [torch.logsumexp(h @ s["weight"][a:a + piece].double().T * scale, 1) for a in range(0, rows, piece)]
        lse = torch.logsumexp(torch.stack(parts), 0)
        inverse = 1.0 / len(live) if len(live) else 0.0
        mean = torch.tensor([float((lse - at).sum()) * inverse, inverse], dtype=torch.float64, device="cuda")
        return {"loss": everyone(lse - at), "lse": everyone(lse), "mean": mean}
    g = s["dloss"][live].double() if c["upstream"] == "tokens" else s["mean"][1].double().expand(len(live))
    lse = s["lse"][live].double()
    dh, dw = torch.zeros_like(h), torch.zeros(rows, c["dim"], dtype=torch.float64, device="cuda")
    for a in range(0, rows, piece):
        w = s["weight"][a:a + piece].double()
        dz = (h @ w.T * scale - lse[:, None]).exp()
        own_rows = torch.nonzero((t >= a) & (t < a + len(w)))[:, 0]
        dz[own_rows, t[own_rows] - a] -= 1
        dz *= (g * scale)[:, None]
        dh += dz @ w
        dw[a:a + len(w)] = dz.T @ h
    return {"dhidden": everyone(dh, c["dim"]), "dweight": dw}
