"""The operators of include/tbe_tokens.h in 64 bits (numpy), written from their formulas, with bounds on what evaluation with
fp32 sums may be off by.  Nothing here uses the library.

u = 2^-24 is fp32's unit roundoff.  A sum of n terms whose every addition may lose a whole last place (tensor cores need not
round to nearest) is within 2 n u sum|terms| of the exact one."""
import numpy as np

U = 2.0 ** -24
STORE = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # relative rounding of a store to the type
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # and its least absolute one


def rounded(v, store):
    return STORE[store] * np.abs(v) * 1.01 + TINY[store]


# ------------------------------------------------------------------------------------------
# Lookup
# ------------------------------------------------------------------------------------------
def lookup(table, ids, scale, store):
    """out [N, D] and the bound of its error."""
    table, scale = table.astype(np.float64), float(np.float32(scale))
    live = (ids >= 0) & (ids < len(table))
    out = np.where(live[:, None], scale * table[np.where(live, ids, 0)], 0.0)
    return out, U * np.abs(out) + np.where(out != 0, rounded(out, store), 0.0)


def lookup_gradient(dout, ids, rows, scale, store, old=None):
    """grad [rows, D] (added to `old`) and the bound of its error: zero where there is nothing to add."""
    dout, scale = dout.astype(np.float64), float(np.float32(scale))
    live = (ids >= 0) & (ids < rows)
    grad, size = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1]))
    np.add.at(grad, ids[live], dout[live])
    np.add.at(size, ids[live], np.abs(dout[live]))
    n = np.bincount(ids[live], minlength=rows)[:, None]
    bound = (n + 2) * U * size * abs(scale) * 1.01
    grad = grad * scale
    if old is not None:
        grad = grad + old
        bound = bound + 2 * U * (np.abs(grad) + np.abs(old))
    return grad, np.where(n > 0, bound + rounded(grad, store), 0.0)


# ------------------------------------------------------------------------------------------
# Softmax cross entropy
# ------------------------------------------------------------------------------------------
def logits(hidden, weight, scale):
    """z and the bound of its error: products of 16-bit values are exact in fp32, their sum has D terms."""
    scale = float(np.float32(scale))
    z = scale * (hidden @ weight.T)
    e = scale * (2 * hidden.shape[1] + 4) * U * (np.abs(hidden) @ np.abs(weight).T)
    return z, e


def masked(hidden, targets, rows):
    """The tokens that count, and hidden with nothing in the others' rows."""
    live = (targets >= 0) & (targets < rows)
    return live, np.where(live[:, None], hidden.astype(np.float64), 0.0)


def exponent_error(z, lse, ez):
    """Relative error of exp(z - lse) as 2^(z c - lse c): the product's and the constant's rounding act on the exponents'
    sizes, 2^x itself is good to 2 ulp."""
    return ez + 4 * U * (np.abs(z) + np.abs(lse)) + 6 * U


def loss(hidden, weight, targets, scale):
    """(loss, lse, mean) and their bounds."""
    weight = weight.astype(np.float64)
    live, hidden = masked(hidden, targets, len(weight))
    z, ez = logits(hidden, weight, scale)
    top = z.max(1)
    lse = np.log(np.exp(z - top[:, None]).sum(1)) + top
    # of the sum of exponentials, relative: its terms', and a chain of additions (32 columns and 4 blocks in a thread,
    # then the parts: 2 for 256 rows of the table, dealt out to 32 warps, each joined with two factors)
    chain = 48 + len(weight) // 2048 * 3 + 64
    p = np.exp(z - lse[:, None])
    rel = (p * exponent_error(z, top[:, None], ez)).sum(1) + chain * U
    e = np.where(live, rel + 4 * U * (np.abs(lse) + np.abs(top)) + 4 * U, 0.0)
    at = np.where(live, targets, 0)
    i = np.arange(len(at))
    zt, et = z[i, at], ez[i, at]
    out = np.where(live, lse - zt, 0.0)
    lse = np.where(live, lse, 0.0)
    eo = np.where(live, e + et + 2 * U * (np.abs(zt) + np.abs(out)), 0.0)
    n = live.sum()
    mean = np.array([out.sum() / n, 1 / n]) if n else np.zeros(2)
    em = np.array([eo.sum() / n + 2 * U * abs(mean[0]), U / n * 2]) if n else np.zeros(2)
    return (out, lse, mean), (eo, e, em)


def loss_gradients(hidden, weight, targets, lse, coef, scale, store):
    """dhidden, dweight with lse as given, and their bounds.  dz is held in 16 bits, scaled so that the largest coefficient
    is 2^13 or more: it is off by half a step of the type, or by that of the type's least values."""
    weight = weight.astype(np.float64)
    live, hidden = masked(hidden, targets, len(weight))
    lse = np.where(live, lse.astype(np.float64), 0.0)
    coef = np.where(live, coef.astype(np.float64), 0.0)
    z, ez = logits(hidden, weight, scale)
    with np.errstate(over="ignore"):
        p = np.exp(z - lse[:, None])
    dp = p * (exponent_error(z, lse[:, None], ez) * 1.01)
    i = np.nonzero(live)[0]
    dz = p.copy()
    dz[i, targets[i]] -= 1
    dz *= coef[:, None]
    top = np.abs(coef).max() if len(coef) else 0.0
    edz = np.abs(coef)[:, None] * (dp + 4 * U * p) + np.abs(dz) * (STORE[store] * 1.01 + 4 * U) + top * 2.0 ** -13 * TINY[store] * 2
    edz = np.where(live[:, None], edz, 0.0)
    s = float(np.float32(scale))
    N, V = z.shape
    out = []
    for a, ea, b in ((dz, edz, weight), (dz.T, edz.T, hidden)):
        got = s * (a @ b)
        e = s * (ea @ np.abs(b) * 1.01 + (2 * a.shape[1] + 64) * U * (np.abs(a) @ np.abs(b))) + 4 * U * np.abs(got)
        out.append((got, e + rounded(got, store)))
    (dh, eh), (dw, ew) = out
    return (dh, dw), (np.where(live[:, None], eh, 0.0), ew)
