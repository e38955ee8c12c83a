"""The operators of include/tbe_dense.h in 64 bits (numpy), written from their formulas, with bounds on what fp32
evaluation may be off by.  Nothing here uses the library.

u = 2^-24 is fp32's unit roundoff.  A sum of n terms in which each term passes through at most k additions is within
k u sum|terms| of the exact one (first order; the factors below leave room for the second)."""
import numpy as np

U = 2.0 ** -24
STORE = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # relative rounding of a store to the type
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}         # and its least absolute one (fp16 subnormals)


def chain(n):
    """Additions that a term of a row's sum of n passes through at most: 32 in a thread (more in the rows that
    1024 threads walk through), 5 across a warp, 5 across the warps."""
    return 42 + n // 1024


def segments(widths):
    at = np.concatenate([[0], np.cumsum(widths)])
    return [slice(a, b) for a, b in zip(at[:-1], at[1:])]


def layer_norm(x, widths, weight, bias, eps, store="f32"):
    """x [R, N] -> y, mean, rstd and the bounds of their errors."""
    x = x.astype(np.float64)
    N = x.shape[1]
    w = np.ones(N) if weight is None else weight.astype(np.float64)
    b = np.zeros(N) if bias is None else bias.astype(np.float64)
    y, ey = np.empty_like(x), np.empty_like(x)
    mean, rstd, em, er = ([], [], [], [])
    for c in segments(widths):
        xs, n = x[:, c], c.stop - c.start
        k = chain(n)
        mu = xs.mean(1, keepdims=True)
        d = xs - mu
        var = (d * d).mean(1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            rs = 1 / np.sqrt(var + eps)
            big = np.abs(xs).max(1, keepdims=True)
            d_mu = (k + 2) * U * np.abs(xs).mean(1, keepdims=True)  # of the mean
            d_d = d_mu + 2 * U * big                                # of x - mean
            # of rstd, relative: half that of var + eps, whose part from d is at most 2 sigma d_d + d_d^2 (Cauchy)
            sig = np.sqrt(var)
            rel = 0.5 * ((k + 6) * U + (2 * sig * d_d + d_d * d_d) / (var + eps)) + 4 * U
            y[:, c] = d * rs * w[c] + b[c]
            ey[:, c] = np.abs(w[c]) * (rs * d_d + np.abs(d * rs) * (rel + 4 * U)) * (1 + rel) + 4 * U * np.abs(b[c])
        ey[:, c] += STORE[store] * np.abs(y[:, c]) * 1.01 + TINY[store]
        mean.append(mu), rstd.append(rs), em.append(d_mu + U * np.abs(mu)), er.append(rel * rs)
    cat = lambda v: np.concatenate(v, 1)  # noqa: E731
    return (y, cat(mean), cat(rstd)), (ey, cat(em), cat(er))


def layer_norm_gradients(dy, x, mean, rstd, widths, weight, store_x="f32", store_w="f32"):
    """dx, dweight, dbias with mean and rstd as given, and the bounds of their errors."""
    dy, x, mean, rstd = (v.astype(np.float64) for v in (dy, x, mean, rstd))
    R, N = x.shape
    w = np.ones(N) if weight is None else weight.astype(np.float64)
    dx, ex = np.empty_like(x), np.empty_like(x)
    hat = np.empty_like(x)
    for s, c in enumerate(segments(widths)):
        n, k = c.stop - c.start, chain(c.stop - c.start)
        rs = rstd[:, s, None]
        hat[:, c] = xh = (x[:, c] - mean[:, s, None]) * rs
        h = dy[:, c] * w[c]
        c1, c2 = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
        dx[:, c] = rs * (h - c1 - xh * c2)
        e1 = (k + 4) * U * np.abs(h).mean(1, keepdims=True)
        e2 = (k + 8) * U * np.abs(h * xh).mean(1, keepdims=True)
        ex[:, c] = rs * (e1 + np.abs(xh) * e2 + 8 * U * (np.abs(h) + np.abs(c1) + np.abs(xh * c2)))
    ex += STORE[store_x] * np.abs(dx) * 1.01 + TINY[store_x]
    dw, db = (dy * hat).sum(0), dy.sum(0)
    ew = (R + 16) * U * np.abs(dy * hat).sum(0) + STORE[store_w] * np.abs(dw) * 1.01 + TINY[store_w]
    eb = (R + 16) * U * np.abs(dy).sum(0) + STORE[store_w] * np.abs(db) * 1.01 + TINY[store_w]
    return (dx, dw, db), (ex, ew, eb)


# ------------------------------------------------------------------------------------------
# AdamW
# ------------------------------------------------------------------------------------------
def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay, coef=1.0, store="f32"):
    """One step in 64 bits: p, m, v and the bounds of their errors (m, v: fp32 as given; p: `store` rounds it)."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    b1, b2 = float(np.float32(beta1)), float(np.float32(beta2))
    o1, o2 = float(np.float32(1 - beta1)), float(np.float32(1 - beta2))
    g = g * coef
    m2, v2 = b1 * m + o1 * g, b2 * v + o2 * g * g
    em = 4 * U * (np.abs(b1 * m) + np.abs(o1 * g))
    ev = 6 * U * (b2 * v + o2 * g * g)
    with np.errstate(divide="ignore", invalid="ignore"):
        mh = m2 / (1 - beta1 ** t)
        update = lr * mh / (np.sqrt(v2 / (1 - beta2 ** t)) + eps)
        # of m2 relative to the denominator; then 2^-19 for the root, the quotient (2 ulp each) and the corrections' logarithms
        e_upd = lr * em / (1 - beta1 ** t) / (np.sqrt(v2 / (1 - beta2 ** t)) + eps) + 2.0 ** -19 * np.abs(update)
    p2 = p * (1 - lr * decay) - update
    ep = e_upd + 4 * U * (np.abs(p) + np.abs(update)) + STORE[store] * np.abs(p2) * 1.01 + TINY[store]
    return (p2, m2, v2), (ep, em, ev)


def q8_levels(bits):
    """What each code of `bits` bits of magnitude stands for: its leading zeros count powers of 8, the bits below the leading
    one divide the power's interval evenly, its upper end included."""
    out = [0.0]
    for c in range(1, 1 << bits):
        k = c.bit_length() - 1
        out.append(8.0 ** (k - bits) + (8.0 ** (k + 1 - bits) - 8.0 ** (k - bits)) * (c - (1 << k) + 1) / (1 << k))
    return np.array(out)


def q8_decode(codes, scale, signed, block=256):
    codes = np.asarray(codes, np.int64)
    mag = q8_levels(7)[codes & 127] if signed else q8_levels(8)[codes]
    out = mag * np.repeat(np.asarray(scale, np.float64), block)[:codes.size]
    return np.where(codes >= 128, -out, out) if signed else out


def q8_encode(x, signed, block=256):
    """Nearest codes and scales of fp32 values, by search over the levels."""
    x = np.asarray(x, np.float64)
    blocks = -(-x.size // block)
    padded = np.zeros(blocks * block)
    padded[:x.size] = np.abs(x)
    padded = padded.reshape(blocks, block)
    scale = padded.max(1)
    scale = np.where(scale < 2.0 ** -120, 0.0, scale)
    r = padded / np.where(scale > 0, scale, np.inf)[:, None]
    levels = q8_levels(7 if signed else 8)
    middle = (levels[1:] + levels[:-1]) / 2
    # the line of the lowest interval starts at 8^-bits, not at 0
    middle[0] = (levels[1] + 8.0 ** -(7 if signed else 8)) / 2 if signed else 0.0
    codes = np.searchsorted(middle, r, side="left").reshape(-1)[:x.size]
    gap = np.abs(r[..., None] - middle).min(-1).reshape(-1)[:x.size] if x.size <= 1 << 16 else None
    return codes + np.where(signed & (x < 0), 128, 0), scale, gap
