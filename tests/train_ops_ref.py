"""64-bit references and error bounds of the grouped products and the 8-bit
checkpoints, written from their definitions (numpy, CPU).

Bounds.  A product of bf16 or fp32 numbers summed in fp32 is off by at most
GAMMA times the sum of its terms' magnitudes:
  tensor cores: every step adds 16 products with truncation.  The running sum,
    the alignment of the 16 products and their own sum lose at most one unit
    of the last place each, 3 * 2^-23 of the magnitudes a step; at most 32
    steps (512 terms) run before the partial sum is taken out, except for bf16
    outputs, where all K / 16 steps do;
  CUDA cores: at most 128 rounded additions in a row, 2^-24 each;
  the partial sums: one rounded addition, 2^-24, for every 128 terms at most.
A result in bf16 adds half a step, 2^-8 of its value.
"""
import math

import numpy as np

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def gamma(terms, out):
    steps = -(-terms // 16)
    if out == "f32":
        steps = min(steps, 32)
    return 3 * steps * 2.0 ** -23 + (128 + terms / 128) * 2.0 ** -24


def segments(offsets, rows):
    """[(g, first, end)] with bounds clamped to [0, rows]; a segment that ends before it starts is empty."""
    o = [min(max(int(v), 0), rows) for v in offsets]
    return [(g, o[g], max(o[g], o[g + 1])) for g in range(len(o) - 1)]


def grouped_gemm(x, w, bias, offsets, y0):
    """(y, sum of magnitudes), fp64; rows of no segment are y0's."""
    y, m = y0.astype(np.float64).copy(), np.zeros(y0.shape)
    for g, b, e in segments(offsets, len(x)):
        y[b:e] = x[b:e] @ w[g].T
        m[b:e] = np.abs(x[b:e]) @ np.abs(w[g]).T
        if bias is not None:
            y[b:e] += bias[g]
            m[b:e] += np.abs(bias[g])
    return y, m


def grouped_dgrad(dy, w, offsets, dx0):
    return grouped_gemm(dy, w.transpose(0, 2, 1), None, offsets, dx0)


def grouped_wgrad(x, dy, offsets, dw0=None, db0=None):
    """(dw, db, magnitudes of dw, of db); dw0, db0: what is added onto."""
    G, N, K = len(offsets) - 1, dy.shape[1], x.shape[1]
    dw = np.zeros((G, N, K)) if dw0 is None else dw0.astype(np.float64).copy()
    db = np.zeros((G, N)) if db0 is None else db0.astype(np.float64).copy()
    mw, mb = np.abs(dw), np.abs(db)
    for g, b, e in segments(offsets, len(x)):
        dw[g] += dy[b:e].T @ x[b:e]
        mw[g] += np.abs(dy[b:e]).T @ np.abs(x[b:e])
        db[g] += dy[b:e].sum(0)
        mb[g] += np.abs(dy[b:e]).sum(0)
    return dw, db, mw, mb


# ------------------------------------------------------------------ 8 bits
def keep(x, halves=1):
    """(q, e, values) of rows x, fp64 in, from the definition: per block of 32
    columns of each half, e = the fp32 exponent field of the largest magnitude."""
    rows, cols = x.shape
    c = cols // halves
    nb = -(-c // 32)
    q = np.zeros((rows, cols), np.int64)
    e = np.zeros((rows, halves * nb), np.int64)
    v = np.zeros((rows, cols))
    for r in range(rows):
        for h in range(halves):
            for b in range(nb):
                s = slice(h * c + 32 * b, h * c + min(32 * (b + 1), c))
                blk = x[r, s]
                if not np.isfinite(blk).all():
                    e[r, h * nb + b], v[r, s] = 255, math.nan
                    continue
                top = float(np.abs(blk).max())
                ex = max(0, math.frexp(top)[1] - 1 + 127) if top > 0 else 0  # 2^(ex - 127) <= top
                k = np.clip(np.rint(np.ldexp(blk, 133 - ex)), -127, 127)
                e[r, h * nb + b], q[r, s], v[r, s] = ex, k, np.ldexp(k, ex - 133)
    return q, e, v


def _sig(x):
    z = np.exp(-np.abs(x))
    return np.where(x < 0, z / (1 + z), 1 / (1 + z))


C2 = 2 * math.sqrt(2 / math.pi)
# exp(-|w|) below the smallest normal number may be taken as 0: that is
# 2^-126 times whatever it is multiplied with
TINY = 2.0 ** -126


def act(h, swiglu):
    """(a, bound of an fp32 evaluation).  sigmoid(w) costs exp (2^-22 and w's
    own rounding, 4 2^-24 |w|), a sum and a division (2 ulp each); the bound
    is that many ulp of the value, with a few more for the products."""
    if swiglu:
        g, u = np.split(h, 2, 1)
        a = g * _sig(g) * u
        return a, np.abs(a) * (2.0 ** -20 + np.abs(g) * 2.0 ** -21) + np.abs(g * u) * TINY
    w = C2 * (h + 0.044715 * h ** 3)
    a = h * _sig(w)
    return a, np.abs(a) * (2.0 ** -20 + np.abs(w) * 2.0 ** -21) + np.abs(h) * TINY


def act_grad(h, swiglu):
    """(act'(h) per column of h, bound), the bound over the summands' magnitudes."""
    if swiglu:
        g, u = np.split(h, 2, 1)
        s, n = _sig(g), _sig(-g)
        d = np.concatenate([u * s * (1 + g * n), g * s], 1)
        m = np.concatenate([np.abs(u) * s * (1 + np.abs(g) * n), np.abs(g) * s], 1)
        rel = 2.0 ** -19 + np.abs(g) * 2.0 ** -20
        z = np.concatenate([np.abs(u) * (1 + np.abs(g)), np.abs(g)], 1) * TINY
        return d, m * np.concatenate([rel, rel], 1) + z
    w = C2 * (h + 0.044715 * h ** 3)
    s, n, dw = _sig(w), _sig(-w), C2 * (1 + 3 * 0.044715 * h * h)
    return s + h * s * n * dw, (s + np.abs(h) * s * n * dw) * (2.0 ** -19 + np.abs(w) * 2.0 ** -20) + (1 + np.abs(h * dw)) * TINY
