"""Plain 64-bit forms of the fp8 expert path's operators, for the tests: the
formulas of include/moe_gb300.h in numpy, and the error bounds that 32-bit
arithmetic with one rounding per output can be held to."""
import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
FLOOR = 2.0 ** -100


def blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------ e4m3

def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        t[c] = s * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
        if e == 15 and m == 7:
            t[c] = np.nan
    return t


E4M3 = _e4m3_table()


def e4m3_step(v):
    """Spacing of the e4m3 numbers around |v|."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)


def round_e4m3(v):
    s = e4m3_step(v)
    return np.rint(v / s) * s          # rint: to even, as the conversion


def expand(s, n, axis):
    return np.take(np.repeat(s, BLOCK, axis), np.arange(n), axis)


def quantise(v):
    """(codes' values, scales, unrounded codes) of fp64 rows."""
    n, H = v.shape
    nb = blocks(H)
    p = np.zeros((n, nb * BLOCK))
    p[:, :H] = v
    a = np.maximum(np.abs(p.reshape(n, nb, BLOCK)).max(2), FLOOR)
    s = a / E4M3_MAX
    u = v / expand(s, H, 1)
    return round_e4m3(u), s, u


# ------------------------------------------------------------------ norm

def add_rms_norm(x, residual, w, eps):
    h = x if residual is None else x + residual
    v = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w
    return h, v


# ------------------------------------------------------------------ gate

CLOSED = -1e30


def gate_keys(logits, bias, mask, score, groups, topk_groups, group_score):
    """(keys with the groups' choice applied, scores, group values or None)."""
    T, E = logits.shape
    with np.errstate(all="ignore"):
        open_ = logits > CLOSED
        if mask is not None:
            open_ &= (mask != 0)[:, None]
        l = np.where(open_, np.minimum(logits, np.finfo(np.float32).max), -np.inf)
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            m = np.where(open_.any(1), l.max(1), 0.0)[:, None]
            ex = np.exp(l - m)
            s = ex / np.maximum(ex.sum(1, keepdims=True), 1e-300)
    s = np.where(open_, s, 0.0)
    key = np.where(open_, s if bias is None else s + bias, -np.inf)
    gv = None
    if groups > 1:
        per = np.sort(key.reshape(T, groups, -1), axis=2)[:, :, ::-1]
        gv = per[:, :, 0].copy()
        if group_score == "top2" and per.shape[2] > 1:
            gv = np.where(per[:, :, 1] > -np.inf, per[:, :, 0] + per[:, :, 1], gv)
        keep = np.zeros((T, groups), bool)
        best = np.argsort(-gv, axis=1, kind="stable")[:, :topk_groups]
        np.put_along_axis(keep, best, True, axis=1)
        key = np.where(np.repeat(keep, E // groups, 1), key, -np.inf)
    return key, s, gv


def gate(logits, bias, mask, K, score, groups, topk_groups, group_score, renormalize, scale):
    key, s, _ = gate_keys(logits, bias, mask, score, groups, topk_groups, group_score)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    on = np.take_along_axis(key, ids, 1) > -np.inf
    w = np.where(on, np.take_along_axis(s, ids, 1), 0.0)
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return np.where(on, ids, -1), w * scale, on.astype(np.uint8)


def near_ties(v):
    """Rows in which two of the largest values differ by less than their
    32-bit rounding could decide (equal values are not near: they tie)."""
    with np.errstate(invalid="ignore"):
        d = v[:, :-1] - v[:, 1:]
        return ((d > 0) & (d < 4e-6 * np.abs(v[:, :-1]) + 1e-30)).any(1)


# ------------------------------------------------------------------ products

def product(rows, offsets, w):
    """Rows of expert e times w[e]^T and the sum of the terms' magnitudes."""
    out = np.zeros((rows.shape[0], w.shape[1]))
    mag = np.zeros_like(out)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        out[a:b] = rows[a:b] @ w[e].T
        mag[a:b] = np.abs(rows[a:b]) @ np.abs(w[e]).T
    return out, mag


def product_bound(mag, Kd):
    """|error| of a product summed in fp32: the at most 128 products of a block
    and the blocks' sums, one ulp (2^-23) each relative to the magnitudes' sum,
    and the scales' product and its application."""
    return mag * (min(Kd, BLOCK) + blocks(Kd) + 4) * 2.0 ** -23


def ffn(rows, offsets, w1, w2):
    """The FFN in 64 bits on dequantised rows and weights: (y, bound of a bf16
    result whose every step is in fp32).  An intermediate code may round the
    other way where its exact value is within the first product's error of a
    rounding boundary; the bound adds one code step there."""
    Nh = w1.shape[1] // 2
    h, mag = product(rows, offsets, w1)
    err = product_bound(mag, rows.shape[1])
    a, b = h[:, :Nh], h[:, Nh:]
    sig = 1.0 / (1.0 + np.exp(-a))
    g = a * sig * b
    # |d silu| <= 1.1; exp, division and products a few ulp
    eg = 1.1 * err[:, :Nh] * np.abs(b) + np.abs(a * sig) * err[:, Nh:] + 16 * 2.0 ** -24 * np.abs(g)
    q, s, u = quantise(g)
    se = expand(s, Nh, 1)
    gb = np.abs(g) + eg
    rel_s = np.zeros_like(s)
    for i in range(s.shape[1]):
        blk = slice(i * BLOCK, (i + 1) * BLOCK)
        rel_s[:, i] = eg[:, blk].max(1) / np.maximum(gb[:, blk].max(1) - eg[:, blk].max(1), 1e-300)
    rel_s = expand(rel_s, Nh, 1) + 4 * 2.0 ** -24
    eu = eg / se + np.abs(u) * rel_s              # how far an unrounded code may be off
    step = e4m3_step(np.abs(u) + eu)
    frac = np.abs(u) / step - np.floor(np.abs(u) / step)
    flips = np.abs(frac - 0.5) <= eu / step + 1e-12
    dq = np.where(flips, step, 0.0) * se + np.abs(q) * se * rel_s
    y, mag2 = product(q * se, offsets, w2)
    _, dy = product(dq, offsets, np.abs(w2))
    return y, dy + product_bound(mag2, Nh) + np.abs(y) * 2.0 ** -8 + 1e-30
