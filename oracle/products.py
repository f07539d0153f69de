"""Oracle: the experts' products in 16-bit types and in e4m3, fp64.

The pages run a gated feed-forward block in each of the k experts of a token
("How it works"); written here for rows in expert order (rows.py), one matrix
of each kind an expert:

  linear   y = x W^T               dx = dy W, dW = dy^T x
  gated    h = act(g) u, g = x Wg^T, u = x Wu^T
           dg = dh u act'(g), du = dh act(g)
           dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
  fp8      code = e4m3(448 v / a), scale = a / 448, a = max |v| of the block
           (2^-96 at least); y = sum over blocks of the scaled products

act: "silu" g / (1 + e^-g), "gelu" g (1 + erf(g / sqrt 2)) / 2, "gelu_tanh"
g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2.  Rows outside the borders
are zeros in every output.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("silu", "gelu", "gelu_tanh")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(name: str, g):
    g = np.asarray(g, np.float64)
    if name == "silu":
        return g / (1 + np.exp(-g))
    if name == "gelu":
        return g * (1 + _erf(g / math.sqrt(2))) / 2
    return g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) / 2


def act_slope(name: str, g):
    g = np.asarray(g, np.float64)
    if name == "silu":
        s = 1 / (1 + np.exp(-g))
        return s + g * s * (1 - s)
    if name == "gelu":
        return (1 + _erf(g / math.sqrt(2))) / 2 + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    t = np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    return (1 + t) / 2 + g * (1 - t * t) / 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)


def _buckets(offsets):
    return [(e, slice(int(offsets[e]), int(offsets[e + 1]))) for e in range(len(offsets) - 1)]


def linear(W, x, offsets):
    """W [E][out][in], x [N][in]."""
    y = np.zeros((x.shape[0], W.shape[1]))
    for e, r in _buckets(offsets):
        y[r] = x[r] @ W[e].T
    return y


def linear_grad(dy, W, x, offsets):
    """(dx, dW)."""
    dx, dW = np.zeros(x.shape), np.zeros(W.shape)
    for e, r in _buckets(offsets):
        dx[r], dW[e] = dy[r] @ W[e], dy[r].T @ x[r]
    return dx, dW


def gated(Wg, Wu, x, offsets, name: str):
    """(h, g, u)."""
    g, u = linear(Wg, x, offsets), linear(Wu, x, offsets)
    return act(name, g) * u, g, u


def gated_grad(dh, Wg, Wu, x, offsets, name: str):
    """(dx, dWg, dWu)."""
    _, g, u = gated(Wg, Wu, x, offsets, name)
    dg, du = dh * u * act_slope(name, g), dh * act(name, g)
    (xg, dWg), (xu, dWu) = linear_grad(dg, Wg, x, offsets), linear_grad(du, Wu, x, offsets)
    return xg + xu, dWg, dWu


# ------------------------------------------------------------------- e4m3
# every number >= 0 of the format in order: exponent field 0 holds m / 8 2^-6
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])


def e4m3_codes(v):
    """Byte of the e4m3 number nearest to v (|v| <= 448), the even one where two are as near."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 0, len(E4M3) - 1)
    lo = np.maximum(hi - 1, 0)
    below, above = a - E4M3[lo], E4M3[hi] - a
    k = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (k | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def e4m3_values(codes):
    c = np.asarray(codes, np.uint8)
    return np.where(c >> 7, -1.0, 1.0) * E4M3[c & 127]


def quantize_fp8(x, block_rows: int):
    """(codes uint8, scales fp64) of x [rows][n]."""
    x = np.asarray(x, np.float64)
    rb, cb = -(-x.shape[0] // block_rows), -(-x.shape[1] // 128)
    codes, scales = np.zeros(x.shape, np.uint8), np.zeros((rb, cb))
    for i in range(rb):
        for j in range(cb):
            b = x[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]       # 448 b is exact
            a = max(np.abs(b).max(), 2.0 ** -96)
            codes[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128] = e4m3_codes(448 * b / a)
            scales[i, j] = a / 448
    return codes, scales


def linear_fp8(w, sw, x, sx, offsets):
    """w [E][out][in] and x [N][in] uint8 codes, sw [E][blocks][blocks], sx [N][blocks]."""
    up = lambda s, n, axis: np.take(np.repeat(s, 128, axis), np.arange(n), axis)
    W = e4m3_values(w) * up(up(np.asarray(sw, np.float64), w.shape[1], 1), w.shape[2], 2)
    return linear(W, e4m3_values(x) * up(np.asarray(sx, np.float64), x.shape[1], 1), offsets)
