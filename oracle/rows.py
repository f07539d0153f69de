"""Oracle: token rows in expert order and back, the router's gradient, and
4-bit products of single matrices, fp64.

The pages apply k of E experts to each token and sum their outputs with the
routing weights ("How it works"); the sorted order is the stable bucketing of
bucket.py (a pair whose expert lies outside [0, E) is in no bucket), the
gradients are those of the formulas in layer.py:

  sort     X[row(i)] = x[t], i = t k + r        dx[t] = sum_r dX[row(t,r)]
  unsort   y[t] = sum_r w[t,r] Y[row(t,r)] + s_t o[t]
           dY[row] = w dy[t], dw = <dy[t], Y[row]>, do = s dy, ds = <dy, o>
  router   w = softmax of the chosen logits, s = sigmoid of the shared logit;
           g = w (dw - sum_j w_j dw_j), g_s = s (1 - s) ds,
           over the chosen logits: a pair without an expert is not among them;
           dx = sum_r g W[e_r] + g_s W[E], dW, db the same by expert.
"""
from __future__ import annotations

import numpy as np


def sort_rows(x, idx, E: int):
    """(x_sorted [live][d], offsets, pair_ids [live], row_of [T][k])."""
    T, k = idx.shape
    pairs = [[] for _ in range(E)]
    for i, e in enumerate(np.asarray(idx).ravel().tolist()):
        if 0 <= e < E:
            pairs[e].append(i)
    pair_ids = np.array([i for b in pairs for i in b], np.int32)
    offsets = np.concatenate([[0], np.cumsum([len(b) for b in pairs])]).astype(np.int32)
    row_of = np.full(T * k, -1, np.int32)
    row_of[pair_ids] = np.arange(pair_ids.size)
    return np.asarray(x)[pair_ids // k], offsets, pair_ids, row_of.reshape(T, k)


def sort_rows_grad(dX, row_of):
    dX = np.asarray(dX, np.float64)
    T, k = row_of.shape
    dx = np.zeros((T, dX.shape[1]))
    for r in range(k):
        t = np.nonzero(row_of[:, r] >= 0)[0]
        dx[t] += dX[row_of[t, r]]
    return dx


def unsort(rows, row_of, w, shared=None, gate=None):
    rows = np.asarray(rows, np.float64)
    T, k = row_of.shape
    y = np.zeros((T, rows.shape[1]))
    for r in range(k):
        t = np.nonzero(row_of[:, r] >= 0)[0]
        y[t] += np.asarray(w, np.float64)[t, r][:, None] * rows[row_of[t, r]]
    if shared is not None:
        y += np.asarray(gate, np.float64)[:, None] * np.asarray(shared, np.float64)
    return y


def unsort_grad(dy, rows, row_of, w, shared=None, gate=None):
    """(drows with zeros where no pair points, dw, dshared, dgate)."""
    dy, rows, w = (np.asarray(a, np.float64) for a in (dy, rows, w))
    T, k = row_of.shape
    drows, dw = np.zeros_like(rows), np.zeros((T, k))
    for t in range(T):
        for r in range(k):
            p = row_of[t, r]
            if p >= 0:
                drows[p] = w[t, r] * dy[t]
                dw[t, r] = dy[t] @ rows[p]
    if shared is None:
        return drows, dw, None, None
    g = np.asarray(gate, np.float64)
    return drows, dw, g[:, None] * dy, np.sum(dy * np.asarray(shared, np.float64), axis=1)


def router_logit_grad(idx, w, gate, dw, dgate, E: int):
    """Dense [T][E+1] gradient of the logits (column E the shared gate's)."""
    w, dw = np.asarray(w, np.float64), np.asarray(dw, np.float64)
    T, k = w.shape
    dl = np.zeros((T, E + 1))
    for t in range(T):
        chosen = [r for r in range(k) if 0 <= idx[t, r] < E]
        z = w[t, chosen] @ dw[t, chosen]
        for r in chosen:
            dl[t, idx[t, r]] += w[t, r] * (dw[t, r] - z)
    if dgate is not None:
        s = np.asarray(gate, np.float64)
        dl[:, E] = s * (1 - s) * np.asarray(dgate, np.float64)
    return dl


def router_grad(x, W, idx, w, gate, dw, dgate):
    """(dx, dW, dbias)."""
    x, W = np.asarray(x, np.float64), np.asarray(W, np.float64)
    E = W.shape[0] - 1
    dl = router_logit_grad(idx, w, gate, dw, dgate, E)
    return dl @ W, dl.T @ x, dl[:, :E].sum(0)


# ------------------------------------------------------------ 4-bit matrices
def linear_weights(codes, scales, biases):
    """fp64 [out][in] of MLX affine codes with one (scale, bias) per in / scales.shape[1] inputs."""
    group = codes.shape[1] // scales.shape[1]
    s, b = (np.repeat(np.asarray(a, np.float64), group, axis=1) for a in (scales, biases))
    return s * np.asarray(codes, np.float64) + b


def pack_linear(codes, scales, biases) -> np.ndarray:
    """Codes [in/32][out][16 bytes] (input 32c + 2b in the low nibble of byte b), then (scale, bias) [in/group][out]."""
    out, n_in = codes.shape
    c = np.asarray(codes, np.uint8).reshape(out, n_in // 32, 16, 2)
    body = (c[..., 0] | (c[..., 1] << 4)).transpose(1, 0, 2).ravel()
    sb = np.stack([np.asarray(scales, np.float16).T, np.asarray(biases, np.float16).T], axis=-1)
    return np.concatenate([body, np.ascontiguousarray(sb).view(np.uint8).ravel()])
