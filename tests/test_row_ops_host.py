"""Row operators, 4-bit products and the router's gradient, without a GPU: the
oracle's gradients against central differences of its own forward, the packer
of single matrices against the oracle's and against an expert blob, workspace
sizes, and the refusal of bad calls before any device work."""
import ctypes as C

import numpy as np
import pytest

import moe_synth as ms
import sparse_moe_decode_router_amd as moe
from oracle import layer as olayer
from oracle import quant as oquant
from oracle import rows as orows

LIB = moe._lib
BAD, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK
P = 4096          # a stand-in address: no call below reaches a kernel
WS = 1 << 30


# ------------------------------------------------------------------- oracle
def _routing(rng, T, k, E, drop=0.2):
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[rng.random((T, k)) < drop] = -1
    return idx


def test_oracle_sort_places_every_live_pair_once():
    rng = np.random.default_rng(0)
    idx = _routing(rng, 9, 3, 5)
    idx[4] = -1
    idx[5, 0] = 5
    x = rng.standard_normal((9, 4))
    X, off, pairs, row_of = orows.sort_rows(x, idx, 5)
    live = [(e, i) for i, e in enumerate(idx.ravel()) if 0 <= e < 5]
    assert [i for _, i in sorted(live)] == pairs.tolist()          # by expert, then by pair
    assert off[-1] == len(live) and (row_of[4] == -1).all() and row_of[5, 0] == -1
    for p, i in enumerate(pairs):
        assert off[idx.ravel()[i]] <= p < off[idx.ravel()[i] + 1]
        assert np.array_equal(X[p], x[i // 3]) and row_of[i // 3, i % 3] == p


def _differences(f, a, h=1e-5):
    g = np.zeros_like(a)
    for j in np.ndindex(a.shape):
        up, dn = a.copy(), a.copy()
        up[j] += h
        dn[j] -= h
        g[j] = (f(up) - f(dn)) / (2 * h)
    return g


def test_oracle_row_gradients_against_differences():
    """Sort and unsort are linear in each argument: central differences are
    exact up to rounding (1e-16 / 1e-5 relative to values of order ten)."""
    rng = np.random.default_rng(1)
    T, k, E, d = 4, 3, 5, 3
    idx = _routing(rng, T, k, E)
    x, dY = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    X, _, _, row_of = orows.sort_rows(x, idx, E)
    G = rng.standard_normal(X.shape)
    dx = _differences(lambda a: np.sum(G * orows.sort_rows(a, idx, E)[0]), x)
    assert np.allclose(dx, orows.sort_rows_grad(G, row_of), atol=1e-8)
    rows, w = rng.standard_normal(X.shape), rng.random((T, k))
    sh, gate = rng.standard_normal((T, d)), rng.random(T)
    f = lambda a, b, c, e: np.sum(dY * orows.unsort(a, row_of, b, c, e))
    dr, dw, ds, dg = orows.unsort_grad(dY, rows, row_of, w, sh, gate)
    assert np.allclose(_differences(lambda a: f(a, w, sh, gate), rows), dr, atol=1e-8)
    assert np.allclose(_differences(lambda a: f(rows, a, sh, gate), w), dw, atol=1e-8)
    assert np.allclose(_differences(lambda a: f(rows, w, a, gate), sh), ds, atol=1e-8)
    assert np.allclose(_differences(lambda a: f(rows, w, sh, a), gate), dg, atol=1e-8)


def test_oracle_router_gradient_against_differences():
    """The whole router (softmax over the chosen logits, sigmoid gate) against
    central differences; h^2 times third derivatives of order ten stays below
    the 1e-7 taken here."""
    rng = np.random.default_rng(2)
    T, k, E, d = 5, 2, 6, 4
    x, W = rng.standard_normal((T, d)), rng.standard_normal((E + 1, d))
    b, dw, dg = rng.standard_normal(E), rng.standard_normal((T, k)), rng.standard_normal(T)
    idx = olayer.select_topk(olayer.router_logits(x, W, b)[0], k)

    def loss(x_, W_, b_):
        l, g = olayer.router_logits(x_, W_, b_)
        return np.sum(dw * olayer.topk_weights(l, idx)) + np.sum(dg * olayer.sigmoid(g))

    l, g = olayer.router_logits(x, W, b)
    gx, gW, gb = orows.router_grad(x, W, idx, olayer.topk_weights(l, idx), olayer.sigmoid(g), dw, dg)
    assert np.allclose(_differences(lambda a: loss(a, W, b), x), gx, atol=1e-7)
    assert np.allclose(_differences(lambda a: loss(x, a, b), W), gW, atol=1e-7)
    assert np.allclose(_differences(lambda a: loss(x, W, a), b), gb, atol=1e-7)


def test_oracle_router_gradient_with_dropped_pairs_against_differences():
    """With some of the chosen pairs dropped, the weights are the softmax over
    the others; what a dropped pair's weight and gradient hold is not used.
    Tolerance as above."""
    rng = np.random.default_rng(3)
    T, k, E, d = 6, 3, 7, 4
    x, W = rng.standard_normal((T, d)), rng.standard_normal((E + 1, d))
    idx, dw = _routing(rng, T, k, E, drop=0.4), rng.standard_normal((T, k))
    idx[2], idx[3, 1] = -1, E
    live = (idx >= 0) & (idx < E)
    assert live.any(1).sum() >= 4 and (~live[live.any(1)]).any()

    def weights(x_, W_):
        l = np.take_along_axis(x_ @ W_[:E].T, np.where(live, idx, 0), 1)
        e = np.where(live, np.exp(l), 0)
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)

    loss = lambda x_, W_: np.sum(np.where(live, dw, 0) * weights(x_, W_))
    w, g = np.where(live, weights(x, W), np.nan), np.where(live, dw, np.inf)
    gx, gW, gb = orows.router_grad(x, W, idx, w, None, g, None)
    assert np.allclose(_differences(lambda a: loss(a, W), x), gx, atol=1e-7)
    assert np.allclose(_differences(lambda a: loss(x, a), W), gW, atol=1e-7)
    # moving all logits of a token alike changes no weight
    assert np.allclose(orows.router_logit_grad(idx, w, None, g, None, E).sum(1), 0, atol=1e-14) and abs(gb.sum()) < 1e-13


# ------------------------------------------------------------------ packing
def _matrix(rng, out, n_in, group):
    codes = rng.integers(0, 16, (out, n_in), dtype=np.uint8)
    s = rng.uniform(0.002, 0.02, (out, n_in // group)).astype(np.float16)
    return codes, s, (-8 * s.astype(np.float32) * rng.uniform(0.9, 1.1, s.shape)).astype(np.float16)


@pytest.mark.parametrize("out,n_in,group", [(1, 32, 32), (5, 96, 32), (17, 64, 64), (64, 320, 64), (3, 384, 128)])
def test_pack_linear_matches_oracle_and_round_trips(out, n_in, group):
    c, s, b = _matrix(np.random.default_rng(out), out, n_in, group)
    packed = moe.moe_pack_linear_int4(c, s, b)
    assert packed.size == moe.moe_linear_bytes(n_in, out, group)
    assert np.array_equal(packed, orows.pack_linear(c, s, b))
    for a, w in zip(moe.moe_unpack_linear_int4(packed, n_in, out, group), (c, s, b)):
        assert np.array_equal(a, w)


def test_a_packed_matrix_is_a_section_of_an_expert_blob():
    cfg = ms.CONFIGS["tiny"]
    raw = ms.expert_raw(cfg, 3)
    blob = moe.moe_pack_expert(raw, cfg.d, cfg.I)
    parts = [moe.moe_pack_linear_int4(*(raw[m][f] for f in ("codes", "scales", "biases"))) for m in oquant.MATS]
    assert np.array_equal(np.concatenate(parts), blob[:moe.moe_blob_bytes(cfg.d, cfg.I)])
    assert np.array_equal(orows.linear_weights(*(raw["up"][f] for f in ("codes", "scales", "biases"))),
                          oquant.dequant(raw["up"]))


def test_pack_linear_refusals():
    c, s, b = _matrix(np.random.default_rng(1), 4, 64, 64)
    bad = c.copy()
    bad[3, 63] = 16
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_pack_linear_int4(bad, s, b)
    assert ei.value.status == BAD
    with pytest.raises(ValueError):
        moe.moe_pack_linear_int4(c, s[:2], b[:2])
    with pytest.raises(ValueError):
        moe.moe_unpack_linear_int4(np.zeros(7, np.uint8), 64, 4)
    for n_in, out, g in [(0, 4, 64), (96, 4, 64), (64, 0, 64), (64, 4, 16), (64, 4, 256), (65536 + 64, 4, 64),
                         (64, (1 << 24) + 1, 64), (-64, 4, 64)]:
        assert moe.moe_linear_bytes(n_in, out, g) == 0


@pytest.mark.parametrize("bad", [256, 16 + 256, -256, 7.5, np.nan])
def test_pack_linear_refuses_codes_that_do_not_fit_a_byte(bad):
    """Codes that a conversion to bytes would turn into other codes."""
    c, s, b = _matrix(np.random.default_rng(2), 4, 64, 64)
    wide = c.astype(np.float64 if isinstance(bad, float) else np.int64)
    assert np.array_equal(moe.moe_pack_linear_int4(wide, s, b), moe.moe_pack_linear_int4(c, s, b))
    wide[2, 5] = bad
    with pytest.raises(ValueError):
        moe.moe_pack_linear_int4(wide, s, b)


def test_pack_linear_refuses_scales_that_do_not_fit_fp16():
    c, s, b = _matrix(np.random.default_rng(2), 4, 64, 64)
    assert np.array_equal(moe.moe_pack_linear_int4(c, s.astype(np.float64), b.astype(np.float32)),
                          moe.moe_pack_linear_int4(c, s, b))
    for i in range(2):
        a = [s.astype(np.float32), b.astype(np.float32)]
        a[i][1, 0] = 65520.0                           # halfway past the largest fp16: rounds to infinity
        with pytest.raises(ValueError):
            moe.moe_pack_linear_int4(c, *a)
    with pytest.raises(ValueError):
        moe.moe_unpack_linear_int4(moe.moe_pack_linear_int4(c, s, b).astype(np.int32), 64, 4)


# ----------------------------------------------------------------- refusals
def test_sort_refusals():
    def call(x=P, ty=moe.MOE_TYPE_BF16, T=4, d=8, idx=P, k=2, E=4, out=P, off=P, pairs=P, row=P, ws=P, nws=WS):
        return LIB.moe_sort_tokens(x, ty, T, d, idx, k, E, out, off, pairs, row, ws, nws, None)
    for kw in [dict(x=None), dict(idx=None), dict(out=None), dict(off=None), dict(pairs=None), dict(row=None),
               dict(ws=None), dict(ty=3), dict(ty=-1), dict(T=-1), dict(d=0), dict(k=0), dict(E=0), dict(E=1025),
               dict(x=P + 1), dict(ty=moe.MOE_TYPE_F32, x=P + 2), dict(out=P + 1), dict(ws=P + 4), dict(nws=64),
               dict(row=P + 2), dict(off=P + 1), dict(idx=P + 3)]:
        assert call(**kw) == BAD, kw
    for kw in [dict(k=1025), dict(d=(1 << 20) + 1), dict(T=1 << 28, k=8)]:
        assert call(**kw) == UNS, kw
    assert moe.moe_sort_workspace_bytes(4, 2, 4) > 0
    for a in [(-1, 2, 4), (4, 0, 4), (4, 2, 0), (4, 2, 1025), (4, 1025, 4), (1 << 28, 8, 4)]:
        assert moe.moe_sort_workspace_bytes(*a) == 0


def test_back_refusals():
    def grad(x=P, ty=1, T=4, k=2, d=8, row=P, out=P):
        return LIB.moe_sort_tokens_backward(x, ty, T, k, d, row, out, None)

    def back(x=P, ty=1, T=4, k=2, d=8, row=P, w=P, sh=None, sg=None, y=P):
        return LIB.moe_unsort_combine(x, ty, T, k, d, row, w, sh, sg, y, None)

    def backgrad(dy=P, x=P, ty=1, T=4, k=2, d=8, row=P, w=P, sh=None, sg=None, dx=P, dw=P, dsh=None, dsg=None):
        return LIB.moe_unsort_combine_backward(dy, x, ty, T, k, d, row, w, sh, sg, dx, dw, dsh, dsg, None)
    for f in (grad, back, backgrad):
        assert f(T=0) == OK
        for kw in [dict(x=None), dict(row=None), dict(ty=9), dict(T=-2), dict(k=0), dict(d=0), dict(x=P + 1),
                   dict(row=P + 1)]:
            assert f(**kw) == BAD, (f, kw)
        assert f(k=1025) == UNS and f(d=(1 << 20) + 1) == UNS and f(T=1 << 29, k=4) == UNS
    assert grad(out=None) == BAD and back(y=None) == BAD and back(w=None) == BAD and back(w=P + 2) == BAD
    assert back(sh=P) == BAD and back(sg=P) == BAD and back(y=P + 1) == BAD
    for kw in [dict(dy=None), dict(w=None), dict(dx=None), dict(dw=None), dict(sh=P), dict(sh=P, sg=P),
               dict(sh=P, sg=P, dsh=P), dict(dsh=P, dsg=P), dict(sg=P), dict(dx=P + 1), dict(dw=P + 2)]:
        assert backgrad(**kw) == BAD, kw


def test_linear_refusals():
    sh = lambda i=64, o=8, g=64: C.byref(moe.moe_linear_shape(i, o, g))

    def lin(s=None, w=P, x=P, T=2, y=P):
        return LIB.moe_linear_int4(s or sh(), w, x, T, y, None)

    def exp(s=None, w=P, st=4096, n=4, tab=P, E=4, x=P, N=2, off=P, y=P, err=None):
        return LIB.moe_expert_linear_int4(s or sh(), w, st, n, tab, E, x, N, off, y, err, None)
    assert lin(T=0, w=None, x=None, y=None) == OK and exp(N=0, w=None, x=None, y=None, off=None) == OK
    assert LIB.moe_linear_int4(None, P, P, 1, P, None) == BAD
    for s in [sh(96), sh(64, 0), sh(64, 8, 48), sh(0), sh(65600)]:
        assert lin(s) == BAD and exp(s) == BAD
    for kw in [dict(w=None), dict(x=None), dict(y=None), dict(w=P + 2), dict(x=P + 8), dict(y=P + 2)]:
        assert lin(**kw) == BAD and exp(**kw) == BAD, kw
    assert lin(T=-1) == BAD and exp(N=-1) == BAD
    for kw in [dict(off=None), dict(E=0), dict(E=1025), dict(n=0), dict(tab=None, n=3), dict(st=2), dict(st=256),
               dict(st=4098), dict(err=P + 1), dict(tab=P + 2)]:
        assert exp(**kw) == BAD, kw
    assert exp(N=(1 << 30) + 1) == UNS
    assert LIB.moe_pool_linear_int4(None, 0, P, 1, P, P, None) == BAD


def test_router_backward_refusals():
    def call(x=P, T=4, d=64, W=P, E=8, k=2, idx=P, w=P, sg=P, dw=P, dsg=P, off=P, pairs=P, dx=P, dW=P, db=P, ws=P,
             n=WS):
        return LIB.moe_router_topk_backward(x, T, d, W, E, k, idx, w, sg, dw, dsg, off, pairs, dx, dW, db, ws, n, None)
    for kw in [dict(x=None), dict(W=None), dict(idx=None), dict(w=None), dict(sg=None), dict(dw=None),
               dict(off=None), dict(pairs=None), dict(dx=None, dW=None, db=None), dict(ws=None), dict(n=16),
               dict(T=-1), dict(d=0), dict(d=100), dict(d=8256), dict(E=0), dict(E=1025), dict(k=0), dict(k=9),
               dict(x=P + 8), dict(W=P + 4), dict(dx=P + 4), dict(dW=P + 8), dict(ws=P + 16), dict(T=1 << 29, k=8)]:
        assert call(**kw) == BAD, kw
    f = moe.moe_router_backward_workspace_bytes
    assert f(4, 64, 8, 2) > 0 and f(4, 100, 8, 2) == 0 and f(4, 64, 8, 9) == 0 and f(-1, 64, 8, 2) == 0
    assert f(4096, 2048, 512, 10) < 24 << 20


def test_sizes_past_32_bits_are_not_those_of_their_low_bits():
    big = 1 << 32
    for f, a in [(moe.moe_linear_bytes, (64, 8, 64)), (moe.moe_sort_workspace_bytes, (4, 2, 4)),
                 (moe.moe_router_backward_workspace_bytes, (4, 64, 8, 2))]:
        assert f(*a) > 0
        for i in range(len(a)):
            for v in (a[i] + big, a[i] - big):
                assert f(*a[:i], v, *a[i + 1:]) == 0, (f, i, v)
    with pytest.raises(ValueError):
        moe.moe_unpack_linear_int4(np.zeros(moe.moe_linear_bytes(64, 8), np.uint8), 64, 8 + big)


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 1, dtype=torch.int32)
    off = torch.zeros(9, dtype=torch.int32)
    f = torch.zeros(2, 1)
    packed = torch.zeros(8, moe.moe_linear_bytes(64, 8), dtype=torch.uint8)
    for call in [lambda: moe.moe_sort_tokens(x, i, 8), lambda: moe.moe_sort_tokens_backward(x, i),
                 lambda: moe.moe_unsort_combine(x, i, f), lambda: moe.moe_unsort_combine_backward(x, x, i, f),
                 lambda: moe.moe_linear_int4(packed[0], x, 8),
                 lambda: moe.moe_expert_linear_int4(packed, None, x, off, 8),
                 lambda: moe.moe_router_topk_backward(x, torch.zeros(9, 64), i, f, f[:, 0], f, None, off, i[:, 0])]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        moe.moe_sort_tokens(x.to(torch.float64), i, 8)
    with pytest.raises(ValueError):
        moe.moe_sort_tokens(x[0], i, 8)
