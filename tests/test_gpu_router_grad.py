"""Gradient of the router on the GPU, against the fp64 oracle, and a run of the
row operators, 4-bit products and gradients together as a caller of its own
expert products makes it.

Tolerance of the router's gradient, derived (u = 2^-24): z = sum w dw has k
terms, off by (k + 2) u sum|w dw|; g = w (dw - z) adds two roundings, so
|dg| <= w ((k + 2) u sum|w dw| + 2 u (|dw| + |z|)); dx is a sum of k + 1
products, off by sum |W| |dg| + (k + 3) u sum|g W|; dW and db are sums of at
most n products (n pairs of the expert), off by sum |x| |dg| + (n + 2) u sum|g x|."""
import numpy as np
import pytest

import moe_synth as ms
from gpu_support import DeviceLayer
from oracle import layer as olayer
from oracle import quant as oquant
from oracle import rows as orows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

U = 2.0 ** -24


def _np(t):
    return t.detach().cpu().double().numpy()


def _inputs(T, d, E, k, seed=0, drop=False, skew=False):
    g = np.random.default_rng([T, d, E, k, seed])
    bits = ms.f32_to_bf16_bits(g.standard_normal((T, d), dtype=np.float32))
    W = (0.05 * g.standard_normal((E + 1, d))).astype(np.float32)
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    if skew and T:
        idx[:, 0] = np.where((idx == 1).any(1), idx[:, 0], 1)      # one expert of every token
    if drop and T:
        idx[g.random((T, k)) < 0.2] = -1
    w = g.random((T, k)).astype(np.float32)
    w /= np.maximum(w.sum(1, keepdims=True), 1e-6)
    s, dw, ds = g.random(T).astype(np.float32), g.standard_normal((T, k)).astype(np.float32), g.standard_normal(T).astype(np.float32)
    return olayer.bf16_to_f64(bits), bits, W, idx, w, s, dw, ds


def _dev(bits, *a):
    return (torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16),) + tuple(torch.from_numpy(v).cuda() for v in a)


def _check(got, x, W, idx, w, s, dw, ds):
    T, k = idx.shape
    E = W.shape[0] - 1
    dx, dW, db = (_np(a) for a in got)
    rx, rW, rb = orows.router_grad(x, W, idx, w, s, dw, ds)
    g = np.abs(orows.router_logit_grad(idx, w, s, dw, ds, E))
    w64, dw64 = w.astype(np.float64), dw.astype(np.float64)
    z = np.sum(np.abs(w64 * dw64), 1, keepdims=True)
    dg_pair = w64 * ((k + 2) * U * z + 2 * U * (np.abs(dw64) + z))
    dg = np.zeros((T, E + 1))
    for r in range(k):
        t = np.nonzero((idx[:, r] >= 0) & (idx[:, r] < E))[0]
        dg[t, idx[t, r]] += dg_pair[t, r]
    dg[:, E] = 4 * U * g[:, E]
    n = np.concatenate([np.bincount(idx[(idx >= 0) & (idx < E)].ravel(), minlength=E), [T]])[:, None]
    aW, ax = np.abs(W.astype(np.float64)), np.abs(x)
    tiny = 2.0 ** -120
    assert (np.abs(dx - rx) <= dg @ aW + (k + 3) * U * (g @ aW) + tiny).all()
    assert (np.abs(dW - rW) <= dg.T @ ax + (n + 2) * U * (g.T @ ax) + tiny).all()
    assert (np.abs(db - rb) <= (dg.sum(0) + (n[:, 0] + 2) * U * g.sum(0))[:E] + tiny).all()


@pytest.mark.parametrize("T,d,E,k,kw", [
    (1, 64, 1, 1, {}), (1, 2048, 512, 10, {}), (3, 192, 7, 7, {}), (64, 576, 16, 4, dict(drop=True)),
    (65, 64, 4, 2, {}), (200, 512, 32, 3, dict(skew=True)), (129, 8192, 9, 2, {}), (300, 128, 1024, 16, {}),
    (1000, 320, 5, 3, dict(drop=True)), (40, 64, 128, 100, {}),
    (1500, 704, 16, 8, dict(drop=True, skew=True)), (5000, 64, 2, 1, {})])
def test_router_gradient(T, d, E, k, kw):
    x, bits, W, idx, w, s, dw, ds = _inputs(T, d, E, k, **kw)
    xd, Wd, idxd, wd, sd, dwd, dsd = _dev(bits, W, idx, w, s, dw, ds)
    _, off, pairs = moe.moe_bucket_tokens(idxd, E)
    got = moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dwd, dsd, off, pairs)
    _check(got, x, W, idx, w, s, dw, ds)
    # each output alone, and without the shared gate's gradient
    for i in range(3):
        out = [None] * 3
        out[i] = torch.full_like(got[i], float("nan"))
        moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dwd, dsd, off if i else None, pairs if i else None,
                                     out=tuple(out))
        assert torch.equal(out[i], got[i])
    none = moe.moe_router_topk_backward(xd, Wd, idxd, wd, None, dwd, None, off, pairs)
    assert torch.equal(none[1][:E], got[1][:E]) and (none[1][E] == 0).all() and torch.equal(none[2], got[2])


def test_router_gradient_without_tokens():
    x, bits, W, idx, w, s, dw, ds = _inputs(0, 128, 6, 2)
    xd, Wd, idxd, wd, sd, dwd, dsd = _dev(bits, W, idx, w, s, dw, ds)
    off = torch.zeros(7, dtype=torch.int32, device="cuda")
    out = (torch.empty(0, 128, device="cuda"), torch.full((7, 128), 5.0, device="cuda"), torch.full((6,), 5.0, device="cuda"))
    _, dW, db = moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dwd, dsd, off, idxd.view(-1), out=out)
    assert (dW == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T,d,E,k", [(90, 128, 8, 3), (40, 64, 128, 100), (1500, 128, 8, 4), (60, 64, 256, 130)])
def test_router_gradient_does_not_read_dropped_pairs(T, d, E, k):
    """Weights and their gradients at pairs without an expert change no bit of
    the results, whatever they hold (the pairs' g in the roles and, past 4096
    pairs, in a launch of their own)."""
    x, bits, W, idx, w, s, dw, ds = _inputs(T, d, E, k, drop=True)
    idx[0] = E
    out = (idx < 0) | (idx >= E)
    w, dw = np.where(out, 0, w).astype(np.float32), np.where(out, 0, dw).astype(np.float32)
    xd, Wd, idxd, wd, sd, dwd, dsd = _dev(bits, W, idx, w, s, dw, ds)
    _, off, pairs = moe.moe_bucket_tokens(idxd, E)
    want = moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dwd, dsd, off, pairs)
    _check(want, x, W, idx, w, s, dw, ds)
    z, nan, inf = torch.from_numpy(out).cuda(), float("nan"), float("inf")
    for a, b in [(nan, 0.0), (0.5, 2.0), (nan, nan), (inf, -inf)]:
        got = moe.moe_router_topk_backward(xd, Wd, idxd, wd.masked_fill(z, a), sd, dwd.masked_fill(z, b), dsd, off, pairs)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), (a, b)


@pytest.mark.parametrize("T", [60, 2100])
def test_dropped_pairs_through_the_way_back_and_the_router(T):
    """sort -> way back's gradient -> router's gradient with NaN in the weights
    of dropped pairs: the gradients of the same step without those weights."""
    d, E, k = 64, 16, 2
    x, bits, W, idx, w, s, dw, ds = _inputs(T, d, E, k, drop=True)
    xd, Wd, idxd, wd, sd, dwd, dsd = _dev(bits, W, idx, np.where(idx < 0, np.nan, w).astype(np.float32), s, dw, ds)
    X, off, pairs, row = moe.moe_sort_tokens(xd, idxd, E)
    _, dw2, _, ds2 = moe.moe_unsort_combine_backward(xd, X, row, wd, xd, sd)
    got = moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dw2, ds2, off, pairs)
    assert all(torch.isfinite(a).all() for a in got)
    _check(got, x, W, idx, np.where(idx < 0, 0, w), s, dw2.cpu().numpy(), ds2.cpu().numpy())


@pytest.mark.parametrize("T", [40, 2100])
def test_router_gradient_without_a_gate_gradient(T):
    """No gradient of the shared gate: its row gets zeros and adds nothing, also
    with NaN in the token rows of padding and in the gate's own weights."""
    d, E, k = 192, 8, 2
    x, bits, W, idx, w, s, dw, ds = _inputs(T, d, E, k)
    idx[3] = -1
    xd, Wd, idxd, wd, sd, dwd, _ = _dev(bits, W, idx, w, s, dw, ds)
    _, off, pairs = moe.moe_bucket_tokens(idxd, E)
    for gate in (None, sd):
        want = moe.moe_router_topk_backward(xd, Wd, idxd, wd, gate, dwd, None, off, pairs)
        bad_x, bad_W = xd.clone(), Wd.clone()
        bad_x[3], bad_W[E] = float("nan"), float("inf")
        got = moe.moe_router_topk_backward(bad_x, bad_W, idxd, wd, gate, dwd, None, off, pairs)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and (got[1][E] == 0).all()
        assert (got[0][3] == 0).all()


def test_router_gradient_of_more_tokens_than_blocks():
    """dx of 2^26 tokens and some (2^24 blocks of four if each had its own,
    more threads than a launch counts), offsets past 2^32 elements.  One expert
    a token, so g = w (dw - w dw) and dx = g W[e] + g_s W[E]: two products and
    a sum on values off as in the tolerance above, 8 u of the magnitudes."""
    T, d, E = (1 << 26) + 5, 64, 2
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    W, w, s, dw, ds = rand(E + 1, d) - 0.5, rand(T, 1), rand(T), rand(T, 1) - 0.5, rand(T) - 0.5
    idx = torch.randint(0, E, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    dx = torch.full((T, d), float("nan"), device="cuda")
    moe.moe_router_topk_backward(x, W, idx, w, s, dw, ds, None, None, out=(dx, None, None))
    for a in range(0, T, 1 << 22):
        b = min(T, a + (1 << 22))
        wd, dwd, sd, dsd, Wd = (t.double() for t in (w[a:b], dw[a:b], s[a:b, None], ds[a:b, None], W))
        g, gs, We = wd * (dwd - wd * dwd), dsd * (sd - sd * sd), Wd[idx[a:b, 0].long()]
        mag = wd * (dwd.abs() + (wd * dwd).abs()) * We.abs() + gs.abs() * Wd[E].abs()
        assert ((dx[a:b].double() - (g * We + gs * Wd[E])).abs() <= 8 * U * mag).all(), a


def test_router_gradient_in_a_graph_and_on_a_stream():
    T, d, E, k = 150, 256, 12, 3
    x, bits, W, idx, w, s, dw, ds = _inputs(T, d, E, k, skew=True)
    xd, Wd, idxd, wd, sd, dwd, dsd = _dev(bits, W, idx, w, s, dw, ds)

    def step(stream=None):
        _, off, pairs, _ = moe.moe_sort_tokens(xd, idxd, E, stream=stream)
        return moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dwd, dsd, off, pairs, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for rep in range(4):
        dwd.copy_(torch.randn(T, k, device="cuda"))
        idxd.copy_(torch.roll(idxd, 3, 0))
        graph.replay()
        got = [a.clone() for a in held]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step())), rep


def test_two_streams_at_once():
    """The same calls on two streams, nothing waiting between them, give each stream its own results."""
    T, d, E, k = 120, 512, 24, 4
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets, want = [], []
    w4 = torch.from_numpy(moe.moe_pack_linear_int4(
        np.full((96, d), 7, np.uint8), np.full((96, d // 64), 0.01, np.float16), np.full((96, d // 64), -0.05, np.float16))).cuda()
    for seed in (1, 2):
        x, bits, W, idx, w, s, dw, ds = _inputs(T, d, E, k, seed=seed, skew=True)
        sets.append(_dev(bits, W, idx, w, s, dw, ds))

    def step(a, stream=None):
        xd, Wd, idxd, wd, sd, dwd, dsd = a
        X, off, pairs, row = moe.moe_sort_tokens(xd, idxd, E, stream=stream)
        y = moe.moe_unsort_combine(X, row, wd, xd, sd, stream=stream)
        return (y, moe.moe_linear_int4(w4, y, 96, stream=stream), moe.moe_sort_tokens_backward(X, row, stream=stream),
                *moe.moe_unsort_combine_backward(y, X, row, wd, xd, sd, stream=stream)[1:],
                *moe.moe_router_topk_backward(xd, Wd, idxd, wd, sd, dwd, dsd, off, pairs, stream=stream))

    want = [step(a) for a in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [step(a, st) for a, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for g, r in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, r))


# ------------------------------------------------------------- all together
def test_the_layer_from_its_parts():
    """router -> sort -> gate, up, down products -> back equals the layer: the
    parts carry the activation rows of the last product in bf16 (2^-9 of each
    value, averaging far below), within the layer's own bar of 2e-3 max|y|
    of the oracle with that rounding made there too."""
    L = DeviceLayer(ms.CONFIGS["tiny"])
    cfg = L.cfg
    xb, x = L.x(0, 40)
    idx, w, s = moe.moe_router_topk(x, L.Wr, L.bias, cfg.k)
    X, off, _, row = moe.moe_sort_tokens(x, idx, cfg.E)
    gate, up = (moe.moe_pool_linear_int4(L.pool, m, X, off) for m in ("gate", "up"))
    h = (torch.nn.functional.silu(gate) * up).bfloat16()
    Y = moe.moe_pool_linear_int4(L.pool, "down", h, off)
    sh = [torch.from_numpy(moe.moe_pack_linear_int4(*(L.shared_raw[m][f] for f in ("codes", "scales", "biases")))).cuda()
          for m in oquant.MATS]
    hs = (torch.nn.functional.silu(moe.moe_linear_int4(sh[0], x, cfg.I_shared)) *
          moe.moe_linear_int4(sh[1], x, cfg.I_shared)).bfloat16()
    y = _np(moe.moe_unsort_combine(Y, row, w, moe.moe_linear_int4(sh[2], hs, cfg.d), s))
    idx = idx.cpu().numpy()

    def ffn(raw, v):
        g, u = v @ oquant.dequant(raw["gate"]).T, v @ oquant.dequant(raw["up"]).T
        return olayer.bf16_to_f64(ms.f32_to_bf16_bits((g * olayer.sigmoid(g) * u).astype(np.float32))) @ \
            oquant.dequant(raw["down"]).T

    v = olayer.bf16_to_f64(xb)
    ref = _np(s)[:, None] * ffn(L.shared_raw, v)
    for t in range(40):
        for r in range(cfg.k):
            ref[t] += _np(w)[t, r] * ffn(L.raw(int(idx[t, r])), v[t:t + 1])[0]
    assert np.abs(y - ref).max() <= 2e-3 * np.abs(ref).max()
    whole = _np(moe.moe_layer_forward(L.layer, x)[0])
    assert np.abs(y - whole).max() <= 2 * 2e-3 * np.abs(whole).max()
    assert L.pool.check_error() == moe.MOE_OK


def test_a_training_step_through_the_routing():
    """Forward and backward of y = sum_r w_r tanh-free linear experts (dense
    fp32 products of the caller's own on the sorted rows) and a shared expert,
    router included, against torch's autograd of the same model in fp64 on the
    CPU.  Every sum has at most d = 128 (products), T = 90 (weight gradients)
    or k terms of fp32, chained three deep: 2^-24 (3 (128 + 90 + 8)) = 4e-5 of
    the magnitudes summed; those exceed the largest result by at most the
    square root of the number of terms times a constant of order one (random
    signs), so 1e-3 of the largest value is taken."""
    T, d, E, k = 90, 128, 6, 2
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x = r(T, d).bfloat16()
    Wr, A, S, dy = 0.1 * r(E + 1, d).float(), (0.1 * r(E, d, d)).float(), (0.1 * r(d, d)).float(), r(T, d).float()
    # on the device
    xd, Wd, Ad, Sd, dyd = (t.cuda() for t in (x, Wr, A, S, dy))
    idx, w, s = moe.moe_router_topk(xd, Wd, None, k)
    xf = xd.float()
    X, off, pairs, row = moe.moe_sort_tokens(xf, idx, E)
    o = off.tolist()
    Y = torch.cat([X[o[e]:o[e + 1]] @ Ad[e].t() for e in range(E)])
    sh = xf @ Sd.t()
    y = moe.moe_unsort_combine(Y, row, w, sh, s)
    dY, dw, dsh, ds = moe.moe_unsort_combine_backward(dyd, Y, row, w, sh, s)
    dX = torch.cat([dY[o[e]:o[e + 1]] @ Ad[e] for e in range(E)])
    dA = torch.stack([dY[o[e]:o[e + 1]].t() @ X[o[e]:o[e + 1]] for e in range(E)])
    dxr, dWr, _ = moe.moe_router_topk_backward(xd, Wd, idx, w, s, dw, ds, off, pairs)
    dx = moe.moe_sort_tokens_backward(dX, row) + dxr + dsh @ Sd
    # the same in fp64
    x64, Wr64, A64, S64 = (t.double().requires_grad_() for t in (x, Wr, A, S))
    l = x64 @ Wr64.t()
    sel = idx.cpu().long()
    w64 = torch.softmax(l.gather(1, sel), 1)
    y64 = torch.sigmoid(l[:, E:]) * (x64 @ S64.t())
    for q in range(k):
        y64 = y64 + w64[:, q:q + 1] * torch.bmm(A64[sel[:, q]], x64.unsqueeze(2)).squeeze(2)
    (y64 * dy.double()).sum().backward()
    for got, ref in [(y, y64), (dx, x64.grad), (dWr, Wr64.grad), (dA, A64.grad), (dsh.t() @ xf, S64.grad)]:
        ref = ref.detach()
        assert (got.cpu().double() - ref).abs().max() <= 1e-3 * ref.abs().max()
