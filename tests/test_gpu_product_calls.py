"""How the experts' products are called, on the GPU: a training step and an
e4m3 forward made of the package's calls, other streams, captured graphs, wrong
borders, long tensors, the same call twice, and what is refused."""
import math

import numpy as np
import pytest

from oracle import products as oproducts
from oracle import rows as orows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U, S = 2.0 ** -8, 2.0 ** -23                     # a rounding to bfloat16; an fp32 addition (half of that at least)


def _np(t):
    return t.detach().double().cpu().numpy()


def _layer(T=48, k=3, E=8, d=72, I=40, seed=0):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E - 1)[:k] for _ in range(T)]).astype(np.int32)     # the last expert: no rows
    idx[rng.random((T, k)) < 0.1] = -1
    r = lambda *s: torch.from_numpy(rng.standard_normal(s)).cuda()
    x, dy = r(T, d).to(BF16), r(T, d).to(BF16)
    w = torch.softmax(r(T, k), 1).float()
    wg, wu = (r(E, I, d) / math.sqrt(d)).to(BF16), (r(E, I, d) / math.sqrt(d)).to(BF16)
    wd = (r(E, d, I) / math.sqrt(I)).to(BF16)
    return rng, idx, torch.from_numpy(idx).cuda(), x, dy, w, wg, wu, wd


def _step(idx, x, dy, w, wg, wu, wd, E):
    """Forward and gradients of y = sum_r w W_d (silu(W_g x) W_u x) by the package's calls."""
    X, off, _, row_of = moe.moe_sort_tokens(x, idx, E)
    h, pre = moe.moe_gated(wg, wu, X, off, save=True)
    Y = moe.moe_linear(wd, h, off)
    y = moe.moe_unsort_combine(Y, row_of, w)
    dY, dw, _, _ = moe.moe_unsort_combine_backward(dy, Y, row_of, w)
    dh, dwd = moe.moe_linear_backward(dY, wd, h, off)
    dX, dwg, dwu = moe.moe_gated_backward(dh, pre, wg, wu, X, off)
    return y, moe.moe_sort_tokens_backward(dX, row_of), dw, dwg, dwu, dwd


def test_training_step_of_the_routed_experts():
    """Against the fp64 oracle, with what each rounding along the way may do
    carried to the end: every product takes |operand error| through |other
    operand| and adds its own sums (S per addition) and rounding (U)."""
    rng, idx, idx_d, x, dy, w, wg, wu, wd = _layer()
    E = wg.shape[0]
    y, dx, dw, dwg, dwu, dwd = _step(idx_d, x, dy, w, wg, wu, wd, E)
    xn, dyn, wn, G, V, D = (_np(a) for a in (x, dy, w, wg, wu, wd))
    X, off, _, row_of = orows.sort_rows(xn, idx, E)
    d, I = X.shape[1], G.shape[1]
    ab, lin, grad = np.abs, oproducts.linear, oproducts.linear_grad

    def product(W, a, ea, K):                              # values and bound of a W^T, rounded
        v = lin(W, a, off)
        e = lin(ab(W), ea, off) + (K + 2) * S * lin(ab(W), ab(a) + ea, off)
        return v, e + U * (ab(v) + e)
    hn, g, u = oproducts.gated(G, V, X, off, "silu")
    f, df = oproducts.act("silu", g), oproducts.act_slope("silu", g)
    eg, eu = (d + 2) * S * lin(ab(G), ab(X), off), (d + 2) * S * lin(ab(V), ab(X), off)
    own = (g * g + ab(g) + 8) * 2 * S
    eh = 1.13 * eg * ab(u) + ab(f) * eu + 1.13 * eg * eu + (own + U) * ab(hn)
    Yn, eY = product(D, hn, eh, I)
    yn = orows.unsort(Yn, row_of, wn)
    ey = orows.unsort(eY, row_of, wn) + (len(wn[0]) + 2) * S * orows.unsort(ab(Yn) + eY, row_of, wn)
    assert (ab(_np(y) - yn) <= ey + U * (ab(yn) + ey)).all()
    dYn, dwn, _, _ = orows.unsort_grad(dyn, Yn, row_of, wn)
    edw = orows.unsort_grad(ab(dyn), eY + (d + 2) * S * (ab(Yn) + eY), row_of, wn)[1]
    assert (ab(_np(dw) - dwn) <= edw).all()
    edY = (U + S) * ab(dYn)
    # dh = dY D, dD = dY^T h
    dhn, dDn = grad(dYn, D, hn, off)
    edh, _ = grad(edY, ab(D), hn, off)
    sdh, _ = grad(ab(dYn) + edY, ab(D), hn, off)
    edh = edh + (d + 2) * S * sdh
    edh = edh + U * (ab(dhn) + edh)
    n = np.diff(off).max()
    eD = (grad(edY, ab(D), ab(hn) + eh, off)[1] + grad(ab(dYn), ab(D), eh, off)[1] +
          (n + 2) * S * grad(ab(dYn) + edY, ab(D), ab(hn) + eh, off)[1])
    assert (ab(_np(dwd) - dDn) <= eD + U * (ab(dDn) + eD)).all()
    dg, du = dhn * u * df, dhn * f
    edg = (ab(dhn) + edh) * (ab(u) * (0.8 * eg + 1.13 * own) + 1.13 * eu) * (1 + U) + edh * ab(u * df)
    edu = (ab(dhn) + edh) * (1.13 * eg + own * ab(f)) + edh * ab(f)
    edg, edu = edg + U * (ab(dg) + edg), edu + U * (ab(du) + edu)
    dXn, eX = np.zeros_like(X), np.zeros_like(X)
    for W, v, e, got in ((G, dg, edg, dwg), (V, du, edu, dwu)):
        a, b = grad(v, W, X, off)
        ea, eb = grad(e, ab(W), ab(X), off)
        sa, sb = grad(ab(v) + e, ab(W), ab(X), off)
        dXn, eX = dXn + a, eX + ea + (2 * I + 2) * S * sa
        eb = eb + (n + 2) * S * sb
        assert (ab(_np(got) - b) <= eb + U * (ab(b) + eb)).all()
    assert (_np(dwg)[-1] == 0).all()
    eX = eX + U * (ab(dXn) + eX)
    dxn, ex = orows.sort_rows_grad(dXn, row_of), orows.sort_rows_grad(eX, row_of)
    ex = ex + 6 * S * orows.sort_rows_grad(ab(dXn) + eX, row_of)
    assert (ab(_np(dx) - dxn) <= ex + U * (ab(dxn) + ex)).all()


def test_gradients_against_differences():
    """y is linear in x and in W: <dy, y(x + v) - y(x)> = <dx, v>, up to the
    rounding of both sides (y in fp32; v a change that x + v holds exactly)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    N, i, o = 60, 72, 40
    off = torch.tensor([0, 11, 11, 60], dtype=torch.int32, device="cuda")
    ints = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").to(BF16)
    x, w, dy, vx, vw = ints(N, i), ints(3, o, i), ints(N, o), ints(N, i), ints(3, o, i)
    f32 = lambda w_, x_: moe.moe_linear(w_, x_, off, out=torch.zeros(N, o, device="cuda")).double()
    dx, dw = moe.moe_linear_backward(dy, w, x, off, out=(torch.zeros_like(x), torch.zeros(3, o, i, device="cuda")))
    # whole numbers: sums below 2^24, so exact but for dx in bfloat16
    assert ((f32(w + vw, x) - f32(w, x)) * dy.double()).sum() == (dw.double() * vw.double()).sum()
    want = ((f32(w, x + vx) - f32(w, x)) * dy.double()).sum()
    assert (want - (dx.double() * vx.double()).sum()).abs() <= (U * (dx.double() * vx.double()).abs().sum())


def _calls(c):
    """Each entry point on c's tensors, writing to its buffers."""
    moe.moe_gated(c["wg"], c["wu"], c["x"], c["off"], save=True, out=(c["h"], c["pre"]))
    moe.moe_gated_backward(c["dh"], c["pre"], c["wg"], c["wu"], c["x"], c["off"], workspace=c["ws"],
                           out=(c["dx"], c["dwg"], c["dwu"]))
    moe.moe_linear(c["wg"], c["x"], c["off"], out=c["y"])
    moe.moe_linear_backward(c["dh"], c["wg"], c["x"], c["off"], out=(c["dx2"], c["dw"]))
    moe.moe_quantize_fp8(c["x"], out=(c["codes"], c["scales"]))
    moe.moe_linear_fp8(c["w8"], c["s8"], c["codes"], c["scales"], c["off"], out=c["y8"])


OUTS = ("h", "pre", "dx", "dwg", "dwu", "y", "dx2", "dw", "scales", "y8")


def _buffers(N, d, I, E, seed, ws=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    counts = torch.bincount(torch.randint(0, E, (N - 2,), generator=g, device="cuda"), minlength=E)
    c = dict(x=r(N, d), wg=r(E, I, d), wu=r(E, I, d), dh=r(N, I), off=torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int())
    c["w8"], c["s8"] = moe.moe_quantize_fp8(c["wg"], 128)
    e = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")
    c.update(h=e(N, I), pre=e(N, 2 * I, t=F32), dx=e(N, d), dwg=e(E, I, d), dwu=e(E, I, d), y=e(N, I), dx2=e(N, d), dw=e(E, I, d),
             codes=e(N, d, t=torch.float8_e4m3fn), scales=e(N, -(-d // 128), t=F32), y8=e(N, I))
    c["ws"] = torch.empty(moe.moe_gated_backward_workspace_bytes(N, I), dtype=torch.uint8, device="cuda") if ws is None else ws
    return c


SIZES = [(9, 512, 136, 16), (150, 144, 200, 3), (2200, 272, 392, 5)]


@pytest.mark.parametrize("N,d,I,E", SIZES)
def test_streams_and_graphs(N, d, I, E):
    c = _buffers(N, d, I, E, 0)
    _calls(c)
    torch.cuda.synchronize()
    want = {k: c[k].clone() for k in OUTS}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for k in OUTS:
            c[k].zero_()
        _calls(c)
    torch.cuda.current_stream().wait_stream(side)
    for k in OUTS:
        assert torch.equal(c[k], want[k]), k
    # stream=: allocated and launched there
    got = moe.moe_gated(c["wg"], c["wu"], c["x"], c["off"], stream=side)
    g8 = moe.moe_linear_fp8(c["w8"], c["s8"], c["codes"], c["scales"], c["off"], stream=side)
    side.synchronize()
    end = int(c["off"][-1])
    assert torch.equal(got[:end], want["h"][:end]) and torch.equal(g8[:end].to(BF16), want["y8"][:end])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _calls(c)
    for i in range(4):
        # other inputs, and the program's own work between the replays
        other = _buffers(N, d, I, E, 10 + i)
        _calls(other)
        torch.cuda.synchronize()
        for k in ("x", "wg", "wu", "dh", "off", "w8", "s8"):
            c[k].copy_(other[k])
        graph.replay()
        torch.cuda.synchronize()
        end = int(other["off"][-1])
        for k in OUTS:
            rows = slice(0, end) if c[k].shape[0] == N and k != "scales" else slice(None)
            assert torch.equal(c[k][rows], other[k][rows]), (i, k)


def test_two_graphs_that_share_a_workspace():
    N, d, I, E = 150, 144, 200, 3
    ws = torch.empty(moe.moe_gated_backward_workspace_bytes(N, I), dtype=torch.uint8, device="cuda")
    sets = []
    for seed in (0, 1):
        c = _buffers(N, d, I, E, seed, ws)
        _calls(c)
        torch.cuda.synchronize()
        want = {k: c[k].clone() for k in OUTS}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _calls(c)
        sets.append((c, want, graph))
    for _ in range(3):
        for c, want, graph in sets:
            for k in OUTS:
                c[k].zero_()
            graph.replay()
        torch.cuda.synchronize()
        for c, want, graph in sets:
            end = int(c["off"][-1])
            for k in OUTS:
                rows = slice(0, end) if c[k].shape[0] == N and k != "scales" else slice(None)
                assert torch.equal(c[k][rows], want[k][rows]), k


@pytest.mark.parametrize("d,I", [(72, 136), (71, 135)])
@pytest.mark.parametrize("N", [7, 200])
def test_borders_that_do_not_fit_the_rows(N, d, I):
    """Borders past the rows, falling or negative: no row outside x is read or
    written, and buckets inside it are right."""
    E = 6
    off = torch.tensor([-3, 2, 5, 4, N + 9, N + 100, N - 1], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(E, I, d, generator=g, device="cuda").to(BF16)
    guard = torch.full((N + 64, I), 5.0, dtype=BF16, device="cuda")
    x = torch.randn(N, d, generator=g, device="cuda").to(BF16)
    dy = torch.randn(N, I, generator=g, device="cuda").to(BF16)
    y = moe.moe_linear(w, x, off, out=guard[32:32 + N])
    moe.moe_gated(w, w, x, off, out=torch.zeros_like(y))
    dx, dw = moe.moe_linear_backward(dy, w, x, off)
    torch.cuda.synchronize()
    assert (guard[:32] == 5).all() and (guard[32 + N:] == 5).all()
    want = x[2:5].double() @ w[1].double().t()                        # the one whole bucket
    assert ((y[2:5].double() - want).abs()[:2] <= U * want.abs()[:2] + (d + 2) * S * (x[2:4].double().abs() @ w[1].double().abs().t())).all()
    assert torch.isfinite(dx).all() and (dw[2] == 0).all() and (dw[4] == 0).all()


def test_tensors_past_two_to_the_31():
    """Rows and matrices whose offsets pass 32 bits (5 GB and 4.3 GB), and codes past 2^31."""
    g = torch.Generator(device="cuda").manual_seed(0)
    N, d, o = 300000, 8192, 24
    x = torch.empty(N, d, dtype=BF16, device="cuda").uniform_(-1, 1, generator=g)
    w = (torch.randn(o, d, generator=g, device="cuda") / 90).to(BF16)
    dy = torch.randn(N, o, generator=g, device="cuda").to(BF16)
    y = moe.moe_linear(w, x)
    dx, dw = moe.moe_linear_backward(dy, w, x)
    rows = torch.tensor([0, 1, 131071, 262143, 262144, 262145, 299998, 299999], device="cuda")
    xr, dyr, W = x[rows].double(), dy[rows].double(), w.double()
    want = xr @ W.t()
    assert ((y[rows].double() - want).abs() <= U * want.abs() + (d + 2) * S * (xr.abs() @ W.abs().t())).all()
    want = dyr @ W
    assert ((dx[rows].double() - want).abs() <= U * want.abs() + (o + 2) * S * (dyr.abs() @ W.abs())).all()
    want, mag = torch.zeros(o, d, dtype=torch.float64, device="cuda"), torch.zeros(o, d, dtype=torch.float64, device="cuda")
    for a in range(0, N, 30000):
        p, q = dy[a:a + 30000].double(), x[a:a + 30000].double()
        want += p.t() @ q
        mag += p.abs().t() @ q.abs()
    assert ((dw.double() - want).abs() <= U * want.abs() + (N + 2) * S * mag).all()
    del dx
    codes, scales = moe.moe_quantize_fp8(x)
    c2, s2 = moe.moe_quantize_fp8(x[rows])
    assert torch.equal(codes.view(torch.uint8)[rows], c2.view(torch.uint8)) and torch.equal(scales[rows], s2)
    w8, ws8 = moe.moe_quantize_fp8(w, 128)
    y8 = moe.moe_linear_fp8(w8, ws8, codes, scales)
    near = moe.moe_linear_fp8(w8, ws8, c2, s2)
    # another form for few rows: the same codes, sums in another order (of 64 blocks, |x| <= 1)
    assert ((y8[rows] - near).double().abs() <= 2 * (7 * 2.0 ** -13 + 84 * S) * (xr.abs() * 1.07 + 0.01) @ (W.abs() * 1.07 + 0.01).t()).all()
    del x, codes, y, y8
    E, i, o = 1024, 2048, 1032
    w = torch.empty(E, o, i, dtype=BF16, device="cuda").uniform_(-1, 1, generator=g)
    x = torch.randn(8, i, generator=g, device="cuda").to(BF16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1001:], off[E:] = 3, 8                                         # 3 rows of expert 1000, 5 of the last
    y = moe.moe_linear(w, x, off)
    dx, dw = moe.moe_linear_backward(y, w, x, off)
    for e, a, b in ((1000, 0, 3), (1023, 3, 8)):
        want, mag = x[a:b].double() @ w[e].double().t(), x[a:b].double().abs() @ w[e].double().abs().t()
        assert ((y[a:b].double() - want).abs() <= U * want.abs() + (i + 2) * S * mag).all()
        want, mag = y[a:b].double().t() @ x[a:b].double(), y[a:b].double().abs().t() @ x[a:b].double().abs()
        assert ((dw[e].double() - want).abs() <= U * want.abs() + 7 * S * mag).all()
    assert (dw[:1000] == 0).all() and (dw[1001:1023] == 0).all()


def test_the_same_call_twice_gives_the_same_bits():
    c = _buffers(2200, 272, 392, 5, 3)
    _calls(c)
    first = {k: c[k].clone() for k in OUTS}
    for _ in range(3):
        _calls(c)
        for k in OUTS:
            assert torch.equal(c[k], first[k]), k


def test_serving_in_e4m3_after_training_in_16_bits():
    """The trained matrices quantised: y differs from the 16-bit layer's by what
    the codes' rounding (2^-4 relative, or 2^-10 of the block's largest) does."""
    rng, idx, idx_d, x, dy, w, wg, wu, wd = _layer(d=144, I=48)
    E = wg.shape[0]
    X, off, _, row_of = moe.moe_sort_tokens(x, idx_d, E)
    q = [moe.moe_quantize_fp8(m, 128) for m in (wg, wu, wd)]
    X8 = moe.moe_quantize_fp8(X)
    g, u = (moe.moe_linear_fp8(*q[i], *X8, off) for i in (0, 1))
    h = (torch.nn.functional.silu(g) * u).to(BF16)
    Y = moe.moe_linear_fp8(*q[2], *moe.moe_quantize_fp8(h), off, out=torch.zeros(X.shape, dtype=BF16, device="cuda"))
    y = moe.moe_unsort_combine(Y, row_of, w)
    y16 = _step(idx_d, x, dy, w, wg, wu, wd, E)[0]
    # three products, each operand off by 2^-4 at most: (1 + 2^-4)^2 - 1 of the magnitudes a product, here far above
    # the random walk of the roundings; what is checked is that the parts belong together
    Xn, offn = orows.sort_rows(_np(x), idx, E)[:2]
    G, V, D = (np.abs(_np(m)) for m in (wg, wu, wd))
    r = 2 * 2.0 ** -4 + 2.0 ** -8
    lin = oproducts.linear
    gn, un = lin(_np(wg), Xn, offn), lin(_np(wu), Xn, offn)
    eg, eu = r * lin(G, np.abs(Xn), offn), r * lin(V, np.abs(Xn), offn)
    hn = oproducts.act("silu", gn) * un
    eh = 1.13 * eg * (np.abs(un) + eu) + np.abs(oproducts.act("silu", gn)) * eu + 0.01 * np.abs(hn)
    eY = lin(D, eh, offn) + r * lin(D, np.abs(hn) + eh, offn)
    ro = orows.sort_rows(_np(x), idx, E)[3]
    assert (np.abs(_np(y) - _np(y16)) <= orows.unsort(1.1 * eY + 0.02, ro, _np(w))).all()
    assert torch.linalg.norm((y - y16).double()) < 0.2 * torch.linalg.norm(y16.double())


def test_refusals_on_the_device():
    r = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")
    x, w, off = r(6, 64), r(3, 16, 64), torch.zeros(4, dtype=torch.int32, device="cuda")
    dy, pre, ws = r(6, 16), r(6, 32, t=F32), torch.empty(4096, dtype=torch.uint8, device="cuda")
    x8, w8 = r(6, 64, t=torch.float8_e4m3fn), r(3, 16, 64, t=torch.float8_e4m3fn)
    sx, sw = r(6, 1, t=F32), r(3, 1, 1, t=F32)
    bad = [
        lambda: moe.moe_linear(w, x), lambda: moe.moe_linear(w[0], x, off), lambda: moe.moe_linear(w, x.half(), off),
        lambda: moe.moe_linear(w.float(), x.float(), off), lambda: moe.moe_linear(w, r(6, 72), off),
        lambda: moe.moe_linear(w, r(6, 128)[:, ::2], off), lambda: moe.moe_linear(w.transpose(1, 2), r(6, 16), off),
        lambda: moe.moe_linear(w[:1].expand(3, 16, 64), x, off), lambda: moe.moe_linear(w, x, off[:3]), lambda: moe.moe_linear(w, x, off.long()),
        lambda: moe.moe_linear(w, x, off.cpu()), lambda: moe.moe_linear(w.cpu(), x, off), lambda: moe.moe_linear(w, x, off, out=r(6, 17)),
        lambda: moe.moe_linear(w, x, off, out=r(6, 16, t=F16)), lambda: moe.moe_linear(w, x, off, out=r(6, 16).cpu()),
        lambda: moe.moe_linear_backward(dy, w, x, off, out=(None, None)), lambda: moe.moe_linear_backward(r(6, 15), w, x, off),
        lambda: moe.moe_linear_backward(dy, w, x, off, out=(r(6, 64), r(3, 16, 63))),
        lambda: moe.moe_linear_backward(dy, w, x, off, out=(r(6, 64), r(3, 16, 64, t=F16))),
        lambda: moe.moe_gated(w, w[:2], x, off), lambda: moe.moe_gated(w, r(3, 17, 64), x, off), lambda: moe.moe_gated(w, w.half(), x, off),
        lambda: moe.moe_gated(w, w, x, off, act="tanh"), lambda: moe.moe_gated(w, w, x, off, save=True, out=(dy, r(6, 32))),
        lambda: moe.moe_gated(w, w, x, off, save=True, out=(dy, r(6, 16, t=F32))),
        lambda: moe.moe_gated_backward(dy, pre.to(BF16), w, w, x, off), lambda: moe.moe_gated_backward(dy, pre, w, w, x, off, workspace=ws[1:]),
        lambda: moe.moe_gated_backward(dy, pre, w, w, x, off, workspace=ws[:64]),
        lambda: moe.moe_gated_backward(dy, pre, w, w, x, off, out=(r(6, 64), r(3, 16, 64), None)),
        lambda: moe.moe_gated_backward(dy, pre, w, w, x, off, out=(r(6, 64), r(3, 16, 64, t=F32), r(3, 16, 64))),
        lambda: moe.moe_quantize_fp8(x.double()), lambda: moe.moe_quantize_fp8(x.t()), lambda: moe.moe_quantize_fp8(x, 2),
        lambda: moe.moe_quantize_fp8(x, 128, out=(x8, sx)), lambda: moe.moe_quantize_fp8(x, out=(x8.view(torch.uint8), sx)),
        lambda: moe.moe_linear_fp8(w8, sw, x8, sx), lambda: moe.moe_linear_fp8(w8, sw[:2], x8, sx, off),
        lambda: moe.moe_linear_fp8(w8, sw, x8, r(6, 2, t=F32), off), lambda: moe.moe_linear_fp8(w8, sw, x, sx, off),
        lambda: moe.moe_linear_fp8(r(3, 16, 72, t=torch.float8_e4m3fn), sw, r(6, 72, t=torch.float8_e4m3fn), sx, off),
        lambda: moe.moe_linear_fp8(w8, None, x8, sx, off), lambda: moe.moe_linear_fp8(w8, sw, x8, sx, off, out=r(6, 16, t=torch.float64))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
            pytest.fail(f"call {i} was taken")
    for i in range(2):                                        # gradients that would be lost
        a = [w.clone(), x.clone()]
        a[i].requires_grad_()
        with pytest.raises(ValueError):
            moe.moe_linear(*a, off)
        with pytest.raises(ValueError):
            moe.moe_gated(a[0], a[0], a[1], off)
        with pytest.raises(ValueError):
            moe.moe_quantize_fp8(a[i])
        with torch.no_grad():
            moe.moe_linear(*a, off)
