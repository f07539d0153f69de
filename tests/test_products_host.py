"""The experts' products without a GPU: the oracle's gradients against central
differences of its own forward, its e4m3 numbers against torch's, workspace
sizes, and the refusal of bad calls before any device work."""
import numpy as np
import pytest

import sparse_moe_decode_router_amd as moe
from oracle import products as oproducts

LIB = moe._lib
BAD, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK
BF16, F16, F32 = moe.MOE_TYPE_BF16, moe.MOE_TYPE_F16, moe.MOE_TYPE_F32
P = 4096          # a stand-in address: no call below reaches a kernel
WS = 1 << 30


def _differences(f, a, h=1e-5):
    g = np.zeros_like(a)
    for j in np.ndindex(a.shape):
        up, dn = a.copy(), a.copy()
        up[j] += h
        dn[j] -= h
        g[j] = (f(up) - f(dn)) / (2 * h)
    return g


OFF = np.array([0, 2, 2, 5])


@pytest.mark.parametrize("act", oproducts.ACTS)
def test_oracle_gated_gradients_against_differences(act):
    """h^2 times third derivatives of order ten, and rounding of 1e-15 / 1e-5."""
    rng = np.random.default_rng(3)
    x, dh = rng.standard_normal((6, 4)), rng.standard_normal((6, 3))
    Wg, Wu = rng.standard_normal((3, 3, 4)), rng.standard_normal((3, 3, 4))
    loss = lambda x_, g_, u_: np.sum(dh * oproducts.gated(g_, u_, x_, OFF, act)[0])
    dx, dg, du = oproducts.gated_grad(dh, Wg, Wu, x, OFF, act)
    assert np.allclose(_differences(lambda a: loss(a, Wg, Wu), x), dx, atol=1e-7)
    assert np.allclose(_differences(lambda a: loss(x, a, Wu), Wg), dg, atol=1e-7)
    assert np.allclose(_differences(lambda a: loss(x, Wg, a), Wu), du, atol=1e-7)
    assert (dx[5] == 0).all() and (dg[1] == 0).all()          # behind the last bucket; an expert without rows


def test_oracle_linear_gradients_against_differences():
    rng = np.random.default_rng(4)
    x, dy, W = rng.standard_normal((6, 4)), rng.standard_normal((6, 3)), rng.standard_normal((3, 3, 4))
    dx, dW = oproducts.linear_grad(dy, W, x, OFF)
    assert np.allclose(_differences(lambda a: np.sum(dy * oproducts.linear(W, a, OFF)), x), dx, atol=1e-8)
    assert np.allclose(_differences(lambda a: np.sum(dy * oproducts.linear(a, x, OFF)), W), dW, atol=1e-8)


def test_oracle_activations_against_torch():
    torch = pytest.importorskip("torch")
    f = torch.nn.functional
    g = torch.linspace(-9, 9, 401, dtype=torch.float64, requires_grad=True)
    for name, fn in [("silu", f.silu), ("gelu", f.gelu), ("gelu_tanh", lambda v: f.gelu(v, approximate="tanh"))]:
        y = fn(g)
        (d,) = torch.autograd.grad(y.sum(), g)
        assert np.allclose(oproducts.act(name, g.detach().numpy()), y.detach().numpy(), rtol=0, atol=1e-14)
        assert np.allclose(oproducts.act_slope(name, g.detach().numpy()), d.numpy(), rtol=0, atol=1e-14)


def test_slopes_are_within_the_bounds_that_the_gpu_tolerances_take():
    g = np.linspace(-30, 30, 60001)
    for name in oproducts.ACTS:
        d = oproducts.act_slope(name, g)
        assert np.abs(d).max() < 1.13 and np.abs(np.diff(d) / np.diff(g)).max() < 0.8


def test_oracle_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    byte = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    t = torch.from_numpy(byte).view(torch.float8_e4m3fn)
    assert np.array_equal(oproducts.e4m3_values(byte), t.double().numpy())
    v = np.random.default_rng(0).uniform(-448, 448, 20000) * np.exp2(-np.random.default_rng(1).integers(0, 18, 20000))
    v = np.concatenate([v, oproducts.E4M3, (oproducts.E4M3[1:] + oproducts.E4M3[:-1]) / 2])
    v = v.astype(np.float32)
    assert np.array_equal(oproducts.e4m3_codes(v), torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_quantization():
    """What a code stands for is within half a step of the value."""
    x = np.random.default_rng(5).standard_normal((130, 300))
    for br in (1, 128):
        c, s = oproducts.quantize_fp8(x, br)
        assert s.shape == (-(-130 // br), 3)
        up = np.repeat(np.repeat(s, br, 0)[:130], 128, 1)[:, :300]
        assert (np.abs(oproducts.e4m3_values(c) * up - x) <= np.maximum(np.abs(x) * 2.0 ** -4, up * 2.0 ** -10) * (1 + 1e-12)).all()
    z, s = oproducts.quantize_fp8(np.zeros((2, 5)), 1)
    assert (z == 0).all() and (s == 2.0 ** -96 / 448).all()


# ----------------------------------------------------------------- refusals
COMMON = [dict(E=0), dict(E=1025), dict(ty=F32), dict(ty=3), dict(N=-1), dict(i=0), dict(o=0), dict(off=None), dict(off=P + 2)]
TOO_LARGE = [dict(i=(1 << 20) + 1, st=1 << 40), dict(o=(1 << 20) + 1, st=1 << 40), dict(N=(1 << 30) + 1)]


def test_linear_refusals():
    def lin(w=P, st=8192, E=4, x=P, ty=BF16, N=3, i=64, o=32, off=P, y=P, yt=None):
        return LIB.moe_linear(w, st, E, x, ty, N, i, o, off, y, ty if yt is None else yt, None)

    def grad(dy=P, w=P, st=8192, E=4, x=P, ty=BF16, N=3, i=64, o=32, off=P, dx=P, dw=P, dst=1 << 41, dt=None):
        return LIB.moe_linear_backward(dy, w, st, E, x, ty, N, i, o, off, dx, dw, dst, ty if dt is None else dt, None)
    for f in (lin, grad):
        for kw in COMMON:
            assert f(**kw) == BAD, (f, kw)
        for kw in TOO_LARGE:
            assert f(**kw) == UNS, (f, kw)
        for kw in [dict(w=None), dict(x=None), dict(w=P + 1), dict(x=P + 1), dict(st=4094), dict(st=8191)]:
            assert f(**kw) == BAD, (f, kw)
    assert lin(N=0, w=None, x=None, y=None) == OK
    for kw in [dict(y=None), dict(y=P + 1), dict(yt=F16), dict(yt=F32, y=P + 2), dict(yt=7)]:
        assert lin(**kw) == BAD, kw
    for kw in [dict(dy=None), dict(dy=P + 1), dict(dx=None, dw=None), dict(dx=P + 1), dict(dw=P + 1), dict(dt=F16),
               dict(dt=F32, dw=P + 2), dict(dst=4094), dict(dst=4097)]:
        assert grad(**kw) == BAD, kw


def test_gated_refusals():
    def fwd(g=P, gs=8192, u=P, us=8192, E=4, x=P, ty=BF16, N=3, i=64, o=32, off=P, act=0, h=P, pre=None, st=None):
        return LIB.moe_gated(g, st or gs, u, st or us, E, x, ty, N, i, o, off, act, h, pre, None)

    def bwd(dh=P, pre=P, g=P, gs=8192, u=P, us=8192, E=4, x=P, ty=BF16, N=3, i=64, o=32, off=P, act=0, dx=P, dg=P, dgs=1 << 41,
            du=P, dus=1 << 41, dt=None, ws=P, n=1 << 60, st=None):
        return LIB.moe_gated_backward(dh, pre, g, st or gs, u, st or us, E, x, ty, N, i, o, off, act, dx, dg, dgs, du, dus,
                                      ty if dt is None else dt, ws, n, None)
    for f in (fwd, bwd):
        for kw in COMMON:
            assert f(**kw) == BAD, (f, kw)
        for kw in TOO_LARGE:
            assert f(**kw) == UNS, (f, kw)
        for kw in [dict(g=None), dict(u=None), dict(x=None), dict(g=P + 1), dict(u=P + 1), dict(x=P + 1), dict(gs=4094),
                   dict(us=4094), dict(us=8193), dict(act=-1), dict(act=3)]:
            assert f(**kw) == BAD, (f, kw)
    assert fwd(N=0, g=None, u=None, x=None, h=None) == OK
    for kw in [dict(h=None), dict(h=P + 1), dict(pre=P + 2)]:
        assert fwd(**kw) == BAD, kw
    for kw in [dict(dh=None), dict(pre=None), dict(ws=None), dict(ws=P + 8), dict(n=3 * 32 * 4), dict(dx=None, dg=None, du=None),
               dict(dg=None), dict(du=None), dict(dx=P + 1), dict(dg=P + 1), dict(dt=F16), dict(dt=F32, du=P + 2),
               dict(dgs=4094), dict(dus=4094)]:
        assert bwd(**kw) == BAD, kw
    f = moe.moe_gated_backward_workspace_bytes
    assert f(3, 32) >= 3 * 32 * 4 and f(0, 32) > 0
    for a in [(-1, 32), (3, 0), ((1 << 30) + 1, 32), (3, (1 << 20) + 1), (3 + (1 << 32), 32), (3, 32 - (1 << 32))]:
        assert f(*a) == 0, a


def test_fp8_refusals():
    def q(x=P, ty=BF16, c=1, r=4, n=64, br=1, codes=P, s=P):
        return LIB.moe_quantize_fp8(x, ty, c, r, n, br, codes, s, None)

    def lin(w=P, st=8192, ws=P, wss=64, E=4, x=P, xs=P, N=3, i=64, o=32, off=P, y=P, yt=F32):
        return LIB.moe_linear_fp8(w, st, ws, wss, E, x, xs, N, i, o, off, y, yt, None)
    assert q(r=0, x=None, codes=None, s=None) == OK and q(c=0) == OK and lin(N=0, x=None, xs=None, y=None) == OK
    for kw in [dict(x=None), dict(codes=None), dict(s=None), dict(ty=3), dict(ty=-1), dict(c=-1), dict(r=-1), dict(n=0),
               dict(br=0), dict(br=64), dict(x=P + 1), dict(ty=F32, x=P + 2), dict(s=P + 2)]:
        assert q(**kw) == BAD, kw
    assert q(n=(1 << 20) + 1) == UNS and q(c=1 << 16, r=1 << 16) == UNS
    for kw in [dict(w=None), dict(ws=None), dict(x=None), dict(xs=None), dict(y=None), dict(yt=3), dict(i=72), dict(i=8),
               dict(w=P + 8), dict(x=P + 8), dict(st=2056), dict(st=1024), dict(wss=0), dict(xs=P + 2), dict(ws=P + 1),
               dict(y=P + 2), dict(E=0), dict(E=1025), dict(N=-1), dict(o=0), dict(off=None), dict(off=P + 1)]:
        assert lin(**kw) == BAD, kw
    for kw in [dict(i=1 << 21, st=1 << 40), dict(o=(1 << 20) + 1, st=1 << 40), dict(N=(1 << 30) + 1)]:
        assert lin(**kw) == UNS, kw


def test_host_tensors_and_wrong_arguments_are_refused():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 64, dtype=torch.float8_e4m3fn), torch.zeros(2, 1)
    dy = torch.zeros(2, 8, dtype=torch.bfloat16)
    pre = torch.zeros(2, 16)
    for call in [lambda: moe.moe_linear(w, x), lambda: moe.moe_linear_backward(dy, w, x), lambda: moe.moe_gated(w, w, x),
                 lambda: moe.moe_gated_backward(dy, pre, w, w, x), lambda: moe.moe_quantize_fp8(x),
                 lambda: moe.moe_linear_fp8(c, s[:1], c, s), lambda: moe.moe_linear(w, x[0]), lambda: moe.moe_linear(w[0], x),
                 lambda: moe.moe_linear(w, x, torch.zeros(2, dtype=torch.int32)), lambda: moe.moe_quantize_fp8(x, 64),
                 lambda: moe.moe_quantize_fp8(x[0]), lambda: moe.moe_gated(w, w, x, act="relu"),
                 lambda: moe.moe_gated(w, w, x, act=0), lambda: moe.moe_gated(w, w, x, save=True, out=(x, None))]:
        with pytest.raises(ValueError):
            call()
