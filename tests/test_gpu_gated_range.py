"""The gated block's gradients at the ends of fp16: dg and du are rounded to it.

Up to 65504 and down to its subnormals they keep the bounds of
test_gpu_products.py (a rounding to fp16 is off by 2^-25 at most where 2^-11
relative is less); 65520 and more is infinite, 2^-25 and less zero."""
import numpy as np
import pytest

from test_gpu_products import BF16, F16, F32, Case, _run_gated, _run_linear, oproducts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

# streams and tiles of 64 x 64 and 128 x 128 (dW in half steps), whole pieces and not
SIZES = [(60, 72, 40, 0), (61, 71, 41, 4), (300, 264, 520, 12), (200, 2047, 1025, 0)]


@pytest.mark.parametrize("act", oproducts.ACTS)
@pytest.mark.parametrize("N,d,I,E", SIZES)
def test_small_gradients(N, d, I, E, act):
    """dh in the subnormals, around 2^-18."""
    c = Case(F16, N, d, I, E, 0, mats=2)
    c.dy = (c.dy.float() * 2.0 ** -18).to(F16)
    assert (c.dy.abs() < 2.0 ** -14).all() and (c.dy != 0).double().mean() > 0.9
    _run_gated(c, d, I, act)
    _run_gated(c, d, I, act, F32)
    c.w = c.w[:1]
    _run_linear(c, d, I)


@pytest.mark.parametrize("N,d,I,E", SIZES[:3])
def test_large_gradients(N, d, I, E):
    """dg and du up to the largest fp16.  x is 8 times and W an eighth of the
    others' size, so that g and u are of order one and dx fits where dg nearly does not."""
    c = Case(F16, N, d, I, E, 0, mats=2)
    c.x, c.w = (c.x.float() * 8).to(F16), [(w.float() / 8).to(F16) for w in c.w]
    top = 0.0
    for e, a, b, (G, U) in c.buckets():
        x, dh = c.x[a:b].double(), c.dy[a:b].double()
        g, u = x @ G.t(), x @ U.t()
        df = torch.from_numpy(oproducts.act_slope("silu", g.cpu().numpy())).cuda()
        f = torch.from_numpy(oproducts.act("silu", g.cpu().numpy())).cuda()
        if b > a:
            top = max(top, (dh * u * df).abs().max().item(), (dh * f).abs().max().item())
    c.dy = (c.dy.double() * (65000 / top)).to(F16)               # (rounded: 2^-11 of 65000 is 32)
    _run_gated(c, d, I, "silu", F32)


@pytest.mark.parametrize("d,I", [(72, 40), (71, 41)])
def test_past_the_ends(d, I):
    """g 0 and u 2 (gelu: act'(0) = 1/2, act(0) = 0), so that dg = dh and du = 0 exactly."""
    N, E = 40, 2
    off = torch.tensor([0, 25, N], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(F16)
    wg, wu, x = r(E, I, d), r(E, I, d), r(N, d)
    pre = torch.cat([torch.zeros(N, I, device="cuda"), torch.full((N, I), 2.0, device="cuda")], 1)

    def run(dh):
        dx, dwg, dwu = moe.moe_gated_backward(dh, pre, wg, wu, x, off, act="gelu",
                                              out=(torch.zeros_like(x), *(torch.zeros(E, I, d, device="cuda") for _ in "gu")))
        assert (dwu == 0).all()
        return dx, dwg
    dh = r(N, I)
    base = run(dh)
    dh[7, 5] = 0
    none = run(dh)
    pre[7, I + 5] = 2.0 ** -25                                   # dg = dh 2^-26
    for v, zero in ((1.0, True), (2.0, True), (3.0, False)):     # 2^-26, 2^-25 and 1.5 2^-25: the last goes up to 2^-24
        dh[7, 5] = v
        got = run(dh)
        assert torch.equal(got[1], none[1]) == zero, v
    pre[7, I + 5] = 4.0                                          # dg = 2 dh
    dh[7, 5] = 32752.0                                           # 65504
    dx, dwg = run(dh)
    assert torch.isfinite(dwg).all() and torch.isfinite(dx[:7]).all()
    assert torch.equal(dwg[0, 5] != none[1][0, 5], x[7] != 0)
    dh[7, 5] = 32768.0                                           # 65536
    dx, dwg = run(dh)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[7] = False
    assert not torch.isfinite(dx[7]).any() and torch.equal(dx[keep], base[0][keep])
    rows = torch.ones(E, I, dtype=torch.bool, device="cuda")
    rows[0, 5] = False
    assert not torch.isfinite(dwg[0, 5]).any() and torch.equal(dwg[rows], base[1][rows])
