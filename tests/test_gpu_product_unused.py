"""The backward calls without the operands that they do not use: no w where no dx
is wanted, no x where no gradient of a matrix is."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

BF16, F32 = torch.bfloat16, torch.float32


def _inputs(E, N=50, d=72, I=40):
    g = torch.Generator(device="cuda").manual_seed(E)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    lead = (E,) if E else ()
    off = torch.tensor([0, 11, 11, 30, N - 3], dtype=torch.int32, device="cuda") if E else None
    return r(*lead, I, d), r(*lead, I, d), r(N, d), r(N, I), off


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("E", [0, 4])
def test_operands_that_are_not_used(E, t):
    wg, wu, x, dy, off = _inputs(E)
    zeros = lambda v: torch.zeros(v.shape, dtype=t, device="cuda")
    dx, dw = moe.moe_linear_backward(dy, wg, x, off, out=(torch.zeros_like(x), zeros(wg)))
    assert torch.equal(moe.moe_linear_backward(dy, wg, None, off, out=(torch.zeros_like(x), None))[0], dx)
    assert torch.equal(moe.moe_linear_backward(dy, None, x, off, out=(None, zeros(wg)))[1], dw)
    h, pre = moe.moe_gated(wg, wu, x, off, save=True)
    dx, dg, du = moe.moe_gated_backward(dy, pre, wg, wu, x, off, out=(torch.zeros_like(x), zeros(wg), zeros(wu)))
    assert torch.equal(moe.moe_gated_backward(dy, pre, wg, wu, None, off, out=(torch.zeros_like(x), None, None))[0], dx)
    got = moe.moe_gated_backward(dy, pre, None, None, x, off, out=(None, zeros(wg), zeros(wu)))
    assert torch.equal(got[1], dg) and torch.equal(got[2], du)


@pytest.mark.parametrize("E", [0, 4])
def test_operands_that_are_used(E):
    wg, wu, x, dy, off = _inputs(E)
    _, pre = moe.moe_gated(wg, wu, x, off, save=True)
    z = torch.zeros_like
    lin, gat = moe.moe_linear_backward, moe.moe_gated_backward
    bad = [lambda: lin(dy, None, x, off), lambda: lin(dy, wg, None, off), lambda: lin(dy, None, x, off, out=(z(x), None)),
           lambda: lin(dy, None, x, off, out=(z(x), z(wg))), lambda: lin(dy, wg, None, off, out=(None, z(wg))),
           lambda: lin(dy, None, None, off, out=(None, z(wg))), lambda: lin(dy, None, x, off, out=(None, None)),
           lambda: lin(dy, None, x, off, out=(None, z(wg)[..., :-8])), lambda: lin(dy, wg, x[:, :-8], off, out=(z(x), None)),
           lambda: gat(dy, pre, None, wu, x, off), lambda: gat(dy, pre, wg, None, x, off, out=(z(x), None, None)),
           lambda: gat(dy, pre, None, None, x, off, out=(z(x), z(wg), z(wu))), lambda: gat(dy, pre, wg, wu, None, off),
           lambda: gat(dy, pre, None, None, None, off, out=(None, z(wg), z(wu))),
           lambda: gat(dy, pre, None, None, x, off, out=(None, None, None)),
           lambda: gat(dy, pre, None, wu[..., :-8], x, off, out=(None, z(wg), z(wu))),
           lambda: gat(dy, pre, None, None, x, off, out=(None, z(wg), None)),
           lambda: gat(dy, pre, None, None, x, off, out=(None, None, z(wu)))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
            pytest.fail(f"call {i} was taken")
