"""Products of e4m3 codes whose two scales, multiplied with each other, leave
fp32's normal range while y does not; in every form that the sizes may take.

The bound is that of test_gpu_fp8.py, to which scaling a block's sum by one scale
and then by the other adds nothing: its (16 + B + 4) s counts two products of the
scales a block.  Most of the smallest y are normal numbers, 2^-126 and larger; a
rounding below that is 2^-150, and (16 + B + 4) s sum |x| |w| 2^-140 and larger."""
import numpy as np
import pytest

from test_gpu_fp8 import BF16, _check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

# streams of 16, 32 and 64 rows (few columns and many), tiles of 64 x 64, 128 x 128, 256 x 256; blocks that end early
DENSE = [(1, 400, 130), (20, 256, 300), (50, 272, 200), (20, 144, 8208), (50, 144, 8209), (1, 144, 16400), (130, 400, 200),
         (1000, 400, 4103), (600, 144, 13210)]
EXPERTS = [(10, 512, 200, 12), (300, 400, 130, 4), (2600, 144, 2056, 12), (2600, 144, 8200, 4)]


def _run(x, w, off, what):
    wc, ws = moe.moe_quantize_fp8(w, 128)
    xc, xs = moe.moe_quantize_fp8(x)
    y = moe.moe_linear_fp8(wc, ws, xc, xs, None if off is None else torch.from_numpy(off).cuda(),
                           out=torch.full((x.shape[0], w.shape[-2]), float("nan"), device="cuda"))
    _check(y, wc, ws, xc, xs, off, what)
    return y, ws, xs


def _inputs(N, n_in, n_out, E):
    g = torch.Generator(device="cuda").manual_seed(N)
    off = _borders(N, E) if E else None
    w = torch.randn(*((E,) if E else ()), n_out, n_in, generator=g, device="cuda")
    return torch.randn(N, n_in, generator=g, device="cuda"), w, off


def _borders(N, E):
    p = 1.0 / np.arange(1, E + 1) ** 0.7
    return np.concatenate([[0], np.cumsum(np.random.default_rng(N).multinomial(N, p / p.sum()))]).astype(np.int32)


@pytest.mark.parametrize("N,n_in,n_out,E", [(*s, 0) for s in DENSE] + EXPERTS)
def test_small_x_and_small_w(N, n_in, n_out, E):
    """Every step of the sums is such a one, with scales whose product has 4 bits
    left; then every other one, a sixteenth of those beside it; then those of some
    rows and columns only."""
    x, w, off = _inputs(N, n_in, n_out, E)
    y, ws, xs = _run((x * 2.0 ** -70).to(BF16), (w * 2.0 ** -58).to(BF16), off, "all")
    assert (xs.double().max() * ws.double().max() < 2.0 ** -138) and (y.abs() >= 2.0 ** -126).double().mean() > 0.5
    even = (torch.arange(n_in, device="cuda") // 128 % 2 == 0).float()
    _run((x * 2.0 ** -70).to(BF16), (w * 2.0 ** -43 * torch.exp2(4 * even)).to(BF16), off, "every other")
    some = (torch.arange(N, device="cuda") % 5 == 0).float().unsqueeze(1)
    cols = (torch.arange(n_out, device="cuda") // 128 % 2 == 0).float().unsqueeze(1)
    _run((x * torch.exp2(-70 * some)).to(BF16), (w * torch.exp2(-58 * cols)).to(BF16), off, "some")


@pytest.mark.parametrize("N,n_in,n_out,E", [(*s, 0) for s in DENSE] + EXPERTS)
def test_large_x_and_large_w_that_do_not_meet(N, n_in, n_out, E):
    """Scales whose product passes fp32's largest: sums of zeros stay zeros."""
    x, w, off = _inputs(N, n_in, n_out, E)
    odd = (torch.arange(n_in, device="cuda") % 2).float()
    y, ws, xs = _run((x * odd * 2.0 ** 95).to(BF16), (w * (1 - odd) * 2.0 ** 80).to(BF16), off, "large")
    assert xs.double().min() * ws.double().min() > 2.0 ** 128
    assert (y == 0).all()


@pytest.mark.parametrize("N,n_in,n_out,E", [(*s, 0) for s in DENSE] + EXPERTS)
def test_sizes_filled_up_with_zeros(N, n_in, n_out, E):
    """Blocks of zeros in x and in W: the smallest scales, no change to the sums."""
    x, w, off = _inputs(N, n_in, n_out, E)
    x, w = x.to(BF16), w.to(BF16)
    pad = lambda v: torch.nn.functional.pad(v, (0, -n_in % 128 + 256))
    y = _run(x, w, off, "plain")[0]
    z, ws, xs = _run(pad(x), pad(w), off, "filled")
    assert (xs[:, -1] == 2.0 ** -96 / 448).all() and torch.equal(y, z)


def test_a_scale_of_zero_and_one_that_is_not_finite():
    """Scales of the caller's own: zero gives zeros, one that is not finite spoils its own rows or columns."""
    for N, n_in, n_out in DENSE:
        x, w, _ = _inputs(N, n_in, n_out, 0)
        (wc, ws), (xc, xs) = moe.moe_quantize_fp8(w, 128), moe.moe_quantize_fp8(x)
        base = moe.moe_linear_fp8(wc, ws, xc, xs)
        xs[0] = 0.0
        assert (moe.moe_linear_fp8(wc, ws, xc, xs)[0] == 0).all()
        for v in (float("inf"), float("nan")):
            xs[0] = v
            y = moe.moe_linear_fp8(wc, ws, xc, xs)
            assert not torch.isfinite(y[0]).any() and torch.equal(y[1:], base[1:])
        xs[0] = 1.0
        base = moe.moe_linear_fp8(wc, ws, xc, xs)
        ws[-1] = float("inf")
        y = moe.moe_linear_fp8(wc, ws, xc, xs)
        first = (n_out - 1) // 128 * 128
        assert not torch.isfinite(y[:, first:]).any() and torch.equal(y[:, :first], base[:, :first])


@pytest.mark.parametrize("v", [float("inf"), float("nan")])
def test_a_scale_that_is_not_finite_beside_zeros(v):
    """A scale of x that is not finite where W is zeros, and the other way round: inf times 0 is no number."""
    for N, n_in, n_out in DENSE:
        x, w, _ = _inputs(N, n_in, n_out, 0)
        w[:, :128] = 0
        (wc, ws), (xc, xs) = moe.moe_quantize_fp8(w, 128), moe.moe_quantize_fp8(x)
        base = moe.moe_linear_fp8(wc, ws, xc, xs)
        xs[0, 0] = v
        y = moe.moe_linear_fp8(wc, ws, xc, xs)
        assert torch.isnan(y[0]).all() and torch.equal(y[1:], base[1:]), (N, n_in, n_out)
        x[:, :128], w[:, :128] = 0, 1
        (wc, ws), (xc, xs) = moe.moe_quantize_fp8(w, 128), moe.moe_quantize_fp8(x)
        ws[0, 0] = v
        y = moe.moe_linear_fp8(wc, ws, xc, xs)
        assert torch.isnan(y[:, :128]).all() and torch.isfinite(y[:, 128:]).all(), (N, n_in, n_out)
