"""Products of 16-bit matrices and the gated block on the GPU against fp64.

Tolerances, derived.  u = eps / 2 of the type is what one rounding changes of a
value (and 2^-25 at most of a subnormal fp16); s = 2^-23 bounds what one fp32
addition does to the partial sum (half of that for an adder that rounds to
nearest), and products of two 16-bit values are exact.

  sums      |y - y*| <= u |y*| + (K + 2) s sum |x| |w|, K the products of a sum
  gated     g and u' as sums without the rounding.  The slope of each activation
            lies within 1.13 and its own slope within 0.8; the activation itself
            is off by at most (g^2 + |g| + 8) 2 s of its value (its argument's
            rounding moves erfc by up to g^2 s, exp by |g| s, and a few ulp each
            of exp, reciprocal and product), so
            dh = 1.13 dg |u'| + |act| du' + 1.13 dg du' + (..) |h| + u |h|
  backward  with dg and du' as above (g and u' are saved in fp32),
            of dg' = dh u' act'(g): |dh| (|u'| (0.8 dg + (..) 1.13) + 1.13 du') (1 + u) + u |dg'|,
            of du'' = dh act(g): |dh| (1.13 dg + (..) |act|) + u |du''|;
            then dx, dW as sums of operands that are off by those.
"""
import math

import numpy as np
import pytest

from oracle import products as oproducts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
S = 2.0 ** -23


def _u(t):
    return torch.finfo(t).eps / 2 if t != F32 else 2.0 ** -24


def _floor(t):
    return 2.0 ** -25 if t == F16 else 0.0


def _offsets(rng, E, N, behind):
    """Borders of E buckets over N - behind rows: some empty, one long."""
    p = rng.permutation(1.0 / np.arange(1, E + 1) ** 1.2)
    counts = rng.multinomial(N - behind, p / p.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _buckets(off, N):
    return [(0, 0, N)] if off is None else [(e, int(off[e]), int(off[e + 1])) for e in range(len(off) - 1)]


def _check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError((what, i, int(bad.sum()), bad.numel(), got[tuple(i)].item(), want[tuple(i)].item(),
                              tol[tuple(i)].item()))


def _sum_tol(t, K, want, mag):
    return _u(t) * want.abs() + (K + 2) * S * mag + _floor(t)


class Case:
    def __init__(self, t, N, n_in, n_out, E=0, behind=0, seed=0, mats=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng([N, n_in, n_out, E])
        self.off = None if E == 0 else _offsets(rng, E, N, behind)
        self.offsets = None if E == 0 else torch.from_numpy(self.off).cuda()
        lead = (E,) if E else ()
        self.w = [(torch.randn(*lead, n_out, n_in, generator=g, device="cuda") / math.sqrt(n_in)).to(t) for _ in range(mats)]
        self.x = torch.randn(N, n_in, generator=g, device="cuda").to(t)
        self.dy = torch.randn(N, n_out, generator=g, device="cuda").to(t)
        self.N, self.t = N, t
        if E:
            end = int(self.off[-1])                  # rows behind the last bucket are not to be used
            self.x[end:], self.dy[end:] = float("nan"), float("nan")

    def buckets(self):
        for e, a, b in _buckets(self.off, self.N):
            yield e, a, b, [w[e].double() if self.off is not None else w.double() for w in self.w]


def _nan(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


# sizes: whole pieces and not, one and many chunks and tiles, tails of k in every place
DENSE = [(1, 8, 8), (1, 1, 1), (3, 7, 5), (1, 2048, 512), (2, 64, 128), (5, 72, 200), (16, 512, 96), (17, 100, 33),
         (33, 1001, 129), (64, 256, 256), (65, 192, 130), (127, 136, 1000), (128, 128, 128), (129, 63, 257), (200, 65, 64),
         (300, 1032, 520), (513, 320, 77), (1000, 31, 40), (257, 2056, 264)]
EXPERTS = [(1, 64, 64, 1, 0), (10, 512, 2048, 64, 0), (10, 2048, 512, 512, 1), (7, 24, 40, 3, 2), (40, 129, 65, 9, 3),
           (96, 256, 136, 8, 11), (300, 72, 88, 5, 0), (700, 200, 264, 3, 77), (640, 33, 100, 64, 5), (1500, 64, 72, 1024, 100),
           (2100, 136, 392, 12, 0), (129, 1000, 56, 2, 1)]


def _run_linear(c, n_in, n_out, out_type=None, what=""):
    w, ty = c.w[0], out_type or c.t
    y = moe.moe_linear(w, c.x, c.offsets, out=_nan(c.N, n_out, dtype=ty))
    dx, dw = moe.moe_linear_backward(c.dy, w, c.x, c.offsets,
                                     out=(_nan(c.N, n_in, dtype=c.t), _nan(*w.shape, dtype=ty)))
    end = c.N
    for e, a, b, (W,) in c.buckets():
        x, dy = c.x[a:b].double(), c.dy[a:b].double()
        _check(y[a:b], x @ W.t(), _sum_tol(ty, n_in, x @ W.t(), x.abs() @ W.abs().t()), (what, "y", e, a, b))
        _check(dx[a:b], dy @ W, _sum_tol(c.t, n_out, dy @ W, dy.abs() @ W.abs()), (what, "dx", e, a, b))
        d = dw[e] if c.off is not None else dw
        _check(d, dy.t() @ x, _sum_tol(ty, b - a, dy.t() @ x, dy.abs().t() @ x.abs()), (what, "dw", e, a, b))
        end = b
    assert torch.isnan(y[end:]).all() and torch.isnan(dx[end:]).all()
    return y, dx, dw


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("N,n_in,n_out", DENSE)
def test_linear_dense(t, N, n_in, n_out):
    c = Case(t, N, n_in, n_out)
    _run_linear(c, n_in, n_out)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("N,n_in,n_out,E,behind", EXPERTS)
def test_linear_experts(t, N, n_in, n_out, E, behind):
    c = Case(t, N, n_in, n_out, E, behind)
    _run_linear(c, n_in, n_out)


# Sizes by the form that they take: tiles of 256 x 256 (long buckets and more
# than two rounds of smaller ones), of 128 x 128 past 256 of them, with rows that
# end in every tile of a wave, whole pieces or not.
@pytest.mark.parametrize("N,n_in,n_out,E", [
    (600, 72, 13208, 0), (520, 13208, 72, 0), (770, 136, 13320, 0), (70, 13208, 1000, 0),      # 256 x 256: y, dx, y, dw
    (3000, 40, 8200, 4), (2700, 8200, 40, 4), (90, 2056, 1032, 12),                          # and for experts
    (1100, 1000, 4104, 0), (1000, 201, 4103, 0), (5000, 264, 520, 40), (5000, 265, 521, 40), (300, 521, 263, 100),
    (700, 2048, 512, 512), (700, 331, 515, 512)])
def test_linear_forms(N, n_in, n_out, E):
    _run_linear(Case(BF16 if N % 3 else F16, N, n_in, n_out, E, N // 50 if E else 0), n_in, n_out)


@pytest.mark.parametrize("N,d,I,E", [(600, 72, 6608, 0), (530, 6608, 264, 0), (2600, 72, 4104, 4), (1030, 520, 2056, 0),
                                     (1000, 201, 2055, 0), (5000, 136, 264, 40), (5000, 137, 263, 40), (600, 1024, 136, 300)])
def test_gated_forms(N, d, I, E):
    _run_gated(Case(BF16 if N % 3 else F16, N, d, I, E, N // 50 if E else 0, mats=2), d, I, oproducts.ACTS[d % 3])


@pytest.mark.parametrize("E,first,N", [(64, 63, 500), (64, 0, 500), (300, 150, 2000), (4, 2, 700)])
@pytest.mark.parametrize("i,o", [(136, 200), (131, 203)])
def test_all_rows_of_one_expert(E, first, N, i, o):
    """Few rows a bucket on average, all of them in one."""
    c = Case(BF16, N, i, o, E, 0, mats=2)
    c.off = np.where(np.arange(E + 1) > first, N, 0).astype(np.int32)
    c.offsets = torch.from_numpy(c.off).cuda()
    c.x, c.dy = (torch.randn(N, w, device="cuda").to(BF16) for w in (i, o))
    _run_gated(c, i, o, "silu")
    c.w = c.w[:1]
    _run_linear(c, i, o)


@pytest.mark.parametrize("N,n_in,n_out,E", [(70, 136, 200, 0), (70, 35, 201, 0), (90, 72, 264, 4), (3, 512, 65, 2)])
def test_linear_fp32_outputs(N, n_in, n_out, E):
    _run_linear(Case(BF16, N, n_in, n_out, E), n_in, n_out, F32)
    _run_linear(Case(F16, N, n_in, n_out, E), n_in, n_out, F32)


def _run_gated(c, d, I, act, grad_type=None, what=""):
    wg, wu = c.w
    t, td = c.t, grad_type or c.t
    u_, fl = _u(t), _floor(t)
    only = moe.moe_gated(wg, wu, c.x, c.offsets, act=act, out=_nan(c.N, I, dtype=t))
    h, pre = moe.moe_gated(wg, wu, c.x, c.offsets, act=act, save=True, out=(_nan(c.N, I, dtype=t), _nan(c.N, 2 * I, dtype=F32)))
    assert torch.equal(torch.nan_to_num(h), torch.nan_to_num(only))
    dx, dwg, dwu = moe.moe_gated_backward(c.dy, pre, wg, wu, c.x, c.offsets, act=act,
                                          out=(_nan(c.N, d, dtype=t), _nan(*wg.shape, dtype=td), _nan(*wu.shape, dtype=td)))
    end = c.N
    for e, a, b, (G, U) in c.buckets():
        x, dh = c.x[a:b].double(), c.dy[a:b].double()
        g, u = x @ G.t(), x @ U.t()
        eg, eu = (d + 2) * S * (x.abs() @ G.abs().t()), (d + 2) * S * (x.abs() @ U.abs().t())
        f = torch.from_numpy(oproducts.act(act, g.cpu().numpy())).cuda()
        df = torch.from_numpy(oproducts.act_slope(act, g.cpu().numpy())).cuda()
        own = (g * g + g.abs() + 8) * 2 * S
        want = f * u
        _check(h[a:b], want, 1.13 * eg * u.abs() + f.abs() * eu + 1.13 * eg * eu + own * want.abs() + u_ * want.abs() + fl,
               (what, "h", e, a, b))
        _check(pre[a:b, :I], g, eg, (what, "g", e, a, b))
        _check(pre[a:b, I:], u, eu, (what, "u", e, a, b))
        dg, du = dh * u * df, dh * f
        edg = dh.abs() * (u.abs() * (0.8 * eg + 1.13 * own) + 1.13 * eu) * (1 + u_) + u_ * dg.abs() + fl
        edu = dh.abs() * (1.13 * eg + own * f.abs()) + u_ * du.abs() + fl
        want = dg @ G + du @ U
        mag = (dg.abs() + edg) @ G.abs() + (du.abs() + edu) @ U.abs()
        _check(dx[a:b], want, _sum_tol(t, 2 * I, want, mag) + edg @ G.abs() + edu @ U.abs(), (what, "dx", e, a, b))
        for name, got, v, ev in (("dw_gate", dwg, dg, edg), ("dw_up", dwu, du, edu)):
            want = v.t() @ x
            _check(got[e] if c.off is not None else got, want,
                   _sum_tol(td, b - a, want, (v.abs() + ev).t() @ x.abs()) + ev.t() @ x.abs(), (what, name, e, a, b))
        end = b
    for v in (h, pre, dx):
        assert torch.isnan(v[end:]).all()


@pytest.mark.parametrize("act", oproducts.ACTS)
@pytest.mark.parametrize("N,d,I", [s for s in DENSE if s[0] < 600])
def test_gated_dense(N, d, I, act):
    t = BF16 if (N + d) % 2 else F16
    _run_gated(Case(t, N, d, I, mats=2), d, I, act)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("N,d,I,E,behind", EXPERTS)
def test_gated_experts(t, N, d, I, E, behind):
    _run_gated(Case(t, N, d, I, E, behind, mats=2), d, I, oproducts.ACTS[N % 3])


@pytest.mark.parametrize("N,d,I,E", [(70, 136, 200, 0), (33, 35, 201, 0), (90, 72, 264, 4)])
def test_gated_fp32_gradients(N, d, I, E):
    _run_gated(Case(BF16, N, d, I, E, mats=2), d, I, "silu", F32)


def test_backward_without_one_of_its_outputs():
    c = Case(BF16, 50, 72, 40, 4, 3, mats=2)
    wg, wu = c.w
    h, pre = moe.moe_gated(wg, wu, c.x, c.offsets, save=True)
    assert (h[int(c.off[-1]):] == 0).all() and (pre[int(c.off[-1]):] == 0).all()      # allocated by the call
    dx, dwg, dwu = moe.moe_gated_backward(c.dy, pre, wg, wu, c.x, c.offsets)
    one = moe.moe_gated_backward(c.dy, pre, wg, wu, c.x, c.offsets, out=(torch.zeros_like(dx), None, None))
    two = moe.moe_gated_backward(c.dy, pre, wg, wu, c.x, c.offsets, out=(None, torch.zeros_like(dwg), torch.zeros_like(dwu)))
    assert torch.equal(one[0], dx) and torch.equal(two[1], dwg) and torch.equal(two[2], dwu)
    y = moe.moe_linear(wg, c.x, c.offsets)
    dx, dw = moe.moe_linear_backward(c.dy, wg, c.x, c.offsets)
    assert (y[int(c.off[-1]):] == 0).all() and (dx[int(c.off[-1]):] == 0).all()
    assert torch.equal(moe.moe_linear_backward(c.dy, wg, c.x, c.offsets, out=(torch.zeros_like(dx), None))[0], dx)
    assert torch.equal(moe.moe_linear_backward(c.dy, wg, c.x, c.offsets, out=(None, torch.zeros_like(dw)))[1], dw)


@pytest.mark.parametrize("E", [0, 5])
def test_no_rows(E):
    """No rows at all: gradients of matrices are zeros."""
    lead = (E,) if E else ()
    w = torch.randn(*lead, 40, 24, device="cuda").bfloat16()
    x, dy = torch.empty(0, 24, dtype=BF16, device="cuda"), torch.empty(0, 40, dtype=BF16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda") if E else None
    assert moe.moe_linear(w, x, off).shape == (0, 40) and moe.moe_gated(w, w, x, off).shape == (0, 40)
    dx, dw = moe.moe_linear_backward(dy, w, x, off, out=(None, torch.full_like(w, 3.0)))
    assert (dw == 0).all()
    dx, dg, du = moe.moe_gated_backward(dy, torch.empty(0, 80, device="cuda"), w, w, x, off)
    assert dx.shape == (0, 24) and (dg == 0).all() and (du == 0).all()


@pytest.mark.parametrize("d,I", [(72, 200), (71, 201)])
def test_a_row_that_is_not_finite_touches_no_other(d, I):
    c = Case(BF16, 300, d, I, 4, 20, mats=2)
    wg, wu = c.w
    bad = int(c.off[np.argmax(np.diff(c.off)) + 1]) - 1         # last row of the longest bucket
    e = int(np.argmax(np.diff(c.off)))

    def run(x, dy):
        h, pre = moe.moe_gated(wg, wu, x, c.offsets, save=True)
        return (h, moe.moe_linear(wg, x, c.offsets), *moe.moe_linear_backward(dy, wg, x, c.offsets),
                *moe.moe_gated_backward(dy, pre, wg, wu, x, c.offsets))
    base = run(c.x, c.dy)
    x, dy = c.x.clone(), c.dy.clone()
    x[bad, d // 2], dy[bad, I // 2] = float("inf"), float("nan")
    got = run(x, dy)
    for a, b in zip(base, got):
        keep = torch.ones(a.shape[0], dtype=torch.bool, device="cuda")
        keep[e if a.dim() == 3 else bad] = False
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(b[~keep]).all()


@pytest.mark.parametrize("shift", [8, 4])
def test_halves_of_a_fused_matrix_and_unaligned_views(shift):
    """Gate and up as views into one [E, 2 I, d], their gradients too; and all
    tensors at addresses that are no multiples of 16 bytes."""
    E, d, I = 5, 72, 88
    c = Case(BF16, 200, d, I, E, 4, mats=2)
    base = torch.empty(E * 2 * I * d + 64, dtype=BF16, device="cuda")
    fused = base[shift:shift + E * 2 * I * d].view(E, 2 * I, d)
    fused[:, :I], fused[:, I:] = c.w[0], c.w[1]
    gfused = torch.full_like(base, 7.0)[shift:shift + E * 2 * I * d].view(E, 2 * I, d)
    xb = torch.zeros(200 * d + 64, dtype=BF16, device="cuda")[shift:shift + 200 * d].view(200, d)
    xb.copy_(c.x)
    h, pre = moe.moe_gated(c.w[0], c.w[1], c.x, c.offsets, save=True)
    hv, prev = moe.moe_gated(fused[:, :I], fused[:, I:], xb, c.offsets, save=True)
    assert torch.equal(h, hv) and torch.equal(pre, prev)
    want = moe.moe_gated_backward(c.dy, pre, c.w[0], c.w[1], c.x, c.offsets)
    got = moe.moe_gated_backward(c.dy, prev, fused[:, :I], fused[:, I:], xb, c.offsets,
                                 out=(torch.zeros_like(want[0]), gfused[:, :I], gfused[:, I:]))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert torch.equal(moe.moe_linear(c.w[0], c.x, c.offsets), moe.moe_linear(fused[:, :I], xb, c.offsets))
