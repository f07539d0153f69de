"""4-bit products on the GPU against fp64.

Tolerance, derived: the products q x and x are exact (4 + 8 significant bits),
their sums over a group of at most 128 inputs are taken in fp32 with each
addition off by at most 2^-23 of the partial sum (half of that for an adder
that rounds to nearest), the two sums are scaled and added (three roundings)
and the groups are added one after the other and across at most 16 partial
sums.  With c = 16 + q <= 31 the error of y[o] is at most
    (128 + 3 + G + 16) 2^-23 sum_g (|s| sum c |x| + |b - 16 s| sum |x|)."""
import numpy as np
import pytest

import moe_synth as ms
from gpu_support import DeviceLayer
from oracle import layer as olayer
from oracle import rows as orows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")


def _matrix(rng, out, n_in, group):
    codes = rng.integers(0, 16, (out, n_in), dtype=np.uint8)
    s = rng.uniform(0.002, 0.02, (out, n_in // group)).astype(np.float16)
    return codes, s, (-8 * s.astype(np.float32) * rng.uniform(0.9, 1.1, s.shape)).astype(np.float16)


def _x(rng, T, n_in):
    bits = ms.f32_to_bf16_bits(rng.standard_normal((T, n_in), dtype=np.float32))
    return olayer.bf16_to_f64(bits), torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def _check(y, x, m, what=""):
    codes, s, b = m
    G = s.shape[1]
    group = codes.shape[1] // G
    up = lambda a: np.repeat(np.asarray(a, np.float64), group, axis=1)
    mag = np.abs(x) @ (np.abs(up(s)) * (16.0 + codes) + np.abs(up(b.astype(np.float64) - 16.0 * s.astype(np.float64)))).T
    err = np.abs(y.cpu().double().numpy() - x @ orows.linear_weights(*m).T)
    tol = (128 + 3 + G + 16) * 2.0 ** -23 * mag
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, (what, bad[:4].tolist(), float(np.nanmax(err / np.maximum(tol, 1e-300))))


@pytest.mark.parametrize("T,n_in,n_out,group", [
    (1, 64, 1, 64), (1, 32, 3, 32), (1, 128, 17, 128), (1, 2048, 512, 64), (2, 320, 100, 64), (7, 96, 33, 32),
    (8, 2048, 130, 64), (15, 192, 16, 64), (16, 1024, 47, 128), (17, 256, 65, 64), (31, 512, 40, 32),
    (33, 4096, 72, 128), (48, 640, 129, 64), (64, 64, 64, 64), (65, 1088, 31, 64), (130, 32, 20, 32),
    (200, 448, 50, 64), (3, 8192, 24, 64), (1, 65536, 5, 64), (300, 128, 1, 128), (5, 1920, 1000, 128),
    (300, 64, 4100, 64), (1100, 128, 1000, 128), (16, 256, 9000, 64), (3, 128, 20000, 32), (2, 64, 70000, 64),
    (12, 2048, 4200, 128), (40, 96, 3100, 32)])
def test_linear(T, n_in, n_out, group):
    rng = np.random.default_rng([T, n_in, n_out, group])
    m = _matrix(rng, n_out, n_in, group)
    w = torch.from_numpy(moe.moe_pack_linear_int4(*m)).cuda()
    x, xd = _x(rng, T, n_in)
    y = moe.moe_linear_int4(w, xd, n_out, group)
    _check(y, x, m)
    # the same row of x gives the same bits wherever it sits among rows of the same number
    assert torch.equal(moe.moe_linear_int4(w, xd.flip(0).contiguous(), n_out, group), y.flip(0))


def _packed_f64(w, n_in, n_out, group):
    """fp64 [n_out][n_in] of a packed matrix on the device."""
    nb = n_in * n_out // 2
    byte = w[:nb].view(n_in // 32, n_out, 16)
    q = torch.stack([byte & 15, byte >> 4], -1).view(n_in // 32, n_out, 32).permute(1, 0, 2).reshape(n_out, n_in).double()
    sb = w[nb:nb + n_in // group * n_out * 4].view(torch.float16).view(n_in // group, n_out, 2).double()
    s, b = sb[..., 0].t().repeat_interleave(group, 1), sb[..., 1].t().repeat_interleave(group, 1)
    return q, s, b


def _device_matrices(g, lead, n_in, n_out, group):
    """Random packed matrices made on the device, scales as in _matrix."""
    nb = n_in * n_out // 2
    w = torch.randint(0, 256, (lead, moe.moe_linear_bytes(n_in, n_out, group)), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.empty(lead, n_in // group, n_out, device="cuda").uniform_(0.002, 0.02, generator=g)
    b = -8 * s * torch.empty_like(s).uniform_(0.9, 1.1, generator=g)
    w[:, nb:] = torch.stack([s, b], -1).half().view(lead, -1).view(torch.uint8)
    return w


def _check_on_device(y, x, w, n_in, n_out, group, what=""):
    q, s, b = _packed_f64(w, n_in, n_out, group)
    mag = x.double().abs() @ (s.abs() * (16 + q) + (b - 16 * s).abs()).t()
    err = (y.double() - x.double() @ (s * q + b).t()).abs()
    assert (err <= (128 + 3 + n_in // group + 16) * 2.0 ** -23 * mag).all(), what


# Sizes by the form that they take: weight rows a wave (16 or 32 or 64), rows of
# x a chunk, shares of the inputs joined through LDS, x in LDS, two tiles a block.
@pytest.mark.parametrize("T,n_in,n_out,group", [
    (2, 96, 4187, 32), (5, 512, 4210, 64), (7, 1152, 4157, 64),             # 32 weight rows; 1, 2, 4 shares
    (3, 288, 8201, 32), (6, 1024, 8442, 64), (7, 2048, 8917, 64),           # and x in LDS; 2, 4, 8 shares
    (33, 1024, 2827, 128), (19, 1024, 4121, 32),                            # 64 weight rows; 4, 8 shares
    (36, 256, 2738, 32), (50, 512, 2192, 32), (10, 1152, 9163, 32), (12, 1024, 16390, 64),      # and x in LDS
    (72, 288, 9603, 32), (200, 1024, 4100, 64), (65, 2176, 8200, 128)])     # 64 rows of x; 2, 4, 4 shares
def test_linear_forms(T, n_in, n_out, group):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = _device_matrices(g, 1, n_in, n_out, group)[0]
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    _check_on_device(moe.moe_linear_int4(w, x, n_out, group), x, w, n_in, n_out, group)


@pytest.mark.parametrize("N,n_in,n_out,group,E", [
    (9, 384, 5, 32, 3), (40, 1088, 33, 64, 9), (70, 4224, 40, 128, 30),      # 16 weight rows; 2, 4, 8 shares
    (460, 32, 1, 32, 276), (654, 256, 3, 32, 268), (473, 512, 5, 32, 449), (2866, 1120, 7, 32, 152),    # 32; 1, 2, 4, 8
    (590, 64, 9, 64, 601), (661, 256, 12, 32, 516), (991, 512, 16, 32, 657), (5, 1536, 9609, 32, 1),   # and x in LDS
    (417, 2048, 36, 128, 393), (737, 1152, 1, 64, 585), (643, 2048, 15, 32, 546), (1541, 1088, 3, 32, 522),  # chunks of 4, 8
    (91, 2048, 1076, 64, 63), (20, 1024, 8300, 64, 10), (1432, 32, 272, 32, 764),   # no shares; chunks of 4, 8, 16
    (9, 2048, 37760, 32, 7), (19, 1024, 14287, 32, 19),                     # two tiles a block; chunks of 4, 8
    (512, 128, 2056, 64, 256), (512, 2048, 520, 64, 256), (512, 4096, 520, 64, 256), (768, 2048, 530, 64, 256),
    (2724, 1216, 21, 64, 135), (3919, 1216, 17, 32, 166), (21, 1024, 105927, 128, 5),      # 64 weight rows
    (3830, 288, 17, 32, 232), (35, 512, 2184, 32, 2), (13, 1184, 12309, 32, 1), (3674, 32, 1031, 32, 229),    # and x in LDS
    (3217, 256, 250, 32, 16), (417, 608, 1578, 32, 11), (359, 32, 47761, 32, 11)])        # 64 rows of x
def test_expert_forms(N, n_in, n_out, group, E):
    """Buckets from empty to many chunks, and rows behind the last one."""
    g = torch.Generator(device="cuda").manual_seed(N)
    w = _device_matrices(g, E, n_in, n_out, group)
    x = torch.randn(N, n_in, generator=g, device="cuda").bfloat16()
    rng = np.random.default_rng(N)
    p = rng.permutation(1.0 / np.arange(1, E + 1) ** 1.2)
    counts = rng.multinomial(N - N // 9, p / p.sum())
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    slots = rng.permutation(E).astype(np.int32)
    out = torch.full((N, n_out), float("nan"), device="cuda")
    y = moe.moe_expert_linear_int4(w, torch.from_numpy(slots).cuda(), x, torch.from_numpy(off).cuda(), n_out, group,
                                   out=out)
    for e in np.nonzero(counts)[0]:
        _check_on_device(y[off[e]:off[e + 1]], x[off[e]:off[e + 1]], w[int(slots[e])], n_in, n_out, group, (e, counts[e]))
    assert torch.isnan(y[off[-1]:]).all()


def test_experts_whose_rows_do_not_fit_lds():
    """Long rows and many experts (280 MB of matrices, random bytes made on the
    device): sampled experts against fp64, same tolerance."""
    E, k, T, n_in, n_out = 256, 8, 160, 2112, 1040
    g = torch.Generator(device="cuda").manual_seed(5)
    nb = n_in * n_out // 2
    w = torch.randint(0, 256, (E, moe.moe_linear_bytes(n_in, n_out)), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.empty(E, n_in // 64, n_out, 1, device="cuda").uniform_(0.002, 0.02, generator=g)
    w[:, nb:] = torch.cat([s, -8 * s], -1).half().view(E, -1).view(torch.uint8)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    X, off, _, _ = moe.moe_sort_tokens(x, idx, E)
    y = moe.moe_expert_linear_int4(w, None, X, off, n_out)
    o = off.tolist()
    for e in range(0, E, 17):
        if o[e + 1] > o[e]:
            q, sc, b = _packed_f64(w[e], n_in, n_out, 64)
            xe = X[o[e]:o[e + 1]].double()
            mag = xe.abs() @ (sc.abs() * (16 + q) + (b - 16 * sc).abs()).t()
            err = (y[o[e]:o[e + 1]].double() - xe @ (sc * q + b).t()).abs()
            assert (err <= (128 + 3 + n_in // 64 + 16) * 2.0 ** -23 * mag).all(), e


@pytest.mark.parametrize("T", [1, 20])
def test_a_matrix_past_2_gib(T):
    """Byte offsets past 2^31 (random bytes made on the device): output rows
    across the matrix against fp64, same tolerance."""
    n_in, n_out = 4096, 1_100_003
    g = torch.Generator(device="cuda").manual_seed(T)
    nb = n_in * n_out // 2
    w = torch.empty(moe.moe_linear_bytes(n_in, n_out), dtype=torch.uint8, device="cuda")
    assert w.numel() > 1 << 31
    w[:nb].random_(0, 256, generator=g)
    s = torch.empty(n_in // 64, n_out, 1, device="cuda").uniform_(0.002, 0.02, generator=g)
    w[nb:] = torch.cat([s, -8 * s], -1).half().view(-1).view(torch.uint8)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    y = moe.moe_linear_int4(w, x, n_out)
    rows = torch.tensor([0, 1, 17, n_out // 2, n_out - 18, n_out - 2, n_out - 1], device="cuda")
    byte = w[:nb].view(n_in // 32, n_out, 16)[:, rows]
    q = torch.stack([byte & 15, byte >> 4], -1).view(n_in // 32, len(rows), 32).permute(1, 0, 2).reshape(len(rows), n_in)
    sb = w[nb:].view(torch.float16).view(n_in // 64, n_out, 2)[:, rows].double()
    sc, b = sb[..., 0].t().repeat_interleave(64, 1), sb[..., 1].t().repeat_interleave(64, 1)
    mag = x.double().abs() @ (sc.abs() * (16 + q.double()) + (b - 16 * sc).abs()).t()
    err = (y[:, rows].double() - x.double() @ (sc * q.double() + b).t()).abs()
    assert (err <= (128 + 3 + n_in // 64 + 16) * 2.0 ** -23 * mag).all()
    assert torch.isfinite(y).all()


def test_linear_small_and_large_values():
    """Subnormal fp16 scales, and activations from 2^-60 to 2^110 in one row."""
    rng = np.random.default_rng(6)
    c, s, b = _matrix(rng, 33, 256, 64)
    s = (s.astype(np.float32) * 2.0 ** -12).astype(np.float16)
    b = (b.astype(np.float32) * 2.0 ** -12).astype(np.float16)
    assert (s.astype(np.float32) < 2.0 ** -14).all()
    w = torch.from_numpy(moe.moe_pack_linear_int4(c, s, b)).cuda()
    x, xd = _x(rng, 5, 256)
    scale = 2.0 ** rng.integers(-60, 110, (5, 1))
    y = moe.moe_linear_int4(w, (xd.float() * torch.from_numpy(scale).float().cuda()).bfloat16(), 33)
    _check(y, x * scale, (c, s, b))


@pytest.mark.parametrize("T,n_in,n_out,group", [(3, 1024, 40, 128), (3, 65536, 17, 32), (20, 512, 8200, 64), (70, 256, 16500, 32)])
def test_linear_at_the_largest_values(T, n_in, n_out, group):
    """Scales up to 16 and biases up to 128 against the largest x that the
    documented bound admits, the sums of magnitudes just below 2^127; the first
    rows of W are zeros made of the largest scale (16 * 8 - 128)."""
    rng = np.random.default_rng([T, n_in])
    c, s, b = _matrix(rng, n_out, n_in, group)
    s = (s.astype(np.float32) * 800).astype(np.float16)
    b = (-8 * s.astype(np.float32)).astype(np.float16)
    c[:4], s[:4], b[:4] = 8, 16.0, -128.0
    assert s.max() <= 16 and np.abs(b).max() <= 128
    x, _ = _x(rng, T, n_in)
    x = np.sign(x) * np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -8))))
    x[0] = 1.0                                          # every term of the same sign
    s64, b64 = s.astype(np.float64), b.astype(np.float64)
    per = ((31 * np.abs(s64) + np.abs(b64 - 16 * s64)).sum(1).max()) * group * np.abs(x).max(1)
    x *= np.exp2(126 - np.ceil(np.log2(per)))[:, None]
    assert (per * np.exp2(126 - np.ceil(np.log2(per))) < 2.0 ** 127).all() and np.abs(x).max() > 2.0 ** 95
    xd = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    assert np.array_equal(xd.double().cpu().numpy(), x)
    y = moe.moe_linear_int4(torch.from_numpy(moe.moe_pack_linear_int4(c, s, b)).cuda(), xd, n_out, group)
    _check(y, x, (c, s, b))
    assert (y[0, :4] == 0).all()                        # equal terms: the two sums cancel exactly


def test_linear_no_rows_and_non_finite_rows():
    rng = np.random.default_rng(3)
    m = _matrix(rng, 40, 256, 64)
    w = torch.from_numpy(moe.moe_pack_linear_int4(*m)).cuda()
    assert moe.moe_linear_int4(w, torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), 40).shape == (0, 40)
    x, xd = _x(rng, 5, 256)
    y = moe.moe_linear_int4(w, xd, 40)
    xd[2, 7], xd[4, 255] = float("nan"), float("inf")
    z = moe.moe_linear_int4(w, xd, 40)
    assert torch.equal(z[[0, 1, 3]], y[[0, 1, 3]]) and not torch.isfinite(z[[2, 4]]).any()


def test_linear_unaligned_weights_and_streams():
    """Packed matrices need 4-byte alignment only; another stream, and a graph."""
    rng = np.random.default_rng(4)
    m = _matrix(rng, 77, 192, 64)
    p = torch.from_numpy(moe.moe_pack_linear_int4(*m)).cuda()
    buf = torch.zeros(p.numel() + 4, dtype=torch.uint8, device="cuda")
    buf[4:] = p
    x, xd = _x(rng, 6, 192)
    y = moe.moe_linear_int4(p, xd, 77)
    assert torch.equal(moe.moe_linear_int4(buf[4:], xd, 77), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = moe.moe_linear_int4(p, xd, 77, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        z = moe.moe_linear_int4(p, xd, 77)
    for _ in range(3):
        xd.copy_(_x(rng, 6, 192)[1])
        graph.replay()
        got = z.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, moe.moe_linear_int4(p, xd, 77))


@pytest.mark.parametrize("T,k,E,n_in,n_out,group", [
    (1, 1, 1, 64, 16, 64), (1, 10, 512, 256, 32, 64), (3, 2, 16, 96, 33, 32), (64, 8, 64, 128, 48, 128),
    (40, 6, 20, 320, 65, 64), (200, 3, 4, 64, 20, 64), (900, 2, 5, 64, 17, 32), (9, 4, 1024, 64, 40, 64),
    (64, 8, 64, 128, 1100, 64), (400, 3, 4, 128, 2100, 32), (30, 8, 16, 192, 600, 64)])
def test_experts(T, k, E, n_in, n_out, group):
    rng = np.random.default_rng([T, k, E, n_in])
    mats = [_matrix(rng, n_out, n_in, group) for _ in range(E)]
    slots = rng.permutation(E + 3)[:E].astype(np.int32)
    nb = moe.moe_linear_bytes(n_in, n_out, group)
    slab = np.zeros((E + 3, nb + 12), np.uint8)
    for e in range(E):
        slab[slots[e], :nb] = moe.moe_pack_linear_int4(*mats[e])
    slab = torch.from_numpy(slab).cuda()
    idx = np.minimum(rng.geometric(0.2, (T, k)) - 1, E).astype(np.int32)      # skewed; some pairs without an expert
    idx[0, 0] = E - 1
    x, xd = _x(rng, T, n_in)
    X, off, pairs, row = moe.moe_sort_tokens(xd, torch.from_numpy(idx).cuda(), E)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T * k, n_out), float("nan"), device="cuda")
    y = moe.moe_expert_linear_int4(slab[:, :nb], torch.from_numpy(slots).cuda(), X, off, n_out, group, error=err,
                                   out=out)
    rX, roff, rpairs, _ = orows.sort_rows(x, idx, E)
    for e in range(E):
        if roff[e + 1] > roff[e]:
            _check(y[roff[e]:roff[e + 1]], rX[roff[e]:roff[e + 1]], mats[e], e)
    assert torch.isnan(y[roff[-1]:]).all() and int(err) == 0
    # without a table: expert e in slot e
    order = torch.from_numpy(np.argsort(slots)).cuda()
    direct = torch.empty(E, nb, dtype=torch.uint8, device="cuda")
    direct[:] = slab[torch.from_numpy(slots).cuda().long(), :nb]
    z = moe.moe_expert_linear_int4(direct, None, X, off, n_out, group)
    assert torch.equal(z[:roff[-1]], y[:roff[-1]])


def test_missing_expert_gives_zeros_and_the_error_bit():
    rng = np.random.default_rng(8)
    E, n_in, n_out = 6, 64, 24
    mats = [_matrix(rng, n_out, n_in, 64) for _ in range(E)]
    slab = torch.from_numpy(np.stack([moe.moe_pack_linear_int4(*m) for m in mats])).cuda()
    idx = torch.tensor([[0, 2], [2, 4], [5, 1]], dtype=torch.int32, device="cuda")
    X, off, _, _ = moe.moe_sort_tokens(_x(rng, 3, n_in)[1], idx, E)
    full = moe.moe_expert_linear_int4(slab, None, X, off, n_out)
    for bad in (-1, 6, 1 << 30):
        table = torch.arange(E, dtype=torch.int32, device="cuda")
        table[2] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = moe.moe_expert_linear_int4(slab, table, X, off, n_out, error=err)
        want = full.clone()
        want[int(off[2]):int(off[3])] = 0
        assert torch.equal(y, want) and int(err) == 1
        assert torch.equal(moe.moe_expert_linear_int4(slab, table, X, off, n_out), want)
    table[2], table[3] = 2, -1                        # an absent expert that no row asks for
    err.zero_()
    assert torch.equal(moe.moe_expert_linear_int4(slab, table, X, off, n_out, error=err), full) and int(err) == 0


def test_offsets_of_other_rows_stay_in_bounds():
    """Offsets that reach past N: the rows there are not touched."""
    rng = np.random.default_rng(9)
    slab = torch.from_numpy(np.stack([moe.moe_pack_linear_int4(*_matrix(rng, 16, 64, 64)) for _ in range(4)])).cuda()
    X = _x(rng, 40, 64)[1]
    buf = torch.full((64, 16), 3.0, device="cuda")
    off = torch.tensor([0, 10, 30, 50, 60], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 10, 30, 40, 40], dtype=torch.int32, device="cuda")
    y = moe.moe_expert_linear_int4(slab, None, X, off, 16, out=buf[:40])
    assert torch.equal(y[:40], moe.moe_expert_linear_int4(slab, None, X, good, 16)) and (buf[40:] == 3).all()


def test_pool_matrices():
    L = DeviceLayer(ms.CONFIGS["tiny"])
    cfg = L.cfg
    rng = np.random.default_rng(10)
    idx = torch.from_numpy(rng.integers(0, cfg.E, (9, 2)).astype(np.int32)).cuda()
    for mat, n_in in (("gate", cfg.d), ("up", cfg.d), ("down", cfg.I)):
        x, xd = _x(rng, 9, n_in)
        X, off, _, _ = moe.moe_sort_tokens(xd, idx, cfg.E)
        y = moe.moe_pool_linear_int4(L.pool, mat, X, off)
        rX, roff, _, _ = orows.sort_rows(x, idx.cpu().numpy(), cfg.E)
        for e in range(cfg.E):
            m = L.raw(e)[mat]
            _check(y[roff[e]:roff[e + 1]], rX[roff[e]:roff[e + 1]], (m["codes"], m["scales"], m["biases"]), (mat, e))
    assert L.pool.check_error() == moe.MOE_OK
    table, _ = L.pool.read_state()
    table[int(idx[0, 0])] = -1
    L.pool.set_slot_table(table)
    moe.moe_pool_linear_int4(L.pool, "down", X, off)
    assert L.pool.check_error() == moe.MOE_ERR_NOT_RESIDENT


def test_pool_rows_behind_the_last_bucket():
    L = DeviceLayer(ms.CONFIGS["tiny"])
    cfg = L.cfg
    X = torch.zeros(50, cfg.d, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(cfg.E + 1, dtype=torch.int32, device="cuda")
    off[1:] = 7                                       # rows 7 to 49 belong to no expert
    left = torch.full((50, cfg.I), float("nan"), device="cuda")
    del left
    assert (moe.moe_pool_linear_int4(L.pool, "gate", X, off) == 0).all()


def test_a_pool_of_another_device_is_refused():
    """The pool's device is compared before the launch (a pool that claims
    another device: nothing runs)."""
    L = DeviceLayer(ms.CONFIGS["tiny"])
    X = torch.zeros(4, L.cfg.d, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(L.cfg.E + 1, dtype=torch.int32, device="cuda")
    assert L.pool.device == X.get_device()
    moe.moe_pool_linear_int4(L.pool, "gate", X, off)
    L.pool.device = X.get_device() + 1
    with pytest.raises(ValueError, match="the pool on"):
        moe.moe_pool_linear_int4(L.pool, "gate", X, off)


def test_refusals_on_the_device():
    L8 = DeviceLayer(ms.CONFIGS["tiny_int8"])
    X = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(17, dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_pool_linear_int4(L8.pool, "gate", X, off)
    assert ei.value.status == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        moe.moe_pool_linear_int4(L8.pool, "sideways", X, off)
    w = torch.zeros(moe.moe_linear_bytes(256, 8), dtype=torch.uint8, device="cuda")
    for call in [lambda: moe.moe_linear_int4(w, X.float(), 8), lambda: moe.moe_linear_int4(w[:-4], X, 8),
                 lambda: moe.moe_linear_int4(w, X.t().contiguous().t(), 8), lambda: moe.moe_linear_int4(w.cpu(), X, 8),
                 lambda: moe.moe_linear_int4(w, X, 8, out=torch.zeros(4, 9, device="cuda")),
                 lambda: moe.moe_expert_linear_int4(w, None, X, off, 8),
                 lambda: moe.moe_expert_linear_int4(w.view(1, -1)[:, ::2], None, X, off, 8)]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoeError):                 # one slot for 16 experts without a table
        moe.moe_expert_linear_int4(w.view(1, -1), None, X, off, 8)
