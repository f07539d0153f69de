"""Rows in expert order and back, with their gradients, on the GPU against the
fp64 oracle.

Tolerances, derived: a sum of m fp32 terms, each product and addition rounded
by at most u = 2^-24 relative, is off by at most (m + 2) u times the sum of the
absolute terms (m <= 1026 here, so m u is far below 1); the result is then
rounded once to the row type, by at most eps/2 of its value (fp16: or half of
its smallest step, 2^-25, below the normal range).  The order of the terms does
not matter to this bound.  Copies and whole numbers must be equal."""
import numpy as np
import pytest

from oracle import rows as orows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SHAPES = [  # T, k, E, d
    (1, 1, 1, 1), (1, 10, 512, 2048), (3, 2, 4, 7), (5, 3, 16, 8), (64, 8, 256, 129), (128, 8, 64, 64),
    (129, 8, 64, 1001), (257, 10, 512, 40), (33, 40, 1024, 33), (700, 3, 8, 515), (2, 300, 512, 24),
    (32, 8, 64, 257), (43, 6, 30, 65), (20, 5, 512, 1500), (1100, 2, 8, 1100), (1030, 3, 4, 3), (13107, 5, 16, 8), (16384, 4, 16, 9), (7000, 10, 3, 2), (5000, 2, 4, 8), (4500, 2, 8, 40),
    (21850, 3, 1024, 2), (35000, 2, 7, 5), (33000, 2, 40, 3),
]


def _np(t):
    return t.detach().cpu().double().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def _within(got, ref, mag, m, t):
    """|got - ref| <= (m + 2) u mag, plus the rounding of the result to type t."""
    e = torch.finfo(t).eps / 2 if t is not torch.float32 else 0.0
    tol = (m + 2) * U * mag
    tol = tol + e * (np.abs(ref) + tol) + (2.0 ** -25 if t is torch.float16 else 2.0 ** -126)
    bad = np.argwhere(~(np.abs(_np(got) - ref) <= tol))
    assert bad.size == 0, (bad[:4].tolist(), np.abs(_np(got) - ref).max())


def _case(T, k, E, d, t, seed=0, drop=0.15):
    g = np.random.default_rng([T, k, E, d, seed])
    idx = np.stack([g.permutation(E)[:k] if k <= E else g.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    if T > 2:
        idx[g.random((T, k)) < drop] = -1
        idx[T - 1] = E                                    # a token without any expert
        idx[0, 0] = idx[0, -1]                            # the same expert twice
    x = torch.from_numpy(g.standard_normal((T, d), dtype=np.float32)).cuda().to(t)
    w = g.random((T, k), dtype=np.float32)
    return g, idx, torch.from_numpy(idx).cuda(), x, w


def _rows(g, n, d, t):
    return torch.from_numpy(g.standard_normal((n, d), dtype=np.float32)).cuda().to(t)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("T,k,E,d", SHAPES)
def test_sort_and_its_gradient(T, k, E, d, t):
    t = TYPES[t]
    g, idx, idx_d, x, _ = _case(T, k, E, d, t)
    n = T * k
    out = (torch.full((n, d), float("nan"), dtype=t, device="cuda"), torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
           torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), -9, dtype=torch.int32, device="cuda"))
    X, off, pairs, row_of = moe.moe_sort_tokens(x, idx_d, E, out=out)
    rX, roff, rpairs, rrow = orows.sort_rows(_np(x), idx, E)
    live = int(roff[-1])
    assert np.array_equal(_np(off), roff) and np.array_equal(_np(row_of), rrow)
    assert np.array_equal(_np(pairs)[:live], rpairs) and (_np(pairs)[live:] == -9).all()
    assert np.array_equal(_np(X)[:live], rX) and torch.isnan(X[live:]).all()
    dX = _rows(g, n, d, t)
    dX[live:] = float("nan")                              # rows no pair has are not read
    dx = moe.moe_sort_tokens_backward(dX, row_of)
    ref = orows.sort_rows_grad(_np(dX)[:max(live, 1)], rrow)
    _within(dx, ref, orows.sort_rows_grad(np.abs(_np(dX)[:max(live, 1)]), rrow), k, t)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("T,k,E,d", SHAPES)
def test_unsort_and_its_gradients(T, k, E, d, t, shared):
    t = TYPES[t]
    g, idx, _, _, w = _case(T, k, E, d, t, 1)
    n = T * k
    row = orows.sort_rows(np.zeros((T, 1)), idx, E)[3]
    w[row < 0] = np.nan                                   # the weight of a pair without a row is not used
    live = int((row >= 0).sum())
    rows = _rows(g, n, d, t)
    rows[live:] = float("nan")
    sh = _rows(g, T, d, t) if shared else None
    sg = torch.from_numpy(g.random(T, dtype=np.float32)).cuda() if shared else None
    row_d, w_d = torch.from_numpy(row).cuda(), torch.from_numpy(w).cuda()
    y = moe.moe_unsort_combine(rows, row_d, w_d, sh, sg)
    wz = np.where(row >= 0, w, 0)
    r64, sh64, sg64 = _np(rows)[:max(live, 1)], None if sh is None else _np(sh), None if sg is None else _np(sg)
    a = lambda v: None if v is None else np.abs(v)
    _within(y, orows.unsort(r64, row, wz, sh64, sg64), orows.unsort(a(r64), row, wz, a(sh64), sg64), k + 1, t)
    dy = _rows(g, T, d, t)
    out = (torch.full((n, d), float("nan"), dtype=t, device="cuda"), torch.full((T, k), -9.0, device="cuda"),
           torch.empty_like(sh) if shared else None, torch.empty_like(sg) if shared else None)
    dr, dw, ds, dg = moe.moe_unsort_combine_backward(dy, rows, row_d, w_d, sh, sg, out=out)
    rdr, rdw, rds, rdg = orows.unsort_grad(_np(dy), r64, row, wz, sh64, sg64)
    _, mw, _, mg = orows.unsort_grad(a(_np(dy)), a(r64), row, wz, a(sh64), sg64)
    _within(dr[:live], rdr[:live], np.abs(rdr[:live]), 0, t)
    assert torch.isnan(dr[live:]).all()                   # rows no pair has keep what they held
    _within(dw, rdw, mw, d, torch.float32)
    if shared:
        _within(ds, rds, np.abs(rds), 0, t)
        _within(dg, rdg, mg, d, torch.float32)


def test_unsort_gradients_against_differences():
    """y is linear in the rows and in the weights apart, so with small whole
    numbers every product and sum below is exact and so are the differences."""
    T, k, E, d = 37, 4, 16, 72
    g = np.random.default_rng(5)
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    row = torch.from_numpy(orows.sort_rows(np.zeros((T, 1)), idx, E)[3]).cuda()
    whole = lambda *s: torch.from_numpy(g.integers(-8, 9, s).astype(np.float32)).cuda()
    rows, w, dy, dr, dw = whole(T * k, d), whole(T, k), whole(T, d), whole(T * k, d), whole(T, k)
    grows, gw, _, _ = moe.moe_unsort_combine_backward(dy, rows, row, w)
    y = moe.moe_unsort_combine(rows, row, w)
    assert torch.equal(((moe.moe_unsort_combine(rows + dr, row, w) - y) * dy).sum(), (grows * dr).sum())
    assert torch.equal(((moe.moe_unsort_combine(rows, row, w + dw) - y) * dy).sum(), (gw * dw).sum())
    x, dX = whole(T, d), whole(T * k, d)
    X = moe.moe_sort_tokens(x, torch.from_numpy(idx).cuda(), E)[0]
    assert torch.equal((X * dX).sum(), (x * moe.moe_sort_tokens_backward(dX, row)).sum())


@pytest.mark.parametrize("T,k", [(1, 3), (200, 8)])
def test_no_pair_has_an_expert(T, k):
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    x = torch.randn(T, 24, device="cuda")
    X, off, pairs, row = moe.moe_sort_tokens(x, idx, 9, out=(
        torch.full((T * k, 24), 7.0, device="cuda"), torch.ones(10, dtype=torch.int32, device="cuda"),
        torch.full((T * k,), 5, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")))
    assert (off == 0).all() and (row == -1).all() and (X == 7).all() and (pairs == 5).all()
    assert (moe.moe_sort_tokens_backward(X, row) == 0).all()
    sh = torch.randn(T, 24, device="cuda")
    one = torch.ones(T, device="cuda")
    assert torch.equal(moe.moe_unsort_combine(X, row, torch.ones(T, k, device="cuda"), sh, one), sh)


def test_no_tokens():
    x = torch.empty(0, 16, device="cuda")
    X, off, pairs, row = moe.moe_sort_tokens(x, torch.empty(0, 4, dtype=torch.int32, device="cuda"), 6)
    assert X.shape == (0, 16) and off.tolist() == [0] * 7 and pairs.numel() == 0 and row.shape == (0, 4)
    assert moe.moe_sort_tokens_backward(X, row).shape == (0, 16)
    assert moe.moe_unsort_combine(X, row, torch.empty(0, 4, device="cuda")).shape == (0, 16)
    assert moe.moe_unsort_combine_backward(x, X, row, torch.empty(0, 4, device="cuda"))[0].shape == (0, 16)


def test_rows_that_start_at_odd_addresses():
    """Odd row lengths and tensors that start one element into an allocation."""
    T, k, E, d = 70, 4, 8, 99
    for t in TYPES.values():
        g, idx, idx_d, x, w = _case(T, k, E, d, t, 3)
        buf = torch.empty(T * d + 1, dtype=t, device="cuda")
        xo = buf[1:].view(T, d)
        xo.copy_(x)
        for a, b in zip(moe.moe_sort_tokens(xo, idx_d, E), moe.moe_sort_tokens(x, idx_d, E)):
            live = int((_np(idx_d) >= 0).sum() - (_np(idx_d) >= E).sum())
            n = a.shape[0] if a.shape[0] != T * k else live
            assert torch.equal(a[:n], b[:n])


def test_sort_matches_bucketing():
    for T, k, E in [(64, 8, 32), (600, 4, 100)]:
        idx = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
        _, off, pairs, _ = moe.moe_sort_tokens(torch.randn(T, 8, device="cuda"), idx, E)
        _, off2, pairs2 = moe.moe_bucket_tokens(idx, E)
        assert torch.equal(off, off2) and torch.equal(pairs, pairs2)


@pytest.mark.parametrize("T", [5, 300, 9000])
def test_streams_and_graphs(T):
    """On another stream, and captured: every replay on new inputs equals the
    eager call, with the program's own work between."""
    k, E, d = 8, 64, 264
    t = torch.bfloat16
    _, _, idx, x, w = _case(T, k, E, d, t, 4)
    w, dy = torch.from_numpy(w).cuda(), torch.randn(T, d, device="cuda").to(t)

    def step(stream=None):
        X, off, pairs, row = moe.moe_sort_tokens(x, idx, E, stream=stream, out=bufs)
        y = moe.moe_unsort_combine(X, row, w, stream=stream)
        dX, dw, _, _ = moe.moe_unsort_combine_backward(dy, X, row, w, stream=stream, out=(bufs2, dwb, None, None))
        return y, dX, dw, moe.moe_sort_tokens_backward(dX, row, stream=stream)

    bufs = (torch.zeros(T * k, d, dtype=t, device="cuda"), torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
            torch.zeros(T * k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"))
    bufs2, dwb = torch.zeros(T * k, d, dtype=t, device="cuda"), torch.zeros(T, k, device="cuda")
    want = [a.clone() for a in step()]
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
        x.copy_(torch.randn(T, d, device="cuda").to(t))
        idx.copy_(torch.roll(idx, 1, 0))
        graph.replay()
        got = [a.clone() for a in held]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step())), rep


@pytest.mark.parametrize("T,k,E,d,skew", [
    (104857, 10, 512, 2, False), (65536, 16, 32, 3, False),       # up to 2^20 pairs, 4096 a block
    (200003, 2, 1024, 1, False), (131072, 8, 64, 1, True),        # one expert of most pairs
    (65537, 16, 40, 1, False)])                                   # one token past one launch
def test_sort_of_many_pairs(T, k, E, d, skew):
    """The sort near the border of one launch, which has two counters an expert
    and up to 64 rounds of ranks a block: whole numbers and copies are equal."""
    g = np.random.default_rng([T, k])
    idx = g.integers(0, E, (T, k)).astype(np.int32)
    if skew:
        idx[g.random((T, k)) < 0.9] = E - 3
    idx[g.random((T, k)) < 0.1] = -1
    idx[-1], idx[T // 2] = E, -7
    n, key = T * k, np.where((idx.ravel() >= 0) & (idx.ravel() < E), idx.ravel(), E)
    order = np.argsort(key, kind="stable")
    live = int((key < E).sum())
    row = np.full(n, -1, np.int32)
    row[order[:live]] = np.arange(live)
    x = torch.randn(T, d, device="cuda")
    out = (torch.full((n, d), float("nan"), device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda"),
           torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda"))
    X, off, pairs, row_of = moe.moe_sort_tokens(x, torch.from_numpy(idx).cuda(), E, out=out)
    assert np.array_equal(_np(off), np.searchsorted(key[order], np.arange(E + 1)))
    assert np.array_equal(_np(pairs)[:live], order[:live]) and (pairs[live:] == -9).all()
    assert np.array_equal(_np(row_of).ravel(), row)
    assert torch.equal(X[:live], x[torch.from_numpy(order[:live] // k).cuda()]) and torch.isnan(X[live:]).all()


def _leave_behind(*shape, dtype=torch.float32):
    """A freed block of that size full of values nobody should see."""
    del_me = torch.full(shape, float("nan") if dtype.is_floating_point else 1 << 30, dtype=dtype, device="cuda")
    del del_me


def test_rows_behind_the_last_bucket_of_allocated_outputs():
    """Buffers that the calls allocate: zeros in the rows (and -1 in the pair
    list) that no pair has, not what the memory held before."""
    T, k, E, d, n_out = 300, 4, 8, 576, 40
    idx = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    idx[200:] = -1
    x, live = torch.randn(T, d, device="cuda").bfloat16(), 800
    _leave_behind(T * k, d, dtype=torch.bfloat16)
    _leave_behind(T * k, dtype=torch.int32)
    X, off, pairs, row = moe.moe_sort_tokens(x, idx, E)
    assert int(off[E]) == live and (X[live:] == 0).all() and (pairs[live:] == -1).all() and (pairs[:live] >= 0).all()
    _leave_behind(T * k, d, dtype=torch.bfloat16)
    dX = moe.moe_unsort_combine_backward(x, X, row, torch.rand(T, k, device="cuda"))[0]
    assert (dX[live:] == 0).all()
    packed = torch.zeros(E, moe.moe_linear_bytes(d, n_out), dtype=torch.uint8, device="cuda")
    _leave_behind(T * k, n_out)
    y = moe.moe_expert_linear_int4(packed, None, X, off, n_out)
    assert (y == 0).all()


def test_two_graphs_that_share_a_workspace():
    """The four launches of many pairs of few experts, captured twice with one
    workspace and replayed in turn on new inputs."""
    T, k, E, d = 35000, 2, 3, 5
    g = torch.Generator(device="cuda").manual_seed(9)
    ws = torch.empty(moe.moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    sets = []
    for _ in range(2):
        x, idx = torch.randn(T, d, generator=g, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
        bufs = (torch.zeros(T * k, d, device="cuda"), torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
                torch.full((T * k,), -1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_sort_tokens(x, idx, E, workspace=ws, out=bufs)
        sets.append((x, idx, bufs, graph))
    for rep in range(3):
        for x, idx, bufs, graph in sets:
            x.normal_(generator=g)
            idx.random_(0, E, generator=g)
        for x, idx, bufs, graph in sets:
            graph.replay()
        for x, idx, bufs, graph in sets:
            want = moe.moe_sort_tokens(x, idx, E)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bufs, want)), rep
            assert torch.equal(bufs[0], x[bufs[2].long() // k])


def test_more_than_2_31_elements():
    """Rows past 4 GiB and 2^31 elements.  Sixteen equal bf16 rows sum to an
    exact sixteenfold, and with weights of 1/16 to the row itself."""
    T, k, E, d = 66000, 16, 32, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    X, off, pairs, row = moe.moe_sort_tokens(x, idx, E)
    assert X.numel() > 1 << 31 and int(off[E]) == T * k
    for a in range(0, T * k, 1 << 17):
        b = min(a + (1 << 17), T * k)
        assert torch.equal(X[a:b], x[pairs[a:b].long() // k])
    assert torch.equal(moe.moe_sort_tokens_backward(X, row), x * 16)
    w = torch.full((T, k), 1 / 16, device="cuda")
    assert torch.equal(moe.moe_unsort_combine(X, row, w), x)
    dX, dw, _, _ = moe.moe_unsort_combine_backward(x, X, row, w)
    at = torch.tensor([0, T * k // 2, T * k - 1], device="cuda")
    assert torch.equal(dX[at], x[pairs[at].long() // k] / 16)
    t = torch.tensor([0, T // 2, T - 1], device="cuda")
    n2 = x[t].double().square().sum(1, keepdim=True)
    assert ((dw[t].double() - n2).abs() <= (d + 2) * U * n2).all()


def test_tensors_that_do_not_fit_are_refused():
    x = torch.randn(4, 64, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w, row = torch.ones(4, 2, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    rows = torch.randn(8, 64, device="cuda")
    for call in [lambda: moe.moe_sort_tokens(x[:, ::2], idx, 4), lambda: moe.moe_sort_tokens(x, idx.long(), 4),
                 lambda: moe.moe_sort_tokens(x, idx[:3], 4), lambda: moe.moe_sort_tokens(x, idx.cpu(), 4),
                 lambda: moe.moe_sort_tokens(x.double(), idx, 4),
                 lambda: moe.moe_sort_tokens_backward(rows[:7], row),
                 lambda: moe.moe_unsort_combine(rows, row, w.half()), lambda: moe.moe_unsort_combine(rows, row, None),
                 lambda: moe.moe_unsort_combine(rows, row, w, x.half(), w[:, 0].contiguous()),
                 lambda: moe.moe_unsort_combine_backward(x.half(), rows, row, w),
                 lambda: moe.moe_sort_tokens(x, idx, 4, workspace=torch.zeros(64, device="cuda"))]:
        with pytest.raises(ValueError):
            call()
    for call in [lambda: moe.moe_unsort_combine(rows, row, w, x, None), lambda: moe.moe_sort_tokens(x, idx, 0),
                 lambda: moe.moe_sort_tokens(x, idx, 4, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(moe.MoeError):
            call()


def _calls():
    """Each call of this kind as (name, function of float tensors by name)."""
    T, k, E, d = 6, 2, 4, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = r(T, d)
    _, off, pairs, row = moe.moe_sort_tokens(x, idx, E)
    packed = torch.zeros(E, moe.moe_linear_bytes(d, 8), dtype=torch.uint8, device="cuda")
    rows, w, sg, b16 = r(T * k, d), r(T, k), r(T), lambda *s: r(*s).bfloat16()
    return [
        (lambda x: moe.moe_sort_tokens(x, idx, E)[0], dict(x=x)),
        (lambda dx: moe.moe_sort_tokens_backward(dx, row), dict(dx=rows)),
        (lambda y, w, s, g: moe.moe_unsort_combine(y, row, w, s, g), dict(y=rows, w=w, s=x, g=sg)),
        (lambda dy, y, w, s, g: moe.moe_unsort_combine_backward(dy, y, row, w, s, g)[0],
         dict(dy=x, y=rows, w=w, s=x.clone(), g=sg)),
        (lambda x: moe.moe_linear_int4(packed[0], x, 8), dict(x=b16(T, d))),
        (lambda x, out: moe.moe_linear_int4(packed[0], x, 8, out=out), dict(x=b16(T, d), out=r(T, 8))),
        (lambda x: moe.moe_expert_linear_int4(packed, None, x, off, 8), dict(x=b16(T * k, d))),
        (lambda x, W, w, s, dw, ds: moe.moe_router_topk_backward(x, W, idx, w, s, dw, ds, off, pairs)[0],
         dict(x=b16(T, d), W=r(E + 1, d), w=w, s=sg, dw=r(T, k), ds=r(T))),
    ]


def test_tensors_whose_gradient_would_be_lost_are_refused():
    import torch.autograd.forward_ad as fwd
    for f, args in _calls():
        want = f(**args)
        for name, v in args.items():
            leaf = dict(args, **{name: v.clone().requires_grad_()})
            with pytest.raises(ValueError, match="requires_grad"):
                f(**leaf)
            with torch.no_grad():
                assert torch.equal(f(**leaf), want)
            with fwd.dual_level(), pytest.raises(ValueError, match="tangent"):
                f(**dict(args, **{name: fwd.make_dual(v.clone(), torch.ones_like(v))}))


def test_sort_and_way_back_as_an_autograd_function():
    """The calls as forward and backward of a torch.autograd.Function, against
    autograd of the same in fp64; tolerance as above: dx is a sum of k rounded
    products, dw one of d products."""
    T, k, E, d = 50, 3, 6, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)

    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            X, _, _, row = moe.moe_sort_tokens(x, idx, E)
            ctx.save_for_backward(X, row, w)
            return moe.moe_unsort_combine(X, row, w)

        @staticmethod
        def backward(ctx, dy):
            X, row, w = ctx.saved_tensors
            dX, dw, _, _ = moe.moe_unsort_combine_backward(dy.contiguous(), X, row, w)
            return moe.moe_sort_tokens_backward(dX, row), dw

    x = torch.randn(T, d, generator=g, device="cuda").requires_grad_()
    w = torch.randn(T, k, generator=g, device="cuda").requires_grad_()
    dy = torch.randn(T, d, generator=g, device="cuda")
    (Route.apply(x, w) * dy).sum().backward()
    x64, w64 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ((w64.sum(1, keepdim=True) * x64) * dy.double()).sum().backward()
    live_x = (w64.abs().sum(1, keepdim=True) * dy.double().abs()).detach()
    live_w = (x64.abs() * dy.double().abs()).sum(1, keepdim=True).detach()
    assert ((x.grad.double() - x64.grad).abs() <= (k + 2) * U * live_x).all()
    assert ((w.grad.double() - w64.grad).abs() <= (d + 2) * U * live_w).all()
