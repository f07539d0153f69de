"""Borders that do not fit the rows, in every output of the experts' products:
one below 0 or past N is taken as 0 or N.  Compared with the same calls on the
borders so cut, bit for bit (the sizes, and with them the forms, are the same),
and those with fp64 through the tests of the products; with guard rows around
what is written."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
G = 64                                           # guard rows on each side


def _guarded(N, cols, t):
    v = torch.full((N + 2 * G, cols), 5.0, dtype=t, device="cuda")
    return v, v[G:G + N]


def _outputs(c, off):
    """Every output of every call with these borders; rows that no bucket holds stay 5."""
    N, E, d, I = c["x"].shape[0], c["w"].shape[0], c["x"].shape[1], c["w"].shape[1]
    got, guards = {}, []

    def rows(cols, t=BF16):
        v, inner = _guarded(N, cols, t)
        guards.append(v)
        return inner
    got["y"] = moe.moe_linear(c["w"], c["x"], off, out=rows(I))
    got["dx"], got["dw"] = moe.moe_linear_backward(c["dy"], c["w"], c["x"], off, out=(rows(d), torch.empty_like(c["w"])))
    got["h"], got["pre"] = moe.moe_gated(c["w"], c["u"], c["x"], off, save=True, out=(rows(I), rows(2 * I, F32)))
    got["gdx"], got["dwg"], got["dwu"] = moe.moe_gated_backward(
        c["dy"], c["pre"], c["w"], c["u"], c["x"], off, out=(rows(d), torch.empty_like(c["w"]), torch.empty_like(c["u"])))
    if d % 16 == 0:
        got["y8"] = moe.moe_linear_fp8(*c["w8"], *c["x8"], off, out=rows(I))
    torch.cuda.synchronize()
    for v in guards:
        assert (v[:G] == 5).all() and (v[N + G:] == 5).all()
    return got


@pytest.mark.parametrize("d,I", [(144, 136), (71, 135)])
@pytest.mark.parametrize("N", [7, 40, 200, 700])               # streamed, and in tiles
def test_borders_outside_the_rows(N, d, I):
    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    E = 6
    c = dict(x=r(N, d), w=r(E, I, d), u=r(E, I, d), dy=r(N, I), pre=r(N, 2 * I).float())
    if d % 16 == 0:
        c["w8"], c["x8"] = moe.moe_quantize_fp8(c["w"], 128), moe.moe_quantize_fp8(c["x"])
    m = max(N // 2, 5)
    for borders in ([-3, 2, 5, 5, m, N + 9, N + 100], [-2 ** 31, -5, m, N - 1, N, 2 ** 31 - 1, 2 ** 31 - 1],
                    [-40, -20, -1, 3, m, m, N - 1], [N + 1] * 7, [-1] * 7, [-2 ** 31] + [2 ** 31 - 1] * 6):
        off = torch.tensor(borders, dtype=torch.int32, device="cuda")
        cut = off.clamp(0, N)
        a, b = _outputs(c, off), _outputs(c, cut)
        for k in a:
            assert torch.equal(a[k], b[k]), (borders, k)
        # and the cut borders' rows are written, the others not
        first, last = int(cut[0]), int(cut[-1])
        for k in ("y", "dx", "h", "pre", "gdx"):
            five = (b[k] == 5).all(1)
            assert five[:first].all() and five[last:].all() and not five[first:last].any(), (borders, k)


@pytest.mark.parametrize("N", [7, 200])
def test_the_first_bucket_from_a_negative_border(N):
    """Rows 0 and 1 of a bucket from -3 to 2: in y and in dW alike, against fp64."""
    d, I = 72, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randint(-8, 9, (N, n), generator=g, device="cuda").to(BF16) for n in (d, I))
    w = torch.randint(-8, 9, (2, I, d), generator=g, device="cuda").to(BF16)
    off = torch.tensor([-3, 2, N + 4], dtype=torch.int32, device="cuda")
    y = moe.moe_linear(w, x, off, out=torch.zeros(N, I, device="cuda"))
    dx, dw = moe.moe_linear_backward(dy, w, x, off, out=(torch.zeros_like(x), torch.zeros(2, I, d, device="cuda")))
    # whole numbers: sums below 2^24 are exact
    for e, a, b in ((0, 0, 2), (1, 2, N)):
        assert torch.equal(y[a:b].double(), x[a:b].double() @ w[e].double().t())
        assert torch.equal(dw[e].double(), dy[a:b].double().t() @ x[a:b].double())
        assert torch.equal(dx[a:b], (dy[a:b].double() @ w[e].double()).to(BF16))
