"""The experts' products, measured.

Each case is one pass through one operator of the package: the gated block
h = act(x Wg^T) (x Wu^T) and the product y = x W^T in 16-bit types, each over
rows of one matrix or over rows in expert order with a matrix per expert, alone
or with its gradients; and the product in 8-bit floating point (e4m3) with a
scale for every 128 inputs of a row of x and every 128 x 128 block of W,
together with the quantisation of x.  Where ``own`` is false ``run`` computes
them in plain torch operations in 32 bits; where it is true it calls the
package.  ``exact`` is the definition in 64 bits.

Shapes are those of the package's own workloads (hidden size 2048, 512 or 256
experts of intermediate size 512, 10 or 8 a token, 1 to 4096 tokens) and
generic ones around them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128                       # inputs, and outputs, that share a scale
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -96             # largest magnitude of a block below which it is taken as this


# ------------------------------------------------------------------- cases
# E = 0: one matrix for all T rows; otherwise T tokens of k rows each, sorted by expert.
def listed():
    return [
        # one decoded token through the first two matrices of its experts
        dict(name="gated_step", op="gated", T=1, k=10, E=512, d=2048, I=512, act="silu", dtype="bf16", pad=0.0,
             grad=False),
        # a batch of decoded tokens
        dict(name="gated_batch", op="gated", T=64, k=8, E=256, d=2048, I=512, act="silu", dtype="f16", pad=0.0,
             grad=False),
        # a training batch of odd sizes whose last tokens are padding
        dict(name="gated_ragged", op="gated", T=777, k=6, E=64, d=1001, I=347, act="gelu", dtype="f16", pad=0.1,
             grad=True),
        # a prompt's training step through the routed experts
        dict(name="gated_prompt", op="gated", T=4096, k=8, E=256, d=2048, I=512, act="silu", dtype="bf16", pad=0.0,
             grad=True),
        # and through one wide block for all rows
        dict(name="gated_dense", op="gated", T=4096, k=1, E=0, d=2048, I=8192, act="gelu_tanh", dtype="bf16", pad=0.0,
             grad=True),
        # one decoded token through the last matrix of its experts
        dict(name="linear_step", op="linear", T=1, k=10, E=512, n_in=512, n_out=2048, dtype="bf16", pad=0.0,
             grad=False),
        # rows of odd length through one matrix, with gradients
        dict(name="linear_odd", op="linear", T=301, k=1, E=0, n_in=1001, n_out=777, dtype="f16", pad=0.0, grad=True),
        # a prompt's training step through the experts' last matrices
        dict(name="linear_prompt", op="linear", T=4096, k=8, E=256, n_in=512, n_out=2048, dtype="bf16", pad=0.0,
             grad=True),
        # one token through an output projection over a vocabulary of odd size
        dict(name="fp8_vocab", op="fp8", T=1, k=1, E=0, n_in=2048, n_out=100003, dtype="bf16", pad=0.0),
        # one token through the first matrix of its experts
        dict(name="fp8_step", op="fp8", T=1, k=10, E=512, n_in=2048, n_out=512, dtype="bf16", pad=0.0),
        # a prompt through them, with some pairs dropped
        dict(name="fp8_prompt", op="fp8", T=4096, k=8, E=256, n_in=2048, n_out=512, dtype="bf16", pad=0.1),
        # a prompt through a wide dense projection
        dict(name="fp8_dense", op="fp8", T=4096, k=1, E=0, n_in=4096, n_out=16384, dtype="bf16", pad=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _size(rng, lo, hi, step):
    """A size spread over its logarithm: whole steps, or (step 0) any number."""
    n = _log(rng, lo, hi)
    return n if step == 0 else max(step, n // step * step)


def draw(rng):
    op = rng.choice(["gated", "linear", "fp8"])
    k, E = rng.choice([(1, 0), (1, 0), (1, 8), (2, 16), (6, 64), (8, 256), (10, 512)])
    mats = max(E, 1)
    # 16-bit rows of any length a third of the time; 8-bit rows come in pieces of 16
    step = 16 if op == "fp8" else rng.choice([0, 8, 64])
    a = _size(rng, 64, 4096, step)
    b = _size(rng, 64, min(8192 if E == 0 else 2048, (1 << 28) // (mats * a)), 0 if op == "fp8" else step)
    T = _log(rng, 1, min(4096, (1 << 35) // (k * a * b)))
    c = dict(op=op, T=T, k=k, E=E, dtype=rng.choice(["bf16", "f16"]), pad=rng.choice([0.0, 0.0, 0.2]))
    if op == "gated":
        c.update(d=a, I=b, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]), grad=rng.random() < 0.5)
    else:
        c.update(n_in=a, n_out=b)
        if op == "linear":
            c["grad"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _buckets(c, g):
    """Borders of the sorted rows [E + 1] as a router with a mild Zipf preference gives them; the rows of padded
    tokens lie behind the last border."""
    T, E, k = c["T"], c["E"], c["k"]
    pop = torch.randperm(E, generator=g, device="cuda").float() + 1.0
    idx = (0.9 * torch.randn(T, E, generator=g, device="cuda") - 0.165 * pop.log()).topk(k, dim=1).indices
    n = torch.bincount(idx[:T - int(T * c["pad"])].reshape(-1), minlength=E)
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)


def _blocks(w):
    """The largest magnitude of every 128 x 128 block of w [m][out][in] as [m][blocks][blocks], and of its element."""
    m, o, i = w.shape
    p = torch.nn.functional.pad(w.abs(), (0, -i % BLOCK, 0, -o % BLOCK))
    a = p.view(m, p.shape[1] // BLOCK, BLOCK, p.shape[2] // BLOCK, BLOCK).amax((2, 4))
    return a, a.repeat_interleave(BLOCK, 1)[:, :o].repeat_interleave(BLOCK, 2)[:, :, :i]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, mats, N = DTYPES[c["dtype"]], max(c["E"], 1), c["T"] * c["k"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def matrices(n_out, n_in):
        w = torch.empty(mats, n_out, n_in, dtype=t, device="cuda")
        for e in range(0, mats, 32):
            w[e:e + 32] = (randn(min(32, mats - e), n_out, n_in) / math.sqrt(n_in)).to(t)
        return w if c["E"] else w[0]

    st = {"case": c, "offsets": _buckets(c, g) if c["E"] else None}
    # what the plain form's loop over the experts needs on the host
    st["borders"] = st["offsets"].tolist() if c["E"] else [0, N]
    if c["op"] == "gated":
        d, I = c["d"], c["I"]
        st["x"], st["w_gate"], st["w_up"] = randn(N, d).to(t), matrices(I, d), matrices(I, d)
        # buffers that a program keeps from step to step; rows behind the last bucket keep what they hold
        st["h_out"] = torch.zeros(N, I, dtype=t, device="cuda")
        if c["grad"]:
            st["dh"] = randn(N, I).to(t)
            st["pre_out"] = torch.zeros(N, 2 * I, dtype=t, device="cuda")
            st["grads"] = (torch.zeros_like(st["x"]), torch.zeros_like(st["w_gate"]), torch.zeros_like(st["w_up"]))
            st["ws"] = torch.empty(N * 2 * I * 2 + 65536, dtype=torch.uint8, device="cuda")
    elif c["op"] == "linear":
        st["x"], st["w"] = randn(N, c["n_in"]).to(t), matrices(c["n_out"], c["n_in"])
        st["y_out"] = torch.zeros(N, c["n_out"], dtype=t, device="cuda")
        if c["grad"]:
            st["dy"] = randn(N, c["n_out"]).to(t)
            st["grads"] = (torch.zeros_like(st["x"]), torch.zeros_like(st["w"]))
    else:
        n_in, n_out = c["n_in"], c["n_out"]
        st["x"] = randn(N, n_in).to(t)
        st["w"] = torch.empty(mats, n_out, n_in, dtype=torch.float8_e4m3fn, device="cuda")
        st["w_scales"] = torch.empty(mats, -(-n_out // BLOCK), -(-n_in // BLOCK), device="cuda")
        for e in range(0, mats, 32):
            w = (randn(min(32, mats - e), n_out, n_in) / math.sqrt(n_in)).to(t).float()
            a, of = _blocks(w)
            st["w"][e:e + 32] = (E4M3_MAX * w / of).to(torch.float8_e4m3fn)
            st["w_scales"][e:e + 32] = a / E4M3_MAX
        if not c["E"]:
            st["w"], st["w_scales"] = st["w"][0], st["w_scales"][0]
        st["codes"] = torch.empty(N, n_in, dtype=torch.float8_e4m3fn, device="cuda")
        st["scales"] = torch.empty(N, -(-n_in // BLOCK), device="cuda")
        st["y_out"] = torch.zeros(N, n_out, dtype=t, device="cuda")
    return st


# ------------------------------------------------------- the package's own
def _run_own(st):
    import sparse_moe_decode_router_amd as moe
    c = st["case"]
    if c["op"] == "gated":
        if not c["grad"]:
            return {"h": moe.moe_gated(st["w_gate"], st["w_up"], st["x"], st["offsets"], act=c["act"],
                                       out=st["h_out"])}
        # what the gradients need, in fp32
        pre = torch.empty(st["x"].shape[0], 2 * c["I"], device="cuda")
        h, pre = moe.moe_gated(st["w_gate"], st["w_up"], st["x"], st["offsets"], act=c["act"], save=True,
                               out=(st["h_out"], pre))
        dx, dwg, dwu = moe.moe_gated_backward(st["dh"], pre, st["w_gate"], st["w_up"], st["x"], st["offsets"],
                                              act=c["act"], workspace=st["ws"], out=st["grads"])
        return {"h": h, "dx": dx, "dw_gate": dwg, "dw_up": dwu}
    if c["op"] == "linear":
        got = {"y": moe.moe_linear(st["w"], st["x"], st["offsets"], out=st["y_out"])}
        if c["grad"]:
            got["dx"], got["dw"] = moe.moe_linear_backward(st["dy"], st["w"], st["x"], st["offsets"], out=st["grads"])
        return got
    codes, scales = moe.moe_quantize_fp8(st["x"], out=(st["codes"], st["scales"]))
    return {"y": moe.moe_linear_fp8(st["w"], st["w_scales"], codes, scales, st["offsets"], out=st["y_out"])}


# -------------------------------------------------------------- plain form
def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    b = math.sqrt(2.0 / math.pi)
    t = torch.tanh(b * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * b * (1.0 + 3.0 * 0.044715 * g * g)


def _live(st):
    """(matrix, first row, end) of the buckets that have rows."""
    b = st["borders"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _stack(w):
    return w if w.dim() == 3 else w.unsqueeze(0)


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    x, t = st["x"], st["x"].dtype
    if c["op"] == "gated":
        wg, wu = _stack(st["w_gate"]), _stack(st["w_up"])
        got = {"h": torch.zeros_like(st["h_out"])}
        if c["grad"]:
            got.update(dx=torch.zeros_like(x), dw_gate=torch.zeros_like(st["w_gate"]),
                       dw_up=torch.zeros_like(st["w_up"]))
        for e, a, b in _live(st):
            xe, g32, u32 = x[a:b].float(), wg[e].float(), wu[e].float()
            g, u = xe @ g32.t(), xe @ u32.t()
            f, df = _act(c["act"], g)
            got["h"][a:b] = (f * u).to(t)
            if c["grad"]:
                dh = st["dh"][a:b].float()
                dg, du = dh * u * df, dh * f
                got["dx"][a:b] = (dg @ g32 + du @ u32).to(t)
                _stack(got["dw_gate"])[e] = (dg.t() @ xe).to(t)
                _stack(got["dw_up"])[e] = (du.t() @ xe).to(t)
        return got
    w = _stack(st["w"])
    got = {"y": torch.zeros_like(st["y_out"])}
    if c["op"] == "linear":
        if c["grad"]:
            got.update(dx=torch.zeros_like(x), dw=torch.zeros_like(st["w"]))
        for e, a, b in _live(st):
            xe, w32 = x[a:b].float(), w[e].float()
            got["y"][a:b] = (xe @ w32.t()).to(t)
            if c["grad"]:
                dy = st["dy"][a:b].float()
                got["dx"][a:b] = (dy @ w32).to(t)
                _stack(got["dw"])[e] = (dy.t() @ xe).to(t)
        return got
    N, n_in = x.shape
    xp = torch.nn.functional.pad(x.float(), (0, -n_in % BLOCK)).view(N, -1, BLOCK)
    a = xp.abs().amax(2, keepdim=True).clamp_min(SMALLEST)
    xq = (E4M3_MAX * xp / a).to(torch.float8_e4m3fn).float() * (a / E4M3_MAX)
    xq = xq.view(N, -1)[:, :n_in]
    ws = _stack(st["w_scales"])
    for e, a, b in _live(st):
        s = ws[e].repeat_interleave(BLOCK, 0)[:c["n_out"]].repeat_interleave(BLOCK, 1)[:, :n_in]
        got["y"][a:b] = (xq[a:b] @ (w[e].float() * s).t()).to(t)
    return got


# ----------------------------------------------------- definition, 64 bits
def _e4m3(v):
    """The e4m3 number nearest to v (ties to even): three bits behind the leading one, exponents from -6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0) - 3.0)
    return torch.round(v / step) * step


def _slope(name, g):
    """Derivative of the activation, written as the derivative of g times a distribution function F: F + g F'."""
    if name == "silu":
        return torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    if name == "gelu":
        return torch.special.ndtr(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    z = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)          # (1 + tanh(z/2)) / 2 = sigmoid(z)
    return torch.sigmoid(z) + g * torch.sigmoid(z) * torch.sigmoid(-z) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g * g)


def _value(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return g * torch.special.ndtr(g)
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def exact(case, seed):
    st = prepare(case, seed)
    c, f64 = st["case"], torch.float64
    E, x = max(c["E"], 1), st["x"]
    ends = st["offsets"].cpu().numpy() if c["E"] else [0, x.shape[0]]

    def zeros(*shape):
        return torch.zeros(*shape, dtype=f64, device="cuda")

    if c["op"] == "gated":
        d, I = c["d"], c["I"]
        wg, wu = st["w_gate"].view(E, I, d), st["w_up"].view(E, I, d)
        h, dx = zeros(x.shape[0], I), zeros(*x.shape) if c["grad"] else None
        dwg, dwu = (zeros(E, I, d), zeros(E, I, d)) if c["grad"] else (None, None)
        for e in range(E):
            rows = slice(int(ends[e]), int(ends[e + 1]))
            if rows.start == rows.stop:
                continue
            xe, g64, u64 = x[rows].to(f64), wg[e].to(f64), wu[e].to(f64)
            g, u = torch.mm(g64, xe.t()), torch.mm(u64, xe.t())              # [I][rows]
            h[rows] = (_value(c["act"], g) * u).t()
            if c["grad"]:
                dh = st["dh"][rows].to(f64).t()
                dg, du = _slope(c["act"], g) * u * dh, _value(c["act"], g) * dh
                dwg[e], dwu[e] = torch.mm(dg, xe), torch.mm(du, xe)
                dx[rows] = torch.mm(dg.t(), g64) + torch.mm(du.t(), u64)
        if not c["grad"]:
            return {"h": h}
        return {"h": h, "dx": dx, "dw_gate": dwg.view(st["w_gate"].shape), "dw_up": dwu.view(st["w_up"].shape)}
    n_in, n_out = c["n_in"], c["n_out"]
    w, y = st["w"].view(E, n_out, n_in), zeros(x.shape[0], n_out)
    if c["op"] == "linear":
        dx, dw = (zeros(*x.shape), zeros(E, n_out, n_in)) if c["grad"] else (None, None)
        for e in range(E):
            rows = slice(int(ends[e]), int(ends[e + 1]))
            if rows.start == rows.stop:
                continue
            xe, we = x[rows].to(f64), w[e].to(f64)
            y[rows] = torch.mm(we, xe.t()).t()
            if c["grad"]:
                dy = st["dy"][rows].to(f64)
                dx[rows], dw[e] = torch.mm(we.t(), dy.t()).t(), torch.mm(xe.t(), dy).t()
        return {"y": y, "dx": dx, "dw": dw.view(st["w"].shape)} if c["grad"] else {"y": y}
    sw = st["w_scales"].to(f64).view(E, -(-n_out // BLOCK), -(-n_in // BLOCK))
    for j in range(0, n_in, BLOCK):                                  # block by block, as the scales are
        xb = x[:, j:j + BLOCK].to(f64)
        a = xb.abs().amax(1, keepdim=True).clamp_min(SMALLEST)
        q, s = _e4m3(xb * E4M3_MAX / a), a / E4M3_MAX
        for e in range(E):
            rows = slice(int(ends[e]), int(ends[e + 1]))
            if rows.start < rows.stop:
                col = sw[e, :, j // BLOCK].repeat_interleave(BLOCK)[:n_out]
                y[rows] += torch.mm(q[rows], w[e, :, j:j + BLOCK].to(f64).t()) * s[rows] * col
    return {"y": y}


# -------------------------------------------------------------------- work
def work(case):
    c = case
    N = (c["T"] - int(c["T"] * c["pad"])) * c["k"] if c["E"] else c["T"]          # rows with a matrix
    # matrices that they reach, chosen evenly
    mats = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"]) if c["E"] else 1
    if c["op"] == "gated":
        d, I = c["d"], c["I"]
        b, f = 2 * (mats * 2 * I * d + N * d + N * I), 4 * N * d * I
        if c["grad"]:
            b += 2 * (2 * max(c["E"], 1) * I * d + N * d + N * I)
            f *= 3
        return {"bytes": b, "flops": f}
    i, o = c["n_in"], c["n_out"]
    if c["op"] == "linear":
        b, f = 2 * (mats * i * o + N * i + N * o), 2 * N * i * o
        if c["grad"]:
            b += 2 * (max(c["E"], 1) * i * o + N * i + N * o)
            f *= 3
        return {"bytes": b, "flops": f}
    blocks = -(-i // BLOCK)
    return {"bytes": mats * (i * o + 4 * blocks * -(-o // BLOCK)) + 2 * N * i + 2 * N * o, "flops": 2 * N * i * o}
