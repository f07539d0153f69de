"""The operators around the routed experts, measured.

Each case is one pass through one operator of the package: token rows sorted by
expert and back (with the routing weights applied, and the gradients of both),
products of activations with 4-bit group-quantised weights (one matrix, and one
matrix per expert over sorted rows), and the gradient of the router.  Where
``own`` is false ``run`` computes them in plain torch operations in 32 bits;
where it is true it calls the package.  ``exact`` is the definition in 64 bits.

Shapes are those of the package's own workloads (hidden size 2048, 512 or 256
experts of intermediate size 512, 10 or 8 a token, 1 to 4096 tokens) and
generic ones around them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token handed to expert products outside the fused layer
        dict(name="sort_step", op="sort", T=1, k=10, E=512, d=2048, dtype="bf16", pad=0.0, grad=False),
        # a batch of odd size and odd row length whose last tokens are padding, with its gradient
        dict(name="sort_ragged", op="sort", T=777, k=8, E=256, d=1001, dtype="f16", pad=0.1, grad=True),
        # a prompt, forward and gradient, as a training step takes it
        dict(name="sort_prefill", op="sort", T=4096, k=10, E=512, d=2048, dtype="bf16", pad=0.0, grad=True),
        # four decoded tokens' expert outputs in 32 bits brought together with the shared expert's
        dict(name="back_step", op="back", T=4, k=10, E=512, d=2048, dtype="f32", pad=0.0, shared=True, grad=False),
        # a prompt's expert outputs brought together, and the gradients of rows, weights and shared expert
        dict(name="back_prefill", op="back", T=4096, k=10, E=512, d=2048, dtype="bf16", pad=0.0, shared=True,
             grad=True),
        # one token through one dense projection of the resident core: latency
        dict(name="linear_token", op="linear", T=1, n_in=2048, n_out=2048, group=64),
        # one token through an output projection over a vocabulary of odd size: bandwidth
        dict(name="linear_vocab", op="linear", T=1, n_in=2048, n_out=100003, group=64),
        # a batch of decoded tokens through a square projection with wide groups
        dict(name="linear_batch", op="linear", T=48, n_in=4096, n_out=4096, group=128),
        # one token through the first matrix of each of its experts
        dict(name="experts_step", op="experts", T=1, k=10, E=512, n_in=2048, n_out=512, group=64),
        # 64 tokens through the last matrix of their experts
        dict(name="experts_batch", op="experts", T=64, k=8, E=256, n_in=512, n_out=2048, group=64),
        # the router's gradient of a small batch
        dict(name="router_batch", op="router", T=64, k=8, E=256, d=2048),
        # and of a prompt
        dict(name="router_prefill", op="router", T=4096, k=10, E=512, d=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "back", "linear", "experts", "router"])
    k, E = rng.choice([(1, 8), (2, 16), (6, 64), (8, 256), (10, 512)])
    if op in ("sort", "back"):
        d = rng.choice([64 * rng.randint(1, 48), rng.randint(33, 2500)])
        t = rng.choice(["bf16", "f16", "f32"])
        c = dict(op=op, T=_log(rng, 1, min(4096, 4096 * 10 * 2048 * 2 // (k * d * SIZE[t]))), k=k, E=E, d=d, dtype=t,
                 pad=rng.choice([0.0, 0.0, 0.25]), grad=rng.random() < 0.5)
        if op == "back":
            c["shared"] = rng.random() < 0.5
        return c
    if op == "linear":
        group = rng.choice([32, 64, 64, 128])
        n_in = group * max(1, _log(rng, 256, 8192) // group)
        return dict(op=op, T=_log(rng, 1, 64), n_in=n_in, n_out=_log(rng, 64, 16384), group=group)
    if op == "experts":
        group = rng.choice([32, 64, 64, 128])
        n_in = group * max(1, _log(rng, 256, 2048) // group)
        n_out = _log(rng, 64, min(2048, (1 << 29) // (E * n_in)))
        T = _log(rng, 1, min(96, (1 << 29) // (k * n_in * n_out)))
        return dict(op=op, T=T, k=k, E=E, n_in=n_in, n_out=n_out, group=group)
    return dict(op=op, T=_log(rng, 1, 4096), k=k, E=E, d=64 * rng.randint(2, 32))


# ------------------------------------------------------------------ inputs
def _kept(c):
    return c["T"] - int(c["T"] * c.get("pad", 0.0))


def _routing(c, g):
    """topk_idx, topk_w as a router with a mild Zipf preference gives them; the
    padded tokens at the end carry expert -1."""
    T, E, k = c["T"], c["E"], c["k"]
    pop = torch.randperm(E, generator=g, device="cuda").float() + 1.0
    logits = 0.9 * torch.randn(T, E, generator=g, device="cuda") - 0.165 * pop.log()
    top, idx = logits.topk(k, dim=1)
    w = torch.softmax(top, 1)
    idx = idx.to(torch.int32)
    idx[_kept(c):] = -1
    return idx.contiguous(), w.contiguous()


def _bucket(idx, E):
    """Stable order of the pairs by expert, the bucket borders and each pair's row (-1: no expert)."""
    key = idx.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    order = torch.sort(key, stable=True).indices
    n = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).index_add_(0, key, torch.ones_like(key))
    ends = n.cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends[:E]])
    row = torch.empty_like(order)
    row[order] = torch.arange(key.numel(), device=idx.device)
    row = torch.where(key < E, row, torch.full_like(row, -1))
    at = torch.arange(key.numel(), device=idx.device)
    pairs = torch.where(at < offsets[E], order, torch.full_like(order, -1))
    return offsets.to(torch.int32), pairs.to(torch.int32), row.to(torch.int32).view(idx.shape)


def _weights(lead, n_in, n_out, group, g):
    """Random 4-bit matrices in the package's layout: codes [in/32][out][16 B], then (scale, bias) fp16
    [in/group][out][2]; scales in 0.002 to 0.02, bias -8 scales and some."""
    codes = torch.randint(0, 256, (lead, n_in * n_out // 2), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.empty(lead, n_in // group, n_out, device="cuda").uniform_(0.002, 0.02, generator=g)
    b = -8.0 * s * torch.empty_like(s).uniform_(0.9, 1.1, generator=g)
    sb = torch.stack([s, b], -1).half().view(lead, -1).view(torch.uint8)
    return torch.cat([codes, sb], 1).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}

    def randn(*shape, dtype="f32"):
        return torch.randn(*shape, generator=g, device="cuda").to(DTYPES[dtype])

    if c["op"] in ("sort", "back"):
        T, k, d, t = c["T"], c["k"], c["d"], c["dtype"]
        st["idx"], st["w"] = _routing(c, g)
        n = T * k
        # buffers that a program keeps from step to step; rows behind the last bucket keep what they hold
        st["rows_out"] = torch.zeros(n, d, dtype=DTYPES[t], device="cuda")
        st["y_out"] = torch.empty(T, d, dtype=DTYPES[t], device="cuda")
        if c["op"] == "sort":
            st["x"] = randn(T, d, dtype=t)
            st["drows"] = randn(n, d, dtype=t)
            st["offsets"] = torch.empty(c["E"] + 1, dtype=torch.int32, device="cuda")
            st["pairs"] = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            st["row_of"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            st["ws"] = torch.zeros((c["E"] + 8) * (n // 64 + 8) * 4 + 65536, dtype=torch.uint8, device="cuda")
        else:
            st["row_of"] = _bucket(st["idx"], c["E"])[2]
            st["rows"] = randn(n, d, dtype=t)
            st["dy"] = randn(T, d, dtype=t)
            st["sh"] = randn(T, d, dtype=t) if c["shared"] else None
            st["sg"] = torch.sigmoid(randn(T)) if c["shared"] else None
            st["dw_out"] = torch.empty(T, k, device="cuda")
            st["dsh_out"] = torch.empty_like(st["dy"]) if c["shared"] else None
            st["dsg_out"] = torch.empty(T, device="cuda") if c["shared"] else None
    elif c["op"] == "linear":
        st["w"] = _weights(1, c["n_in"], c["n_out"], c["group"], g)[0]
        st["x"] = randn(c["T"], c["n_in"], dtype="bf16")
        st["y_out"] = torch.empty(c["T"], c["n_out"], device="cuda")
    elif c["op"] == "experts":
        E, n = c["E"], c["T"] * c["k"]
        st["w"] = _weights(E, c["n_in"], c["n_out"], c["group"], g)
        st["slots"] = torch.randperm(E, generator=g, device="cuda").to(torch.int32)
        idx, _ = _routing(c, g)
        st["offsets"], pairs, _ = _bucket(idx, E)
        x = randn(c["T"], c["n_in"], dtype="bf16")
        st["x"] = x[pairs.long() // c["k"]].contiguous()
        st["y_out"] = torch.empty(n, c["n_out"], device="cuda")
    else:
        T, k, E, d = c["T"], c["k"], c["E"], c["d"]
        st["x"] = randn(T, d, dtype="bf16")
        st["wr"] = 0.02 * randn(E + 1, d)
        st["idx"], st["w"] = _routing(c, g)
        st["sg"] = torch.sigmoid(randn(T))
        st["dw"], st["dsg"] = randn(T, k), randn(T)
        st["offsets"], st["pairs"], _ = _bucket(st["idx"], E)
        st["out"] = (torch.empty(T, d, device="cuda"), torch.empty(E + 1, d, device="cuda"),
                     torch.empty(E, device="cuda"))
        st["ws"] = torch.zeros(4 * T * (k + 2) + 4 * d * (T * (k + 1) // 16 + 64) + 65536, dtype=torch.uint8,
                               device="cuda")
    return st


# ------------------------------------------------------- the package's own
def _run_own(st):
    import sparse_moe_decode_router_amd as moe
    c = st["case"]
    if c["op"] == "sort":
        rows, offsets, pairs, row_of = moe.moe_sort_tokens(
            st["x"], st["idx"], c["E"], workspace=st["ws"],
            out=(st["rows_out"], st["offsets"], st["pairs"], st["row_of"]))
        got = {"rows": rows, "offsets": offsets, "pairs": pairs, "row_of": row_of}
        if c["grad"]:
            got["dx"] = moe.moe_sort_tokens_backward(st["drows"], row_of, out=st["y_out"])
        return got
    if c["op"] == "back":
        got = {"y": moe.moe_unsort_combine(st["rows"], st["row_of"], st["w"], st["sh"], st["sg"], out=st["y_out"])}
        if c["grad"]:
            got["drows"], got["dw"], dsh, dsg = moe.moe_unsort_combine_backward(
                st["dy"], st["rows"], st["row_of"], st["w"], st["sh"], st["sg"],
                out=(st["rows_out"], st["dw_out"], st["dsh_out"], st["dsg_out"]))
            if c["shared"]:
                got["dshared"], got["dgate"] = dsh, dsg
        return got
    if c["op"] == "linear":
        return moe.moe_linear_int4(st["w"], st["x"], c["n_out"], group=c["group"], out=st["y_out"])
    if c["op"] == "experts":
        return moe.moe_expert_linear_int4(st["w"], st["slots"], st["x"], st["offsets"], c["n_out"],
                                          group=c["group"], out=st["y_out"])
    dx, dwr, dbias = moe.moe_router_topk_backward(
        st["x"], st["wr"], st["idx"], st["w"], st["sg"], st["dw"], st["dsg"], st["offsets"], st["pairs"],
        workspace=st["ws"], out=st["out"])
    return {"dx": dx, "dw_router": dwr, "dbias": dbias}


# -------------------------------------------------------------- plain form
def _dequant(w, n_in, n_out, group):
    """fp32 [..., out, in] of matrices in the package's layout."""
    lead, nb = w.shape[:-1], n_in * n_out // 2
    byte = w[..., :nb].reshape(*lead, n_in // 32, n_out, 16)
    q = torch.stack([byte & 15, byte >> 4], -1).reshape(*lead, n_in // 32, n_out, 32).movedim(-3, -2)
    q = q.reshape(*lead, n_out, n_in // group, group).float()
    sb = w[..., nb:].contiguous().view(torch.float16).reshape(*lead, n_in // group, n_out, 2).float()
    s, b = sb[..., 0].movedim(-2, -1).unsqueeze(-1), sb[..., 1].movedim(-2, -1).unsqueeze(-1)
    return (s * q + b).reshape(*lead, n_out, n_in)


def _gather(rows, row_of):
    """fp32 [T][k][d] of the sorted rows of each token's pairs, zero where a pair has none."""
    return torch.where((row_of >= 0).unsqueeze(-1), rows[row_of.clamp_min(0).long()].float(), 0.0)


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    if c["op"] == "sort":
        offsets, pairs, row_of = _bucket(st["idx"], c["E"])
        rows = torch.where((pairs >= 0).unsqueeze(1), st["x"][pairs.clamp_min(0).long() // c["k"]],
                           torch.zeros((), dtype=st["x"].dtype, device="cuda"))
        got = {"rows": rows, "offsets": offsets, "pairs": pairs, "row_of": row_of}
        if c["grad"]:
            got["dx"] = _gather(st["drows"], row_of).sum(1).to(st["x"].dtype)
        return got
    if c["op"] == "back":
        t, live = st["rows"].dtype, st["row_of"] >= 0
        w = torch.where(live, st["w"], 0.0)
        y = (w.unsqueeze(-1) * _gather(st["rows"], st["row_of"])).sum(1)
        if c["shared"]:
            y = y + st["sg"].unsqueeze(1) * st["sh"].float()
        got = {"y": y.to(t)}
        if c["grad"]:
            dy = st["dy"].float()
            drows = torch.zeros_like(st["rows"])
            drows[st["row_of"][live].long()] = (w.unsqueeze(-1) * dy.unsqueeze(1))[live].to(t)
            got["drows"] = drows
            got["dw"] = (_gather(st["rows"], st["row_of"]) * dy.unsqueeze(1)).sum(2)
            if c["shared"]:
                got["dshared"] = (st["sg"].unsqueeze(1) * dy).to(t)
                got["dgate"] = (dy * st["sh"].float()).sum(1)
        return got
    if c["op"] == "linear":
        return st["x"].float() @ _dequant(st["w"], c["n_in"], c["n_out"], c["group"]).t()
    if c["op"] == "experts":
        n = st["x"].shape[0]
        e = (torch.arange(n, device="cuda").unsqueeze(1) >= st["offsets"][1:].unsqueeze(0)).sum(1)
        w = _dequant(st["w"][st["slots"][e].long()], c["n_in"], c["n_out"], c["group"])
        return (w @ st["x"].float().unsqueeze(-1)).squeeze(-1)
    w, dw, E = st["w"], st["dw"], c["E"]
    dl = torch.zeros(c["T"], E + 1, device="cuda")
    dl.scatter_(1, st["idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    dl[:, E] = st["dsg"] * st["sg"] * (1.0 - st["sg"])
    return {"dx": dl @ st["wr"], "dw_router": dl.t() @ st["x"].float(), "dbias": dl[:, :E].sum(0)}


# ----------------------------------------------------- definition, 64 bits
def _exact_product(w, x, n_in, n_out, group):
    """sum over groups of scale * (codes . x) + bias * sum(x), one matrix [bytes] on rows x [n][in]."""
    nb, n = n_in * n_out // 2, x.shape[0]
    sb = w[nb:].view(torch.float16).double().reshape(n_in // group, n_out, 2)
    y = x.new_zeros(n, n_out)
    for a in range(0, n_in, 128 if group == 128 else 64):
        m = min(n_in, a + (128 if group == 128 else 64)) - a
        byte = w[a * n_out // 2:(a + m) * n_out // 2].reshape(m // 32, n_out, 16)
        for h in range(2):
            nib = ((byte >> (4 * h)) & 15).double()                    # inputs a + 32 c + 2 b + h
            xs = x[:, a:a + m].reshape(n, m // 32, 16, 2)[..., h]
            for q in range(m // 32):
                gi = (a + 32 * q) // group
                y += (xs[:, q] @ nib[q].t()) * sb[gi, :, 0] + xs[:, q].sum(1, keepdim=True) * sb[gi, :, 1]
    return y


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "sort":
        T, k, E = c["T"], c["k"], c["E"]
        idx = st["idx"].cpu().reshape(-1).tolist()
        buckets = [[] for _ in range(E)]
        for i, e in enumerate(idx):
            if 0 <= e < E:
                buckets[e].append(i)
        pairs = [i for b in buckets for i in b]
        offsets = [0]
        for b in buckets:
            offsets.append(offsets[-1] + len(b))
        row_of = [-1] * (T * k)
        for p, i in enumerate(pairs):
            row_of[i] = p
        rows = torch.zeros(T * k, c["d"], dtype=torch.float64, device="cuda")
        if pairs:
            rows[:len(pairs)] = st["x"].double()[torch.tensor(pairs, device="cuda") // k]
        got = {"rows": rows, "offsets": torch.tensor(offsets, dtype=torch.int32),
               "pairs": torch.tensor(pairs + [-1] * (T * k - len(pairs)), dtype=torch.int32),
               "row_of": torch.tensor(row_of, dtype=torch.int32).view(T, k)}
        if c["grad"]:
            dx = torch.zeros(T, c["d"], dtype=torch.float64, device="cuda")
            if pairs:
                dx.index_add_(0, torch.tensor(pairs, device="cuda") // k, st["drows"][:len(pairs)].double())
            got["dx"] = dx
        return got
    if c["op"] == "back":
        T, k, d = c["T"], c["k"], c["d"]
        y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        drows = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        dy = st["dy"].double()
        for r in range(k):
            t = torch.nonzero(st["row_of"][:, r] >= 0).squeeze(1)
            p = st["row_of"][t, r].long()
            o, w = st["rows"][p].double(), st["w"][t, r].double().unsqueeze(1)
            y[t] += w * o
            drows[p] = w * dy[t]
            dw[t, r] = (dy[t] * o).sum(1)
        if c["shared"]:
            y += st["sg"].double().unsqueeze(1) * st["sh"].double()
        got = {"y": y}
        if c["grad"]:
            got.update(drows=drows, dw=dw)
            if c["shared"]:
                got.update(dshared=st["sg"].double().unsqueeze(1) * dy, dgate=(dy * st["sh"].double()).sum(1))
        return got
    if c["op"] == "linear":
        return _exact_product(st["w"], st["x"].double(), c["n_in"], c["n_out"], c["group"])
    if c["op"] == "experts":
        x, off, slots = st["x"].double(), st["offsets"].tolist(), st["slots"].tolist()
        y = torch.zeros(x.shape[0], c["n_out"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            if off[e + 1] > off[e]:
                y[off[e]:off[e + 1]] = _exact_product(st["w"][slots[e]], x[off[e]:off[e + 1]], c["n_in"],
                                                      c["n_out"], c["group"])
        return y
    T, k, E, d = c["T"], c["k"], c["E"], c["d"]
    w, dw, wr, x = st["w"].double(), st["dw"].double(), st["wr"].double(), st["x"].double()
    jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)           # of a softmax over the chosen logits
    gl = torch.matmul(jac, dw.unsqueeze(2)).squeeze(2)
    s = st["sg"].double()
    gs = st["dsg"].double() * (s - s * s)
    dx = gs.unsqueeze(1) * wr[E]
    dwr = torch.zeros(E + 1, d, dtype=torch.float64, device="cuda")
    db = torch.zeros(E, dtype=torch.float64, device="cuda")
    for r in range(k):
        e = st["idx"][:, r].long()
        dx += gl[:, r:r + 1] * wr[e]
        dwr.index_add_(0, e, gl[:, r:r + 1] * x)
        db.index_add_(0, e, gl[:, r])
    dwr[E] = (gs.unsqueeze(1) * x).sum(0)
    return {"dx": dx, "dw_router": dwr, "dbias": db}


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("sort", "back"):
        T, k, d, s = c["T"], c["k"], c["d"], SIZE[c["dtype"]]
        n, m, t = T * k, _kept(c) * k, _kept(c)                 # pairs, pairs with an expert, tokens with one
        if c["op"] == "sort":
            b = t * d * s + m * d * s + 4 * (3 * n + c["E"] + 1)
            f = 0
            if c["grad"]:
                b, f = b + m * d * s + T * d * s, m * d
            return {"bytes": b, "flops": f}
        sh = T * d * s + 4 * T if c["shared"] else 0
        b, f = m * d * s + 8 * n + sh + T * d * s, 2 * (m + (T if c["shared"] else 0)) * d
        if c["grad"]:
            b, f = b + T * d * s + m * d * s + 4 * n + sh, f + 3 * (m + (T if c["shared"] else 0)) * d
        return {"bytes": b, "flops": f}
    if c["op"] in ("linear", "experts"):
        one = c["n_in"] * c["n_out"] // 2 + c["n_in"] // c["group"] * c["n_out"] * 4
        rows = c["T"] * c.get("k", 1)
        # experts that T tokens of k each reach, chosen evenly
        mats = 1.0 if c["op"] == "linear" else c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])
        return {"bytes": mats * one + rows * (2 * c["n_in"] + 4 * c["n_out"]), "flops": 2 * rows * c["n_in"] * c["n_out"]}
    T, k, E, d = c["T"], c["k"], c["E"], c["d"]
    return {"bytes": 2 * T * d + 4 * (E + 1) * d + 4 * T * (4 * k + 2) + 4 * T * d + 4 * (E + 1) * d + 4 * E,
            "flops": 4 * T * (k + 1) * d}
