"""The experts' products inside a torch.autograd.Function, as a model trains with
them: the layer from the sort to the combined rows, its parameters leaves, against
the same calls made by hand (bit for bit; test_gpu_product_calls.py has those
against fp64) and against torch's own gradients of the formula in fp64."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_decode_router_amd")

BF16, F32 = torch.bfloat16, torch.float32


class Experts(torch.autograd.Function):
    """y[t] = sum_r w[t, r] W_d (silu(W_g x) W_u x) over the experts idx[t]."""

    @staticmethod
    def forward(ctx, x, w, wg, wu, wd, idx):
        X, off, _, row_of = moe.moe_sort_tokens(x, idx, wg.shape[0])
        h, pre = moe.moe_gated(wg, wu, X, off, save=True)
        Y = moe.moe_linear(wd, h, off)
        ctx.save_for_backward(w, wg, wu, wd, X, off, row_of, h, pre, Y)
        return moe.moe_unsort_combine(Y, row_of, w)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        w, wg, wu, wd, X, off, row_of, h, pre, Y = ctx.saved_tensors
        dY, dw, _, _ = moe.moe_unsort_combine_backward(dy.contiguous(), Y, row_of, w)
        dh, dwd = moe.moe_linear_backward(dY, wd, h, off)
        dX, dwg, dwu = moe.moe_gated_backward(dh, pre, wg, wu, X, off)
        return moe.moe_sort_tokens_backward(dX, row_of), dw, dwg, dwu, dwd, None


def _leaves(T=40, k=3, E=6, d=72, I=40):
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    leaves = [r(T, d).to(BF16), torch.softmax(r(T, k), 1), (r(E, I, d) / math.sqrt(d)).to(BF16),
              (r(E, I, d) / math.sqrt(d)).to(BF16), (r(E, d, I) / math.sqrt(I)).to(BF16)]
    return [v.requires_grad_() for v in leaves], idx, r(T, d).to(BF16)


def _formula(leaves, idx):
    x, w, wg, wu, wd = [v.detach().double().requires_grad_() for v in leaves]
    y = 0
    for r in range(idx.shape[1]):
        e = idx[:, r].long()
        g, u = ((m[e] * x.unsqueeze(1)).sum(2) for m in (wg, wu))
        y = y + w[:, r:r + 1] * (wd[e] * (torch.nn.functional.silu(g) * u).unsqueeze(1)).sum(2)
    return y, [x, w, wg, wu, wd]


def test_a_layer_as_an_autograd_function():
    leaves, idx, dy = _leaves()
    y = Experts.apply(*leaves, idx)
    assert y.requires_grad and y.grad_fn is not None
    grads = torch.autograd.grad(y, leaves, dy)

    class Ctx:                                                    # the same calls by hand
        def save_for_backward(self, *v):
            self.saved_tensors = v
    ctx = Ctx()
    with torch.no_grad():
        again = Experts.forward(ctx, *(v.detach() for v in leaves), idx)
        by_hand = Experts.backward(ctx, dy)
    assert torch.equal(again, y)
    for a, b in zip(grads, by_hand):
        assert torch.equal(a, b)
    want, exact = _formula(leaves, idx)
    for a, b in zip((y, *grads), (want, *torch.autograd.grad(want, exact, dy.double()))):
        # roundings to bfloat16 (2^-8 each) along the way: up to seven of them (h, Y, dY, dh, dg, the rows and the
        # sum), of random sign in sums of many: in norm below seven times one
        assert torch.linalg.norm(a.double() - b) < 7 * 2.0 ** -8 * torch.linalg.norm(b)


def test_gradients_accumulate_over_two_backward_passes_and_through_other_operations():
    leaves, idx, dy = _leaves()
    (Experts.apply(*leaves, idx) * dy).sum().backward()
    once = [v.grad.clone() for v in leaves]
    (Experts.apply(*leaves, idx) * dy).sum().backward()
    for v, g in zip(leaves, once):
        assert torch.equal(v.grad, g + g)
    for v in leaves:
        v.grad = None
    Experts.apply(*leaves, idx).sum().backward()                  # an expanded gradient: made contiguous above
    assert all(torch.isfinite(v.grad).all() for v in leaves)


def test_outside_of_a_function_it_is_refused():
    (x, w, wg, wu, wd), idx, dy = _leaves()
    for call in (lambda: moe.moe_linear(wd[0], dy[:, :40].contiguous()), lambda: moe.moe_gated(wg[0], wu[0], x)):
        with pytest.raises(ValueError):
            call()
        with torch.no_grad():
            call()
