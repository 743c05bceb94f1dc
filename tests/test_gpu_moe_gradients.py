"""What a training step's gradients are made of, beyond each call's own tests: the steps of the example's backward pass that are not
in test_gpu_moe_training.py (the weights' gradient, the codes of dY, the router, how the parts of the input's gradient
are put together), each from the values that the step had; and, in 64 bits and on the CPU, that those steps in that order are the
gradient of the block."""
import math

import numpy as np
import pytest
import torch

from tests import between_ref as B
from tests import operators_ref as R

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k,act", [(300, 512, 256, 8, 2, "silu"), (77, 256, 384, 5, 5, "gelu_tanh"), (1, 256, 128, 4, 1, "silu"), (500, 384, 128, 40, 3, "gelu")])
def test_the_steps_between(T, H, I, E, k, act):
    from examples.moe_block import Experts
    gen = lambda seed: torch.Generator(device=DEV).manual_seed(seed)  # noqa: E731
    block = Experts(H, I, E, k, act=act, seed=T + 1)
    block.norm.normal_(generator=gen(4)).mul_(0.2).add_(1)
    x = torch.randn(T, H, device=DEV, generator=gen(1)).bfloat16()
    dout = (torch.randn(T, H, device=DEV, generator=gen(2)) * 0.1).bfloat16()
    block.train_forward(x)
    block.backward(dout)
    s, b = block.saved, block.steps
    d, y = dout.double(), s["y"].double()
    # the weights' gradient: <Y[rows], dout>. 16 products, 2 halves, 5 exchanges and a running sum a piece, 8 warps
    want, mag = torch.zeros(T, k, dtype=torch.float64, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        terms = s["Y"][s["rows"][:, j].long()].double() * d
        want[:, j], mag[:, j] = terms.sum(1), terms.abs().sum(1)
    assert (s["rows"] >= 0).all() and ((b["dweights"].double() - want).abs() <= (23 * (H // 1024 + 1) + 8) * 2.0 ** -24 * mag).all()
    # the codes of dY in both directions, bit for bit
    for (q, sf), v in ((b["q"], b["dY"].double()), (b["qt"], B.columns(b["dY"].double()))):
        codes, scales = B.quantise(v)
        assert torch.equal(sf.double(), scales) and torch.equal(q.double(), codes)
    # the logits' gradient. The step's own is not kept: its product with y is the router's gradient, its product with the router a part
    # of dy. It is off by what test_gpu_route.py holds it to, 1e-5 of the row's largest dweight
    ids, dw = s["ids"].cpu().numpy().astype(np.int64), b["dweights"].double().cpu().numpy()
    dl = torch.from_numpy(R.route_backward(s["logits"].double().cpu().numpy(), ids, dw, "softmax", True, 1.0)).to(DEV)
    dl_off = 1e-5 * b["dweights"].double().abs().amax(1, keepdim=True).expand(T, E)
    # FP32 products with sums of T and of E terms
    want = dl.t() @ y
    assert ((block.drouter.double() - want).abs() <= dl_off.t() @ y.abs() + (T + 2) * 2.0 ** -24 * (dl.abs().t() @ y.abs()) + 1e-30).all()
    # dy: the sum of a token's rows, rounded to BF16, and the router's part, rounded again
    sums, mag = B.combine(b["dA"], s["rows"], None, None)
    part = dl @ block.router.double()
    off = dl_off @ block.router.double().abs() + (E + 2) * 2.0 ** -24 * (dl.abs() @ block.router.double().abs())
    want = sums + part
    bound = 2.0 ** -8 * (sums.abs() + want.abs()) * (1 + 2.0 ** -7) + (k + 4) * 2.0 ** -24 * mag + off * (1 + 2.0 ** -7) + 2.0 ** -133
    assert ((b["dy"].double() - want).abs() <= bound).all()
    assert k == 1 or (part.abs() > 2 * bound).any()                   # (it could not be left out; one renormalised weight has no gradient)


@pytest.mark.parametrize("T,H,I,E,k,act", [(7, 12, 10, 4, 2, "silu"), (5, 9, 8, 3, 3, "gelu"), (6, 8, 6, 5, 1, "gelu_tanh"), (9, 8, 4, 6, 3, "relu")])
def test_those_steps_are_the_blocks_gradient(T, H, I, E, k, act):
    """loss = <x + sum_j w_j W2[e_j] (act(g) u), dout> with (g; u) = W13[e_j] n, n = norm(x), w = router(n R^t): the steps against automatic
    differentiation, and against differences along a direction."""
    gen = torch.Generator().manual_seed(T)
    new = lambda *shape: torch.randn(*shape, generator=gen, dtype=torch.float64)  # noqa: E731
    x, norm, router, W13, W2, dout = new(T, H), 1 + 0.2 * new(H), new(E, H) / H ** 0.5, new(E, 2 * I, H) / H ** 0.5, new(E, H, I) / I ** 0.5, new(T, H)
    eps = 1e-6
    ids = (B.rmsnorm(x, norm, eps) @ router.t()).topk(k, 1).indices

    def activation(z):
        if act == "gelu":
            return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
        return B.act(z, act)

    def loss(x, norm, router, W13, W2):
        n = x / torch.sqrt(x.square().mean(1, keepdim=True) + eps) * norm
        score = torch.softmax(n @ router.t(), 1).gather(1, ids)
        w = score / score.sum(1, keepdim=True)
        z = torch.einsum("tkih,th->tki", W13[ids], n)
        y = torch.einsum("tkhi,tki->tkh", W2[ids], activation(z[..., :I]) * z[..., I:])
        return ((x + (w.unsqueeze(2) * y).sum(1)) * dout).sum()

    leaves = [t.clone().requires_grad_() for t in (x, norm, router, W13, W2)]
    auto = torch.autograd.grad(loss(*leaves), leaves)

    # the steps, as the example's backward pass takes them
    n = B.rmsnorm(x, norm, eps)
    logits = n @ router.t()
    w = torch.from_numpy(R.route_weights(logits.numpy(), ids.numpy(), "softmax", True, 1.0))
    g, u = torch.einsum("tkih,th->tki", W13[ids], n).split(I, 2)
    h = B.act(g, act) * u
    y = torch.einsum("tkhi,tki->tkh", W2[ids], h)
    dweights = (y * dout.unsqueeze(1)).sum(2)
    dY = w.unsqueeze(2) * dout.unsqueeze(1)
    dH = torch.einsum("tkhi,tkh->tki", W2[ids], dY)
    dz = torch.cat((dH * u * B.slope(g, act), dH * B.act(g, act)), 2)
    dW2, dW13 = torch.zeros_like(W2), torch.zeros_like(W13)
    for t in range(T):
        for j in range(k):
            dW2[ids[t, j]] += torch.outer(dY[t, j], h[t, j])
            dW13[ids[t, j]] += torch.outer(dz[t, j], n[t])
    dlogits = torch.from_numpy(R.route_backward(logits.numpy(), ids.numpy(), dweights.numpy(), "softmax", True, 1.0))
    dn = torch.einsum("tkih,tki->th", W13[ids], dz) + dlogits @ router
    dx, dnorm = B.rmsnorm_backward(dn, x, norm, eps, dout)
    steps = (dx, dnorm, dlogits.t() @ n, dW13, dW2)
    for name, a, got in zip(("x", "norm", "router", "W13", "W2"), auto, steps):
        torch.testing.assert_close(got, a, rtol=1e-9, atol=1e-9, msg=name)
    at = (x, norm, router, W13, W2)
    for i, got in enumerate(steps):
        v, step = new(*got.shape), 1e-6
        move = lambda s: [t + s * v if j == i else t for j, t in enumerate(at)]  # noqa: E731
        along = float(loss(*move(step)) - loss(*move(-step))) / (2 * step)
        assert abs(along - float((got * v).sum())) <= 1e-6 * (1 + abs(along))
