"""The example block: its steps against plain 64-bit forms of the same quantised operands."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import operators_ref as ref

pytestmark = pytest.mark.gpu


def _scaled(q, s, rows):
    """Codes times their scales, float64; rows: 1 (1x128) or 128 (128x128 blocks)."""
    s = s.double().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(128, 1)
    return q.view(torch.float8_e4m3fn).double() * s


@pytest.mark.parametrize("T", [1, 5, 64])
def test_decode_step_and_its_graph(T):
    from examples.moe_block import Block, quantise
    block = Block(512, 256, 16, 4, seed=3)
    x, out, g = block.graph(T)
    x.copy_(torch.randn(T, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)))
    g.replay()
    eager = block.decode(x)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    # the dense layer at the end, from the experts' output that the operators give
    ids = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 4, device="cuda")
    dg.dg_moe_route(x @ block.router.t(), ids, w)
    h = torch.empty_like(x)
    dg.dg_moe_layer(x, ids, w, block.W13, block.s13, block.W2, block.s2, h, block.workspace, residual=x)
    q, s = quantise(h)
    a, b = _scaled(q, s, 1), _scaled(block.W, block.s, 128)
    z = a @ b.t() + block.bias.double()
    want = z * 0.5 * (1 + torch.erf(z / 2 ** 0.5)) + h.double()
    # FP32 sums of 512 products: 2^-24 each of the absolute sum; the activation's slope is below 1.13; one BF16
    # rounding of the output
    bound = 1.13 * 520 * 2.0 ** -24 * (a.abs() @ b.abs().t() + block.bias.double().abs()) + 2.0 ** -20 * z.abs()
    bound += 2.0 ** -8 * want.abs() + 2.0 ** -30
    assert ((out.double() - want).abs() <= bound).all()
    # and the weights are a softmax over the chosen experts
    logits = (x @ block.router.t()).double()
    top = logits.gather(1, ids.long())
    assert (top.amin(1) >= logits.scatter(1, ids.long(), float("-inf")).amax(1)).all()
    assert ((w.double() - torch.softmax(top, 1)).abs() <= 1e-5).all()
    assert dg.dg_device_status() == 0


@pytest.mark.parametrize("tokens", [128, 77])
def test_dense_layer_gradients(tokens):
    """dx, dW and dbias against float64 autograd of act(W x + b) + x. Each of a product's two operands is off by
    at most a relative 2^-4 (e4m3 rounding, with 2^-8 more for the arithmetic before it) plus half the
    quantisation's smallest step; dx is rounded to BF16 twice."""
    from examples.moe_block import Dense
    layer = Dense(256, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    layer.bias.normal_(generator=gen)
    x = torch.randn(tokens, 256, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(tokens, 256, device="cuda", generator=gen).bfloat16()
    layer.forward(x)
    dx = layer.backward(dy)
    W = _scaled(layer.W, layer.s, 128)
    z = layer.Z.double().requires_grad_(True)
    a = torch.nn.functional.gelu(z, approximate="tanh")
    a.backward(dy.double())
    dz = z.grad
    d = 2.0 ** -4 + 2.0 ** -8
    step = lambda v: 2.0 ** -10 / 448 * v.abs().max()      # half the smallest code step at the largest scale
    zabs = dz.abs() * (1 + d) + step(dz)
    want = dz @ W + dy.double()
    bound = (d * dz.abs() + step(dz)) @ W.abs() + 2.0 ** -7 * (zabs @ W.abs() + dy.double().abs())
    assert ((dx.double() - want).abs() <= bound).all()
    xd = x.double()
    want = dz.t() @ xd
    bound = zabs.t() @ (xd.abs() * (1 + d) + step(xd)) - dz.abs().t() @ xd.abs() + 2.0 ** -12 * (zabs.t() @ xd.abs())
    assert ((layer.dW.double() - want).abs() <= bound).all()
    assert ((layer.dbias.double() - dz.sum(0)).abs() <= 2.0 ** -16 * (dz.abs() + dy.double().abs()).sum(0)).all()


def test_both_learn():
    from examples.moe_block import train_dense, train_router
    losses = train_dense(H=256, tokens=200, steps=40)
    assert losses[-1] < 0.25 * losses[0]
    means = train_router(steps=40)
    assert means[-1] > means[0] + 0.1
