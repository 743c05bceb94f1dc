"""The example's block of experts keeps its quantised weights in one place: a captured pass reads them by their addresses, so an
update must write them there."""
import pytest
import torch

from examples.moe_block import Experts

NAMES = ("W13", "s13", "W13t", "s13t", "W2", "s2", "W2t", "s2t", "norm", "router")


def test_an_update_keeps_the_weights_where_they_are():
    block = Experts(256, 128, 3, 2, device="cpu")
    at = {n: getattr(block, n).data_ptr() for n in NAMES}
    for name in ("norm", "router", "master13", "master2"):
        setattr(block, "d" + name, torch.randn(getattr(block, name).shape, generator=torch.Generator().manual_seed(len(name))))
    block.step(0.1)
    assert {n: getattr(block, n).data_ptr() for n in NAMES} == at
    # and they are those of the new master weights
    other = Experts(256, 128, 3, 2, device="cpu")
    for name in ("master13", "master2"):
        setattr(other, name, getattr(block, name).clone())
    other.weights = None
    other.update()
    for n in NAMES[:8]:
        assert torch.equal(getattr(block, n).view(torch.uint8), getattr(other, n).view(torch.uint8)), n


@pytest.mark.gpu
def test_a_captured_pass_follows_the_training_steps():
    block = Experts(512, 256, 16, 4, seed=3)
    x, out, g = block.graph(200)
    x.copy_(torch.randn(200, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)))
    g.replay()
    before = out.clone()
    for _ in range(2):
        y = block.train_forward(x.clone())
        block.backward((y.float() / 200).bfloat16())
        block.step(0.5)
    g.replay()
    after = out.clone()
    assert torch.equal(after, block.train_forward(x.clone()))
    assert not torch.equal(after, before)
    # the graph keeps what it reads
    del block
    junk = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(64)]
    g.replay()
    assert torch.equal(out, after) and len(junk) == 64
