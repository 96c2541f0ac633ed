"""GPU: a DiT block of quantized linears and the operators between them, as a
whole: it trains its adapters, two runs give the same bits, and the samples of
a batch do not touch."""
import pytest
import torch

from bit_quantized_amd import dit

from _gpu import DEV, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_block_trains(state):
    say("dit block", state)
    a = dit.train(steps=12, width=256, rank=8, state=state, say=None)
    assert a[-1] < 0.5 * a[0], a
    assert a == dit.train(steps=12, width=256, rank=8, state=state, say=None)


def test_samples_do_not_touch():
    """A sample's rows come out the same bits whatever the other sample holds."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    block = dit.DiTBlock(256, 4, [16, 24, 24], dit.quantized_linears(8, gen, DEV))
    pos = torch.cat([dit.grid_positions(8, 6, 6, DEV), dit.grid_positions(4, 5, 7, DEV)])
    seg = torch.tensor([0, 44, 83], dtype=torch.int32, device=DEV)
    x = torch.randn(83, 256, generator=gen, device=DEV).to(torch.bfloat16)
    cond = torch.randn(2, 256, generator=gen, device=DEV).to(torch.bfloat16)
    with torch.no_grad():
        a = block(x, cond, pos, seg)
        x2, cond2 = x.clone(), cond.clone()
        x2[44:], cond2[1] = -x2[44:], 3.0
        b = block(x2, cond2, pos, seg)
    assert torch.equal(a[:44], b[:44]) and not torch.equal(a[44:], b[44:])
