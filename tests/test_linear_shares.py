"""Prefill with more tiles than SMs: blocks that store a slot and then receive a state,
receive one and hand it on, or hand one on before they receive one, against the float64
oracle within the bounds of test_linear_attention.py. test_linear_schedule.py counts on the
CPU which of these the cases reach.
"""
import pytest
import torch

from test_linear_attention import call, draw, run_and_check
from test_linear_schedule import CHAINS, SKEWED

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,lengths", SKEWED, ids=lambda v: str(v) if isinstance(v, tuple) else "")
def test_one_long_item_among_short_ones(shape, lengths):
    run_and_check(draw(*shape, seed=21, lengths=lengths), "prefill")


@pytest.mark.parametrize("shape,lengths", CHAINS, ids=lambda v: str(v) if isinstance(v, tuple) else "")
def test_slightly_more_tiles_than_sms(shape, lengths):
    run_and_check(draw(*shape, seed=22, lengths=lengths), "prefill")


@pytest.mark.parametrize("shape,lengths", SKEWED[:2] + CHAINS,
                         ids=lambda v: str(v) if isinstance(v, tuple) else "")
def test_shares_repeat(shape, lengths):
    """The same bits every time, other work on the GPU or not."""
    x = draw(*shape, seed=23, lengths=lengths, device="cuda")
    want = call(dict(x, state_pool=x["state_pool"].clone()), "prefill")
    noise = torch.randn(1 << 26, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(12):
        if k % 2:  # copies that keep the memory busy beside the call
            with torch.cuda.stream(side):
                noise.add_(1.0)
        out, pool = call(dict(x, state_pool=x["state_pool"].clone()), "prefill")
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(pool.view(torch.int16), want[1].view(torch.int16))
    torch.cuda.synchronize()
