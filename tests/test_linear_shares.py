"""Prefill with more tiles than SMs: blocks that store a slot and then receive a state,
receive one and hand it on, or hand one on before they receive one, against the float64
oracle within the bounds of test_linear_attention.py. test_linear_schedule.py counts on the
CPU which of these the cases reach.
"""
import functools

import numpy as np
import pytest
import torch

from test_linear_attention import (U, _hooked_call, call, check, draw, f64,  # noqa: F401
                                   hooks, oracle, run_and_check)
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


@functools.lru_cache(None)
def chain_oracle():
    shape, lengths = CHAINS[0]
    x = draw(*shape, seed=24, lengths=lengths)
    return oracle(x), oracle(x, absolute=True)


# Blocks of the first CHAINS case (a tile of 9 chunks a head, shares of 10): 8 stores the slot
# of tile 9 and then receives tile 8's state; 18 hands tile 21's on and then starts tile 20
# from its slot.
@pytest.mark.parametrize("block,warp,place", [(8, 5, 0), (8, 10, 0), (8, 15, 0), (18, 4, 0),
                                              (18, 8, 0), (18, 12, 0), (18, 13, 1), (18, 12, 1)])
def test_one_warp_that_gives_up_alone_ends_the_call(hooks, block, warp, place):
    """Also while the others of its group are let through: nobody stays at a barrier. Slots
    are old or right, and the next call is right."""
    shape, lengths = CHAINS[0]
    x = draw(*shape, seed=24, lengths=lengths)
    ref, mag = chain_oracle()
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    assert hooks.gdrtest_set_hooks(4_000_000, -2 - (2 * (16 * block + warp) + place)) == 0
    _, word = _hooked_call(hooks, xd, "prefill")
    assert hooks.gdrtest_set_hooks(0, -1) == 0
    assert word & 3 and not word & 4, word
    now, was = f64(xd["state_pool"]), f64(x["state_pool"])
    right = np.abs(now - ref[1]) <= U * np.abs(ref[1]) * 1.01 + (U + 2.0 ** -12) * mag[1]
    whole = right.all((2, 3)) | (now == was).all((2, 3))
    assert whole.all()
    assert right.all((2, 3)).sum() >= 8  # of the tiles ahead of it
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out, word = _hooked_call(hooks, xd, "prefill")
    assert word == 0
    check(x, "prefill", (out, xd["state_pool"]), ref, mag, x["state_pool"])


def test_a_state_is_handed_on_before_its_block_waits_for_one(hooks):
    """With block 0 held back, the one state that does not come is tile 1's: the blocks behind
    it hand theirs on before they wait, so tiles 2 .. are right (and not a chain in which each
    block waits for all the ones before it)."""
    shape, lengths = CHAINS[0]
    x = draw(*shape, seed=24, lengths=lengths)
    ref, mag = chain_oracle()
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    assert hooks.gdrtest_set_hooks(4_000_000, 0) == 0
    _, word = _hooked_call(hooks, xd, "prefill")
    assert hooks.gdrtest_set_hooks(0, -1) == 0
    assert word & 3 and not word & 4, word
    now, was = f64(xd["state_pool"]), f64(x["state_pool"])
    right = np.abs(now - ref[1]) <= U * np.abs(ref[1]) * 1.01 + (U + 2.0 ** -12) * mag[1]
    assert (now[0, :2] == was[0, :2]).all()
    assert right[0, 2:].all()
