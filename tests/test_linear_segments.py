"""Prefill of few tiles and long prompts, cut into segments: the launches ahead of the main
kernel, and a first pass that does not get to the end of its sums.
"""
import numpy as np
import pytest
import torch

from test_linear_attention import (U, _hooked_call, call, check, draw, f64,  # noqa: F401
                                   hooks, oracle)

pytestmark = pytest.mark.gpu

# (shape, blocks of the main kernel): the hook counts the first pass's blocks on from there
CASES = [((1, 1, 1, 2000, 64, 64, 1), 8), ((1, 2, 2, 2400, 128, 192, 2), 28)]


@pytest.mark.parametrize("shape,blocks,held", [(*CASES[c], held) for c, held in (
    (0, 0), (0, 3), (0, 6), (1, 0), (1, 17))], ids=str)
def test_no_slot_is_written_without_its_sums(hooks, shape, blocks, held):
    """A block of the first pass whose loads are held back: its tile's slot keeps its bits and
    the others are old or right (the main kernel's blocks start while the first pass waits,
    and their waits may run out with it); the next call is right."""
    x = draw(*shape, seed=25, lengths=[shape[3]])
    ref, mag = oracle(x), oracle(x, absolute=True)
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    assert hooks.gdrtest_set_hooks(4_000_000, blocks + held) == 0
    _, word = _hooked_call(hooks, xd, "prefill")
    assert hooks.gdrtest_set_hooks(0, -1) == 0
    assert word & 3 and not word & 4, word
    slot = int(x["indices"][0])
    now, was = f64(xd["state_pool"])[slot], f64(x["state_pool"])[slot]
    right = np.abs(now - ref[1][slot]) <= U * np.abs(ref[1][slot]) * 1.01 + \
        (U + 2.0 ** -12) * mag[1][slot]
    slices = -(-shape[5] // 128)
    tile = held // (blocks // (shape[2] * slices) - 1)
    for h in range(shape[2]):
        for s in range(slices):
            cols = np.s_[h, :, 128 * s:128 * (s + 1)]
            if h * slices + s == tile:
                assert np.array_equal(now[cols], was[cols]), "a slot without its sums"
            else:
                assert right[cols].all() or np.array_equal(now[cols], was[cols])
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out, word = _hooked_call(hooks, xd, "prefill")
    assert word == 0
    check(x, "prefill", (out, xd["state_pool"]), ref, mag, x["state_pool"])


@pytest.mark.parametrize("shape", [c[0] for c in CASES] + [(2, 4, 4, 4000, 128, 128, 2)], ids=str)
def test_segments_repeat_beside_other_work(shape):
    """The first segment's start does not depend on when its block begins."""
    x = draw(*shape, seed=26, lengths=[shape[3]] * shape[0], device="cuda")
    want = call(dict(x, state_pool=x["state_pool"].clone()), "prefill")
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(12):
        with torch.cuda.stream(side):  # work that takes SMs away
            for _ in range(k % 3):
                a.mul_(1.0)
        out, pool = call(dict(x, state_pool=x["state_pool"].clone()), "prefill")
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(pool.view(torch.int16), want[1].view(torch.int16))
    torch.cuda.synchronize()
