"""How far an infinity or NaN among a prompt's valid tokens reaches in prefill: a value's its
own column from its chunk of 128 on, a key's its row of the state and the outputs from its
token on, a query's its own output. Everything else is right, within the bounds of
test_linear_attention.py against the oracle on the same call.
"""
import numpy as np
import pytest
import torch

from test_linear_attention import U, call, draw, f64, oracle

pytestmark = pytest.mark.gpu

SHAPES = [(2, 2, 2, 300, 64, 128, 2), (2, 1, 2, 300, 128, 64, 2),  # a CTA for each tile
          (1, 1, 2, 1600, 64, 64, 1),                              # segments
          (4, 20, 40, 300, 64, 64, 4)]                             # equal shares


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("what", ["value", "key", "query"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_what_a_token_that_is_no_number_reaches(shape, what, bad):
    B, Hq, Hv, T, Dk, Dv, P = shape
    t, c, h = 200, 13, 1 if what == "value" else 0
    draw_it = lambda: draw(*shape, seed=30, lengths=[T] * B,  # noqa: E731
                           log_decay=[-0.02 * (1 + i) for i in range(Hv)])
    x = draw_it()
    x[what][0, h, t, c] = bad
    with np.errstate(invalid="ignore"):
        ref = oracle(x)
    mag = oracle(draw_it(), absolute=True)
    out, pool = call({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()},
                     "prefill")
    out, pool = f64(out), f64(pool)
    looked_at = np.ones(out.shape, bool)
    if what == "value":  # the tokens before it in its chunk
        looked_at[0, h, t // 128 * 128:t, c] = False
    for got, want, m, extra, see in ((out, ref[0], mag[0], 2 * U + 2.0 ** -12, looked_at),
                                     (pool, ref[1], mag[1], U + 2.0 ** -12, True)):
        number = np.isfinite(want)
        assert not number.all() or what == "query"
        assert np.all((np.isfinite(got) == number) | ~np.asarray(see))
        see = number & see
        assert np.all(np.abs(got[see] - want[see]) <= U * np.abs(want[see]) * 1.01 + extra * m[see])
    if what == "query":  # its own row, and nothing of the state
        heads = [i for i in range(Hv) if i // (Hv // Hq) == h]
        assert not np.isfinite(out[0, heads, t]).any() and np.isfinite(pool).all()
        assert np.isfinite(np.delete(out, t, axis=2)).all()


@pytest.mark.parametrize("shape", [(1, 1, 2, 300, 128, 64, 1), (1, 1, 2, 2000, 128, 64, 1),
                                   (1, 1, 1, 3000, 64, 64, 1), (4, 20, 40, 300, 64, 64, 4)],
                         ids=str)
def test_a_state_that_is_no_number_stays_so_under_a_strong_decay(shape):
    """The weight of an early token is 0 in fp32 by the end of its chunk, of its segment and of
    the prompt; times an infinity or NaN it is not."""
    B, Hq, Hv, T, Dk, Dv, P = shape
    draw_it = lambda: draw(*shape, seed=32, lengths=[T] * B, log_decay=[-5.0] * Hv)  # noqa: E731
    x = draw_it()
    x["value"][0, 0, 5, 3] = float("nan")
    x["key"][0, 0, 7, 9] = float("inf")
    with np.errstate(invalid="ignore"):
        ref = oracle(x)
    mag = oracle(draw_it(), absolute=True)
    out, pool = call({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()},
                     "prefill")
    for got, want, m, extra in ((f64(out)[:, :, 128:], ref[0][:, :, 128:], mag[0][:, :, 128:],
                                 2 * U + 2.0 ** -12),
                                (f64(pool), ref[1], mag[1], U + 2.0 ** -12)):
        number = np.isfinite(want)
        assert not number.all() and np.array_equal(np.isfinite(got), number)
        assert np.all(np.abs(got[number] - want[number]) <=
                      U * np.abs(want[number]) * 1.01 + extra * m[number])
