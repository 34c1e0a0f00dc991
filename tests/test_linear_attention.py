"""Linear attention with one decay per head: decode (one to eight tokens) and prefill.

GPU results are compared with a float64 oracle that runs the recurrence a token at a time.
The bounds count the roundings of the CUDA path, with u = 2^-8 (bf16's half step) and M the
same recurrence over absolute values, which bounds every sum of magnitudes:

* decode: fp32 arithmetic and one rounding on the store, so
  |err| <= u |ref| + c 2^-24 M with c = the longest chain of fp32 operations (D_k = 128 rows,
  2 T <= 16 terms and some factors: below 256, so c 2^-24 <= 2^-16).
* prefill, state: the weighted keys are rounded to bf16 once (u M), then the store
  (u |ref|), and fp32 sums over at most a few thousand tokens (2^-12 M).
* prefill, out: the products P and the weighted keys behind the copy of the state are
  rounded once, the copy once more: at most 2 u of each term, then the store.
Those bound every element; as each rounding has its own sign, the whole is held to a norm as
well: three roundings of rms u / sqrt(3) each and the store give 2 u / sqrt(3) = 4.6e-3 of
the norm in the worst mantissa, so 5e-3.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle.linear_oracle import linear_attention

U = 2.0 ** -8
NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder pointers are for a machine without a GPU")


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def draw(B, Hq, Hv, T, Dk, Dv, pool, seed=0, lengths=None, indices=None, accepted=None,
         log_decay=None, device="cpu"):
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    x = dict(
        query=randn(B, Hq, T, Dk).to(torch.bfloat16),
        key=(randn(B, Hq, T, Dk) * Dk ** -0.5).to(torch.bfloat16),
        value=randn(B, Hv, T, Dv).to(torch.bfloat16),
        log_decay=-torch.exp(-6.0 * torch.rand(Hv, generator=gen)),
        state_pool=(0.3 * randn(pool, Hv, Dk, Dv)).to(torch.bfloat16),
        lengths=torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32),
        indices=torch.randperm(pool, generator=gen)[:B].to(torch.int32),
        accepted=None, scale=Dk ** -0.5)
    for name, v in (("lengths", lengths), ("indices", indices), ("accepted", accepted)):
        if v is not None:
            x[name] = torch.tensor(v, dtype=torch.int32)
    if log_decay is not None:
        x["log_decay"] = torch.tensor(log_decay, dtype=torch.float32)
    return {k: v.to(device) if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def oracle(x, absolute=False):
    f = (lambda t: np.abs(f64(t))) if absolute else f64
    return linear_attention(f(x["query"]), f(x["key"]), f(x["value"]), f64(x["log_decay"]),
                            f(x["state_pool"]), x["lengths"].cpu().numpy(),
                            x["indices"].cpu().numpy(),
                            None if x["accepted"] is None else x["accepted"].cpu().numpy(),
                            x["scale"])


def poison_padding(x):
    """NaN in every token behind its item's length: none of them may be read."""
    T = x["query"].shape[2]
    for b, L in enumerate(x["lengths"].tolist()):
        L = min(max(L, 0), T)
        for name in ("query", "key", "value"):
            x[name][b, :, L:] = float("nan")


def call(x, op, out=None):
    import gated_delta_rule_recurrent_b200 as gdr

    args = [x["query"], x["key"], x["value"], x["log_decay"], x["state_pool"], x["lengths"],
            x["indices"]]
    if op == "decode":
        return gdr.linear_attention_decode(*args, x["accepted"], x["scale"], out=out)
    return gdr.linear_attention_prefill(*args, x["scale"], out=out)


def check(x, op, got, ref, mag, before):
    """The call's results against the oracle's, padding and untouched slots bit for bit."""
    out, pool = f64(got[0]), f64(got[1])
    T, P = x["query"].shape[2], before.shape[0]
    out_extra = 2.0 ** -16 if op == "decode" else 2 * U + 2.0 ** -12
    pool_extra = 2.0 ** -16 if op == "decode" else U + 2.0 ** -12
    touched = set()
    for b, (s, L) in enumerate(zip(x["indices"].tolist(), x["lengths"].tolist())):
        L = min(max(L, 0), T) if 0 <= s < P else 0
        assert not got[0][b, :, L:].cpu().view(torch.int16).any(), f"item {b}: padding not +0.0"
        n = L if x["accepted"] is None else min(max(int(x["accepted"][b]), 0), L)
        if not L:
            continue
        if n:
            touched.add(s)
        for what, g, r, m, extra in ((f"out of item {b}", out[b, :, :L], ref[0][b, :, :L],
                                      mag[0][b, :, :L], out_extra),
                                     (f"slot of item {b}", pool[s], ref[1][s], mag[1][s],
                                      pool_extra)):
            if what.startswith("slot") and not n:
                continue
            bad = ~(np.abs(g - r) <= U * np.abs(r) * 1.01 + extra * m)
            assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of bounds, first at "
                                   f"{np.argwhere(bad)[0]}: {g[bad][0]} for {r[bad][0]}")
            assert np.linalg.norm(g - r) <= 5e-3 * np.linalg.norm(r), what
    for s in set(range(P)) - touched:
        assert torch.equal(got[1][s].cpu().view(torch.int16), before[s].cpu().view(torch.int16)), s


def run_and_check(x, op):
    poison_padding(x)
    ref, mag = oracle(x), oracle(x, absolute=True)
    before = x["state_pool"].clone()
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    got = call(xd, op)
    torch.cuda.synchronize()
    assert got[1] is xd["state_pool"]
    check(x, op, got, ref, mag, before)
    import gated_delta_rule_recurrent_b200 as gdr

    assert gdr.device_error() == 0
    return got


# ------------------------------------------------------------------ CPU: the oracle, refusals


def test_oracle_is_the_unrolled_sum():
    """o_t = scale (lambda^{t+1} S_0^T q_t + sum_{s <= t} lambda^{t-s} (q_t.k_s) v_s)."""
    x = draw(2, 1, 2, 5, 64, 64, 3, seed=3, lengths=[5, 3])
    out, pool = oracle(x)
    q, k, v, S = (f64(x[n]) for n in ("query", "key", "value", "state_pool"))
    g = f64(x["log_decay"])
    for b, L in enumerate([5, 3]):
        s = int(x["indices"][b])
        for h in range(2):
            for t in range(L):
                o = np.exp(g[h] * (t + 1)) * (q[b, 0, t] @ S[s, h])
                for u in range(t + 1):
                    o = o + np.exp(g[h] * (t - u)) * (q[b, 0, t] @ k[b, 0, u]) * v[b, h, u]
                np.testing.assert_allclose(out[b, h, t], x["scale"] * o, rtol=1e-11, atol=1e-12)
            end = np.exp(g[h] * L) * S[s, h]
            for u in range(L):
                end = end + np.exp(g[h] * (L - 1 - u)) * np.outer(k[b, 0, u], v[b, h, u])
            np.testing.assert_allclose(pool[s, h], end, rtol=1e-11, atol=1e-12)


def test_oracle_commits_the_accepted_tokens_only():
    x = draw(1, 1, 1, 4, 64, 64, 1, seed=4, lengths=[4], accepted=[2])
    some = oracle(x)
    x["lengths"][0], x["accepted"] = 2, None
    np.testing.assert_array_equal(some[1], oracle(x)[1])


def _c_call(dims, op="decode", ptr=16, nulls=()):
    from gated_delta_rule_recurrent_b200 import binding

    L = binding.lib()
    a = [None if i in nulls else ctypes.c_void_p(ptr) for i in range(8)]
    d = None if dims is None else ctypes.byref(binding.Dims(*dims))
    if op == "decode":
        return L.gdr_linear_attention_decode(d, *a[:7], None, ctypes.c_float(1.0), a[7], None)
    return L.gdr_linear_attention_prefill(d, *a[:7], ctypes.c_float(1.0), a[7], None, 0, None)


@NO_DEVICE
@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("dims,status", [
    ((2, 0, 4, 4, 64, 64, 2), 2),
    ((2, 2, 3, 4, 64, 64, 2), 2),          # H_v not a multiple of H_qk
    ((2, 2, 0, 4, 64, 64, 2), 2),
    ((2, 2, 4, 4, 64, 64, 0), 2),
    ((-1, 2, 4, 4, 64, 64, 2), 2),
    ((2, 2, 4, 4, 96, 64, 2), 4),
    ((2, 2, 4, 4, 256, 64, 2), 4),
    ((2, 2, 4, 4, 64, 96, 2), 4),
    ((2, 2, 4, 4, 64, 64, 2, 1), 4),       # k-contiguous pool
    ((2, 2, 4, 4, 64, 64, 2, 2), 2),
    ((2 ** 30, 1, 1, 64, 64, 512, 2), 2),  # grid overflow
    ((2, 2 ** 31 - 1, 4, 4, 64, 512, 2), 2),
    (None, 1),
])
def test_bad_sizes_are_refused(built_library, op, dims, status):
    from gated_delta_rule_recurrent_b200 import binding

    assert _c_call(dims, op) == status
    assert binding.lib().gdr_last_error().decode() != ""


@NO_DEVICE
def test_more_than_eight_tokens_go_to_prefill(built_library):
    assert _c_call((2, 9, 4, 4, 64, 64, 2)) == 2


@NO_DEVICE
@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_null_misaligned_and_empty(built_library, op):
    good = (2, 2, 4, 4, 64, 64, 2)
    for i in range(8):
        assert _c_call(good, op, nulls=(i,)) == 1, i
    assert _c_call(good, op, ptr=24) == 3
    assert _c_call((0, 2, 4, 4, 64, 64, 2), op, nulls=range(8)) == 0


def test_binding_refuses_cpu_tensors(built_library):
    x = draw(1, 1, 1, 2, 64, 64, 1)
    for op in ("decode", "prefill"):
        with pytest.raises(RuntimeError, match="CUDA"):
            call(x, op)


# ------------------------------------------------------------------ GPU

DECODE = [
    # B, Hq, Hv, T, Dk, Dv, pool
    (1, 1, 1, 1, 64, 64, 1),
    (3, 2, 4, 1, 128, 64, 5),
    (2, 1, 3, 1, 64, 320, 2),
    (5, 4, 4, 1, 128, 128, 7),
    (40, 8, 8, 1, 64, 512, 41),      # more than 8 tiles for each SM: one warp a tile
    (80, 16, 16, 1, 128, 128, 80),
    (2, 1, 1, 2, 64, 64, 2),
    (3, 1, 4, 3, 128, 64, 4),
    (4, 2, 2, 4, 64, 192, 6),
    (3, 3, 3, 5, 128, 320, 3),
    (2, 2, 4, 7, 64, 512, 2),
    (6, 2, 2, 8, 128, 128, 9),
    (4, 1, 2, 8, 64, 448, 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", DECODE, ids=str)
def test_decode(shape):
    for seed in (0, 1):
        x = draw(*shape, seed=seed)
        T = shape[3]
        if seed:
            gen = torch.Generator().manual_seed(9)
            x["accepted"] = torch.randint(-1, T + 2, (shape[0],), generator=gen,
                                          dtype=torch.int32)
        run_and_check(x, "decode")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 8])
def test_decode_lengths_slots_and_counts_out_of_range(T):
    x = draw(8, 2, 2, T, 64, 128, 6, seed=5, lengths=[T, 0, -3, T + 5, 1, T, T, 1],
             indices=[0, 1, 2, 3, 4, -1, 6, 5], accepted=[T, 1, 1, T + 9, 0, 1, 1, -7])
    run_and_check(x, "decode")


@pytest.mark.gpu
@pytest.mark.parametrize("op,T", [("decode", 1), ("decode", 6), ("prefill", 150)])
def test_extreme_decays(op, T):
    """No decay, a decay of exactly 0, one that underflows at once, and a growing state."""
    x = draw(2, 5, 5, T, 64, 64, 2, seed=6, lengths=[T, max(1, T - 1)],
             log_decay=[0.0, float("-inf"), -200.0, 0.01, -1e-8])
    run_and_check(x, op)


@pytest.mark.gpu
def test_infinities_of_tokens_that_are_not_committed_stay_out_of_the_state():
    x = draw(1, 1, 1, 6, 64, 64, 1, seed=7, lengths=[6], accepted=[3])
    x["value"][0, 0, 4, 5] = float("inf")
    x["key"][0, 0, 5, 7] = float("nan")
    clean = draw(1, 1, 1, 6, 64, 64, 1, seed=7, lengths=[6], accepted=[3])
    ref = oracle(clean)
    out, pool = call({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()},
                     "decode")
    assert np.all(np.abs(f64(pool) - ref[1]) <= U * np.abs(ref[1]) * 1.01 + 1e-4)
    assert torch.isfinite(out[0, 0, :4]).all()  # the tokens before the infinity
    assert not torch.isfinite(out[0, 0, 4, 5])


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("Dk", [64, 128])
def test_committed_infinities_stay_in_their_rows_and_columns(op, Dk):
    """Eight tokens: an infinite value, then an infinite key component, in the head that has
    them; the slot holds no number exactly where the recurrence has none."""
    x = draw(1, 2, 2, 8, Dk, 128, 1, seed=11, lengths=[8])
    x["value"][0, 0, 2, 70] = float("inf")
    x["key"][0, 0, 5, 9] = float("-inf")
    with np.errstate(invalid="ignore"):
        ref = oracle(x)
    mag = oracle(draw(1, 2, 2, 8, Dk, 128, 1, seed=11, lengths=[8]), absolute=True)
    out, pool = call({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()},
                     op)
    for got, want, m in ((f64(out), ref[0], mag[0]), (f64(pool), ref[1], mag[1])):
        number = np.isfinite(want)
        assert not number.all() and np.array_equal(np.isfinite(got), number)
        got, want, m = got[number], want[number], m[number]
        assert np.all(np.abs(got - want) <= U * np.abs(want) * 1.01 + 2.0 ** -16 * m)


PREFILL = [
    (1, 1, 1, 1, 64, 64, 1),
    (2, 1, 2, 2, 128, 64, 2),
    (2, 2, 2, 63, 64, 128, 3),
    (1, 1, 1, 127, 128, 128, 1),
    (2, 1, 1, 128, 64, 192, 2),
    (2, 1, 4, 129, 128, 128, 2),
    (1, 2, 2, 256, 64, 320, 1),
    (3, 1, 2, 257, 128, 192, 4),
    (2, 1, 1, 640, 128, 128, 2),
    (2, 1, 1, 900, 64, 64, 2),
    (1, 1, 1, 1300, 128, 64, 1),
    # few tiles and 12 chunks or more: cut into segments
    (1, 1, 1, 1536, 64, 128, 2),
    (2, 1, 2, 1700, 128, 192, 3),
    (3, 1, 1, 2900, 64, 320, 3),
    (1, 1, 1, 5000, 128, 64, 1),
    # more tiles than SMs: equal shares of the chunks, tiles that go on in the next CTA
    (5, 40, 40, 300, 64, 64, 6),
    (3, 30, 60, 700, 128, 128, 4),
    (40, 2, 4, 130, 64, 192, 40),
    (9, 10, 20, 13, 128, 64, 9),
    # and more items than a CTA counts
    (300, 1, 1, 10, 64, 64, 300),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", PREFILL, ids=str)
def test_prefill(shape):
    x = draw(*shape, seed=2)
    x["lengths"][0] = shape[3]  # one full item, the others ragged (some may be empty)
    run_and_check(x, "prefill")


@pytest.mark.gpu
@pytest.mark.parametrize("Dk", [64, 128])
def test_prefill_lengths_and_slots_out_of_range(Dk):
    T = 300
    x = draw(9, 1, 2, T, Dk, 128, 7, seed=8, lengths=[T, 0, -3, T + 5, 1, 128, 129, 256, 200],
             indices=[0, 1, 2, 3, 4, 5, 6, -1, 7])
    run_and_check(x, "prefill")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 1, 2, 200, 64, 128, 2), (4, 40, 40, 140, 128, 64, 4),
                                   (1, 1, 1, 3000, 64, 64, 1)], ids=str)
def test_prefill_of_nothing(shape):
    """Every item empty or without a slot: zeros out, no slot touched."""
    x = draw(*shape, seed=16, lengths=[0] * shape[0])
    run_and_check(x, "prefill")
    x = draw(*shape, seed=16, lengths=[shape[3]] * shape[0], indices=[shape[6]] * shape[0])
    run_and_check(x, "prefill")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 1, 2, 2500, 64, 64, 1), (4, 20, 40, 300, 64, 64, 4)],
                         ids=str)
def test_two_prefills_on_two_streams_do_not_share_a_workspace(shape):
    """Calls that need a workspace, queued side by side: each has its own."""
    x = draw(*shape, seed=17, device="cuda")
    want = call(dict(x, state_pool=x["state_pool"].clone()), "prefill")
    y = draw(*shape, seed=18, device="cuda")
    want_y = call(dict(y, state_pool=y["state_pool"].clone()), "prefill")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for z, stream in zip((x, y), streams):
            with torch.cuda.stream(stream):
                got.append(call(dict(z, state_pool=z["state_pool"].clone()), "prefill"))
    torch.cuda.synchronize()
    for k, (out, pool) in enumerate(got):
        w = (want, want_y)[k % 2]
        assert torch.equal(out.view(torch.int16), w[0].view(torch.int16))
        assert torch.equal(pool.view(torch.int16), w[1].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T", [(1, 2, 9000), (8, 20, 1000), (1, 3, 1000)])
def test_prefill_of_short_items_in_a_long_call(B, H, T):
    """Most of the output is padding, which every mode writes as zeros."""
    x = draw(B, H, H, T, 64, 192, B, seed=20, lengths=[3 + 20 * b for b in range(B)])
    run_and_check(x, "prefill")


@pytest.mark.gpu
@pytest.mark.parametrize("Dk", [64, 128])
def test_prefill_in_two_calls_and_then_decode(Dk):
    """A prompt given in two calls and its next tokens, against one run of the oracle."""
    B, Hq, Hv, Dv, n1, n2, n3 = 2, 1, 2, 128, 200, 77, 5
    T = n1 + n2 + n3
    x = draw(B, Hq, Hv, T, Dk, Dv, 3, seed=11, lengths=[T, T])
    ref, mag = oracle(x), oracle(x, absolute=True)
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    outs, at = [], 0
    for n, op in ((n1, "prefill"), (n2, "prefill"), (n3, "decode")):
        part = dict(xd)
        for name in ("query", "key", "value"):
            part[name] = xd[name][:, :, at:at + n].contiguous()
        part["lengths"] = torch.full((B,), n, dtype=torch.int32, device="cuda")
        outs.append(call(part, op)[0])
        at += n
    out = f64(torch.cat(outs, 2))
    # two more roundings of the state than one call
    assert np.all(np.abs(out - ref[0]) <= U * np.abs(ref[0]) + 4 * U * mag[0] + 1e-6)
    assert np.linalg.norm(out - ref[0]) <= 6e-3 * np.linalg.norm(ref[0])


# the last three: a CTA for each tile, tiles cut into segments, equal shares
REPEATS = [("decode", (2, 2, 2, 1, 64, 128, 3)), ("decode", (2, 2, 2, 5, 128, 64, 3)),
           ("prefill", (2, 2, 2, 200, 128, 192, 3)), ("prefill", (1, 1, 2, 2500, 64, 64, 1)),
           ("prefill", (4, 20, 40, 500, 128, 128, 4))]


@pytest.mark.gpu
@pytest.mark.parametrize("op,shape", REPEATS, ids=str)
def test_results_repeat_and_do_not_depend_on_the_stream(op, shape):
    x = draw(*shape, seed=12, device="cuda")
    pools, outs = [], []
    side = torch.cuda.Stream()
    for where in (None, side, None):
        y = dict(x, state_pool=x["state_pool"].clone())
        torch.cuda.synchronize()
        if where is None:
            out, pool = call(y, op)
        else:
            with torch.cuda.stream(where):
                out, pool = call(y, op)
        torch.cuda.synchronize()
        outs.append(out)
        pools.append(pool)
    for o, p in zip(outs[1:], pools[1:]):
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
        assert torch.equal(p.view(torch.int16), pools[0].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("op,shape", REPEATS, ids=str)
def test_graph_replay(op, shape):
    x = draw(*shape, seed=13, device="cuda")
    start = x["state_pool"].clone()
    want, after = call(dict(x, state_pool=start.clone()), op)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, op, out=out)
    for _ in range(2):
        x["state_pool"].copy_(start)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert torch.equal(x["state_pool"].view(torch.int16), after.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("op,T", [("decode", 1), ("decode", 3), ("prefill", 140)])
def test_a_slot_behind_two_to_the_31_values(op, T):
    """Element offsets of the last slots pass 32 bits."""
    H, Dk, Dv = 16, 128, 512
    pool = (2 ** 31) // (H * Dk * Dv) + 3
    x = draw(1, H, H, T, Dk, Dv, 1, seed=14, lengths=[T])
    ref, mag = oracle(x), oracle(x, absolute=True)
    big = torch.empty(pool, H, Dk, Dv, dtype=torch.bfloat16, device="cuda")
    big[pool - 1] = x["state_pool"][0].cuda()
    big[pool - 2] = 0.0
    xd = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    xd["state_pool"], xd["indices"] = big, torch.tensor([pool - 1], dtype=torch.int32).cuda()
    out, _ = call(xd, op)
    check(dict(x, indices=torch.tensor([0])), op, (out, big[pool - 1:]), ref, mag,
          x["state_pool"])
    assert not big[pool - 2].any()


GUARD = 4096


@pytest.mark.gpu
@pytest.mark.parametrize("op,shape", [("decode", (2, 2, 4, 1, 64, 192, 4)),
                                      ("decode", (2, 2, 4, 6, 128, 192, 4)),
                                      ("prefill", (2, 2, 4, 150, 128, 192, 4)),
                                      ("prefill", (2, 2, 4, 150, 64, 64, 4)),
                                      ("prefill", (1, 1, 2, 1700, 64, 64, 2)),
                                      ("prefill", (4, 20, 40, 200, 64, 64, 5))])
def test_nothing_is_written_outside(op, shape):
    """Every tensor sits between guard bands; bands and inputs keep their bits."""
    x = draw(*shape, seed=15)
    x["out"] = torch.zeros(shape[0], shape[2], shape[3], shape[5], dtype=torch.bfloat16)
    held, whole = {}, {}
    for name, t in x.items():
        if not isinstance(t, torch.Tensor):
            held[name] = t
            continue
        raw = t.contiguous().view(torch.uint8).reshape(-1)
        buf = torch.full((raw.numel() + 2 * GUARD,), 0xA5, dtype=torch.uint8)
        buf[GUARD:GUARD + raw.numel()] = raw
        whole[name] = (buf, buf.cuda())
        held[name] = whole[name][1][GUARD:GUARD + raw.numel()].view(t.dtype).view(t.shape)
    call(held, op, out=held["out"])
    torch.cuda.synchronize()
    for name, (was, now) in whole.items():
        now = now.cpu()
        assert torch.equal(now[:GUARD], was[:GUARD]) and torch.equal(now[-GUARD:], was[-GUARD:])
        if name not in ("out", "state_pool"):
            assert torch.equal(now, was), name


@pytest.mark.gpu
def test_binding_refusals():
    import gated_delta_rule_recurrent_b200 as gdr

    x = draw(2, 2, 4, 3, 64, 64, 2, device="cuda")
    for name, bad in (("query", x["query"].float()), ("key", x["key"][:, :, :2]),
                      ("value", x["value"].transpose(2, 3)),
                      ("log_decay", x["log_decay"].double()), ("log_decay", x["log_decay"][:2]),
                      ("state_pool", x["state_pool"][:, :2]),
                      ("lengths", x["lengths"].long()), ("indices", x["indices"][:1]),
                      ("lengths", x["lengths"].cpu()), ("state_pool", x["state_pool"][0])):
        for op in ("decode", "prefill"):
            with pytest.raises(RuntimeError):
                call(dict(x, **{name: bad}), op)
    with pytest.raises(RuntimeError):
        call(x, "decode", out=torch.empty(2, 4, 3, 64, device="cuda"))
    y = draw(1, 1, 1, 9, 64, 64, 1, device="cuda")
    with pytest.raises(gdr.GdrError):
        call(y, "decode")
    call(y, "prefill")
    odd = torch.empty(1 + y["query"].numel(), dtype=torch.bfloat16, device="cuda")[1:]
    with pytest.raises(gdr.GdrError):  # not 16-byte aligned
        call(dict(y, query=odd.view_as(y["query"])), "prefill")


@pytest.mark.gpu
def test_empty_batch_queues_nothing():
    import gated_delta_rule_recurrent_b200 as gdr

    x = draw(0, 1, 1, 2, 64, 64, 1, device="cuda")
    for op in ("decode", "prefill"):
        out, _ = call(x, op)
        assert out.shape == (0, 1, 2, 64)
        assert gdr.last_launch()["kernel"] == "none"


# ------------------------------------------------------------------ a wait that runs out


@pytest.fixture(scope="module")
def hooks():
    """The test build, in which a producer can hold a block's loads back and the budget of
    the waits is short."""
    from gated_delta_rule_recurrent_b200 import binding, build

    L = ctypes.CDLL(build.ensure_built(test_hooks=True))
    for name in ("gdr_linear_attention_decode", "gdr_linear_attention_prefill",
                 "gdr_linear_attention_prefill_workspace", "gdr_device_error"):
        getattr(L, name).argtypes = getattr(binding.lib(), name).argtypes
    L.gdrtest_set_hooks.argtypes = [ctypes.c_longlong, ctypes.c_int]
    yield L
    assert L.gdrtest_set_hooks(0, -1) == 0


def _hooked_call(L, x, op):
    from gated_delta_rule_recurrent_b200 import binding

    P = binding._ptr
    B, Hq, T, Dk = x["query"].shape
    Hv, Dv = x["value"].shape[1], x["value"].shape[3]
    d = binding.Dims(B, T, Hq, Hv, Dk, Dv, x["state_pool"].shape[0], 0)
    out = torch.zeros_like(x["value"])
    args = [ctypes.byref(d), *(P(x[n]) for n in ("query", "key", "value", "log_decay",
                                                  "state_pool", "lengths", "indices"))]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "decode":
        rc = L.gdr_linear_attention_decode(*args, None, x["scale"], P(out), stream)
    else:
        need = ctypes.c_int64(0)
        assert L.gdr_linear_attention_prefill_workspace(ctypes.byref(d), ctypes.byref(need)) == 0
        work = torch.empty(max(need.value, 16), dtype=torch.uint8, device="cuda")
        rc = L.gdr_linear_attention_prefill(*args, x["scale"], P(out), P(work), need.value,
                                            stream)
    assert rc == 0
    torch.cuda.synchronize()
    flags = ctypes.c_uint32(0)
    assert L.gdr_device_error(ctypes.byref(flags), 1) == 0
    return out, flags.value


@pytest.mark.gpu
@pytest.mark.parametrize("op,shape,held", [
    ("decode", (2, 1, 3, 1, 128, 64, 2), 4),
    ("decode", (2, 1, 3, 8, 64, 64, 2), 1),
    ("prefill", (2, 1, 3, 300, 128, 128, 2), 4),     # a CTA for each tile
    ("prefill", (1, 1, 1, 2000, 64, 64, 1), 3),      # segments
    ("prefill", (4, 20, 40, 300, 64, 64, 4), 70),    # equal shares, states handed on
])
def test_held_loads_time_out_cleanly(hooks, op, shape, held):
    """The call ends, says so in the error word, leaves each slot old or right, and the next
    call is right."""
    x = draw(*shape, seed=19, lengths=[shape[3]] * shape[0])
    ref, mag = oracle(x), oracle(x, absolute=True)
    fresh = lambda: {k: v.cuda() if isinstance(v, torch.Tensor) else v  # noqa: E731
                     for k, v in x.items()}
    xd = fresh()
    assert _hooked_call(hooks, xd, op)[1] == 0
    xd = fresh()
    assert hooks.gdrtest_set_hooks(4_000_000, held) == 0
    _, word = _hooked_call(hooks, xd, op)
    assert hooks.gdrtest_set_hooks(0, -1) == 0
    assert word & 3 and not word & 4, word
    now, was = f64(xd["state_pool"]), f64(x["state_pool"])
    right = np.abs(now - ref[1]) <= U * np.abs(ref[1]) * 1.01 + (U + 2.0 ** -12) * mag[1]
    assert np.all(right | (now == was))
    if op == "decode" or shape[0] == 2:  # block `held` is value head `held` of all items
        b, h = divmod(held, shape[2])
        slot = int(x["indices"][b])
        assert np.array_equal(now[slot, h], was[slot, h])
        assert right.reshape(*right.shape[:2], -1).all(-1).sum() >= shape[0] * shape[2] - 1
    xd = fresh()
    out, word = _hooked_call(hooks, xd, op)
    assert word == 0
    check(x, op, (out, xd["state_pool"]), ref, mag, x["state_pool"])
