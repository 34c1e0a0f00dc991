"""The state pool's 8-bit cache: slots written as codes with a scale for each 64 values, and
read back.

Codes and scales are defined by single fp32 operations (a quotient, a product, a rounding to
nearest even), so the CUDA path has to match the oracle bit for bit. What comes back is
within half a code's step of what went in, plus the roundings of the product and to bf16:
int8 |err| <= m/127 (1/2 + 2^-16) + 2^-8 |x'|, e4m3 |err| <= 2^-4 |x| + m/448 2^-10 (below
its smallest normal number) and the same roundings.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import linear_oracle

NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder pointers are for a machine without a GPU")
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make(P, N, H, R, C, kind, seed=0, device="cpu"):
    gen = torch.Generator().manual_seed(seed)
    # magnitudes that differ from row to row, as the keys' do
    size = torch.exp(4.0 * torch.randn(P, H, R, 1, generator=gen))
    pool = (size * torch.randn(P, H, R, C, generator=gen)).to(torch.bfloat16)
    cache = torch.randint(-100, 100, (N, H, R, C), generator=gen, dtype=torch.int8)
    return dict(pool=pool.to(device), cache=cache.to(device).view(KINDS[kind]),
                scales=torch.rand(N, H, R, C // 64, generator=gen).to(device))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ CPU


@pytest.mark.parametrize("kind", KINDS)
def test_oracle_codes_are_the_nearest_ones(kind):
    """Against torch's own rounding to the type, and the bounds above."""
    x = make(2, 1, 1, 8, 192, kind, seed=1)["pool"].float()
    codes, scales = linear_oracle.quantize(x.numpy(), kind)
    back = linear_oracle.dequantize(codes, scales, kind)
    m = x.reshape(*x.shape[:-1], 3, 64).abs().amax(-1)
    top = 448.0 if kind == "e4m3" else 127.0
    y = (x.reshape(*x.shape[:-1], 3, 64) * torch.div(torch.full_like(m, top), m)[..., None]).flatten(-2)
    want = y.to(KINDS[kind]) if kind == "e4m3" else y.round().to(torch.int8)
    assert np.array_equal(codes.view(np.uint8), want.view(torch.uint8).numpy())
    step = np.repeat(scales.astype(np.float64), 64, -1)
    err = np.abs(back - x.numpy())
    bound = 0.5 * step if kind == "int8" else \
        np.maximum(2.0 ** -4 * np.abs(x.numpy()), step * 2.0 ** -10)
    assert np.all(err <= bound * (1 + 2.0 ** -12))


def test_oracle_groups_that_hold_nothing_or_no_numbers():
    x = np.zeros((1, 256), np.float32)
    x[0, 64] = 2.0 ** -101
    x[0, 128] = np.inf
    x[0, 192] = np.nan
    for kind in KINDS:
        codes, scales = linear_oracle.quantize(x, kind)
        assert scales[0, 0] == 0 and scales[0, 1] == 0 and np.isnan(scales[0, 2:]).all()
        back = linear_oracle.dequantize(codes, scales, kind)
        assert not back[0, :128].any() and np.isnan(back[0, 128:]).all()


def _c_call(op, pool=16, slots=16, cache=16, scales=16, entries=16, pool_size=2, cache_size=2,
            n=1, values=64, kind=0):
    from gated_delta_rule_recurrent_b200 import binding

    L, P = binding.lib(), ctypes.c_void_p
    p, s, c, f, e = (P(v) if v else None for v in (pool, slots, cache, scales, entries))
    if op == "quantize":
        return L.gdr_state_quantize(p, pool_size, s, c, f, cache_size, e, n, values, kind, None)
    return L.gdr_state_dequantize(c, f, cache_size, e, p, pool_size, s, n, values, kind, None)


@NO_DEVICE
@pytest.mark.parametrize("op", ["quantize", "dequantize"])
@pytest.mark.parametrize("args,status", [
    (dict(n=-1), 2), (dict(pool_size=0), 2), (dict(cache_size=0), 2), (dict(values=0), 2),
    (dict(values=96), 2), (dict(values=-64), 2), (dict(kind=2), 4), (dict(kind=-1), 4),
    (dict(values=1 << 62), 2), (dict(n=2 ** 31 - 1, values=1 << 20), 2),
    (dict(pool=0), 1), (dict(slots=0), 1), (dict(cache=0), 1), (dict(scales=0), 1),
    (dict(entries=0), 1), (dict(pool=24), 3), (dict(cache=24), 3), (dict(scales=24), 3),
    (dict(n=0, pool=0, slots=0, cache=0, scales=0, entries=0), 0),
])
def test_refusals(built_library, op, args, status):
    from gated_delta_rule_recurrent_b200 import binding

    assert _c_call(op, **args) == status
    if status:
        assert binding.lib().gdr_last_error().decode() != ""


def test_binding_refuses_cpu_tensors(built_library):
    import gated_delta_rule_recurrent_b200 as gdr

    x = make(1, 1, 1, 1, 64, "int8")
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="CUDA"):
        gdr.state_quantize(x["pool"], one, x["cache"], x["scales"], one)


# ------------------------------------------------------------------ GPU

SHAPES = [(3, 2, 1, 1, 64), (4, 5, 3, 64, 64), (5, 3, 2, 64, 512), (3, 3, 4, 128, 128),
          (3, 4, 1, 320, 128), (2, 2, 5, 128, 192), (2, 3, 129, 1, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_and_back(shape, kind):
    import gated_delta_rule_recurrent_b200 as gdr

    P, N = shape[:2]
    x = make(*shape, kind, seed=2, device="cuda")
    x["pool"][0, 0, 0, :8] = torch.tensor([0.0, -0.0, 1.0, -1.0, 448.0, 3e38, -3e38, 1e-38])
    before = {k: v.clone() for k, v in x.items()}
    n = min(P, N) - 1
    slots, entries = list(range(n)), [N - 1 - i for i in range(n)]
    got = gdr.state_quantize(x["pool"], i32(slots), x["cache"], x["scales"], i32(entries))
    assert got[0] is x["cache"] and got[1] is x["scales"]
    for s, e in zip(slots, entries):
        codes, scales = linear_oracle.quantize(x["pool"][s].float().cpu().numpy(), kind)
        assert np.array_equal(x["cache"][e].view(torch.uint8).cpu().numpy(),
                              codes.view(np.uint8))
        assert np.array_equal(x["scales"][e].cpu().numpy(), scales)
    for e in set(range(N)) - set(entries):
        assert torch.equal(x["cache"][e].view(torch.uint8), before["cache"][e].view(torch.uint8))
        assert torch.equal(x["scales"][e], before["scales"][e])
    assert torch.equal(x["pool"].view(torch.int16), before["pool"].view(torch.int16))

    out = torch.full_like(x["pool"], 9.0)
    back = [P - 1 - i for i in range(n)]
    assert gdr.state_dequantize(x["cache"], x["scales"], i32(entries), out, i32(back)) is out
    for e, b in zip(entries, back):
        want = linear_oracle.dequantize(x["cache"][e].view(torch.uint8).cpu().numpy()
                                        .view(np.int8 if kind == "int8" else np.uint8),
                                        x["scales"][e].cpu().numpy(), kind)
        want = torch.from_numpy(want).float().to(torch.bfloat16)
        assert torch.equal(out[b].cpu().view(torch.int16), want.view(torch.int16))
    for s in set(range(P)) - set(back):
        assert (out[s] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_every_code_reads_back(kind):
    import gated_delta_rule_recurrent_b200 as gdr

    cache = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8)
    cache = cache.view(torch.int8).view(1, 1, 4, 64).contiguous()
    scales = torch.tensor([1.0, 0.375, 2.0 ** -120, 3e30], device="cuda").view(1, 1, 4, 1)
    pool = torch.empty(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    gdr.state_dequantize(cache.view(KINDS[kind]), scales, i32([0]), pool, i32([0]))
    want = (cache.view(KINDS[kind]).float() * scales).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(pool.float(), nan=77.0),
                       torch.nan_to_num(want.float(), nan=77.0))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_zeros_tiny_groups_and_groups_that_are_no_numbers(kind):
    import gated_delta_rule_recurrent_b200 as gdr

    pool = torch.zeros(2, 1, 1, 512, dtype=torch.bfloat16, device="cuda")
    g = pool.view(2, 8, 64)
    g[0, 1, 3] = 2.0 ** -101        # below the floor
    g[0, 2, 3] = -(2.0 ** -100)     # on it
    g[0, 3, 3] = float("inf")
    g[0, 4, 3] = float("-inf")
    g[0, 5, 3] = float("nan")
    g[0, 6, 3] = 3.3e38
    g[0, 7] = -5.0
    cache = torch.zeros(1, 1, 1, 512, dtype=torch.int8, device="cuda").view(KINDS[kind])
    scales = torch.zeros(1, 1, 1, 8, device="cuda")
    gdr.state_quantize(pool, i32([0]), cache, scales, i32([0]))
    gdr.state_dequantize(cache, scales, i32([0]), pool, i32([1]))
    back = g[1].float()
    assert not back[0].any() and not back[1].any()
    assert abs(back[2, 3].item() / 2.0 ** -100 + 1) < 2.0 ** -7
    assert torch.isnan(back[3:6]).all()
    assert abs(back[6, 3].item() / 3.3e38 - 1) < 2.0 ** -6
    assert ((back[7] + 5.0).abs() < 5.0 * 2.0 ** -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_pairs_out_of_range_are_skipped_and_one_entry_serves_many(kind):
    import gated_delta_rule_recurrent_b200 as gdr

    x = make(6, 3, 2, 64, 64, kind, seed=3, device="cuda")
    before = {k: v.clone() for k, v in x.items()}
    gdr.state_quantize(x["pool"], i32([-1, 6, 2, 3]), x["cache"], x["scales"],
                       i32([0, 1, 3, -5]))
    for k in before:
        assert torch.equal(x[k].view(torch.uint8), before[k].view(torch.uint8)), k
    gdr.state_quantize(x["pool"], i32([4]), x["cache"], x["scales"], i32([1]))
    gdr.state_dequantize(x["cache"], x["scales"], i32([1, 1, 1, 7]), x["pool"],
                         i32([0, 5, 9, 2]))
    assert torch.equal(x["pool"][0], x["pool"][5])
    assert not torch.equal(x["pool"][0], before["pool"][0])
    for s in (1, 2, 3, 4):
        assert torch.equal(x["pool"][s], before["pool"][s])


@pytest.mark.gpu
def test_offsets_behind_32_bits():
    import gated_delta_rule_recurrent_b200 as gdr

    H, R, C = 64, 64, 512
    values = H * R * C
    P, N = 2 ** 31 // values + 2, 2 ** 31 // values + 3
    pool = torch.empty(P, H, R, C, dtype=torch.bfloat16, device="cuda")
    cache = torch.empty(N, H, R, C, dtype=torch.int8, device="cuda")
    scales = torch.empty(N, H, R, C // 64, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    pool[P - 1] = torch.randn(H, R, C, generator=gen, device="cuda")
    pool[0] = 0.0
    cache[0] = 5
    gdr.state_quantize(pool, i32([P - 1]), cache, scales, i32([N - 1]))
    codes, want = linear_oracle.quantize(pool[P - 1].float().cpu().numpy(), "int8")
    assert np.array_equal(cache[N - 1].cpu().numpy(), codes)
    assert np.array_equal(scales[N - 1].cpu().numpy(), want)
    gdr.state_dequantize(cache, scales, i32([N - 1]), pool, i32([P - 2]))
    back = linear_oracle.dequantize(codes, want, "int8")
    assert torch.equal(pool[P - 2].cpu(), torch.from_numpy(back).float().to(torch.bfloat16))
    assert not pool[0].any() and (cache[0] == 5).all()


@pytest.mark.gpu
def test_binding_refusals():
    import gated_delta_rule_recurrent_b200 as gdr

    x = make(3, 2, 2, 64, 64, "int8", device="cuda")
    one = i32([0])

    def both(pool=x["pool"], slots=one, cache=x["cache"], scales=x["scales"], entries=one):
        with pytest.raises(RuntimeError):
            gdr.state_quantize(pool, slots, cache, scales, entries)
        with pytest.raises(RuntimeError):
            gdr.state_dequantize(cache, scales, entries, pool, slots)

    both(pool=x["pool"].float())
    both(pool=x["pool"].transpose(2, 3))
    both(pool=x["pool"][0])
    both(cache=x["cache"].view(torch.uint8))
    both(cache=x["cache"][:, :1])
    both(scales=x["scales"].half())
    both(scales=x["scales"][:1])
    both(slots=one.long())
    both(entries=i32([0, 1]))
    both(entries=one.cpu())
    both(pool=x["pool"][..., :32].contiguous(), cache=x["cache"][..., :32].contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("kind,limit", [("int8", 0.01), ("e4m3", 0.03)])
@pytest.mark.parametrize("Dk,Dv", [(64, 192), (128, 128)])
def test_a_prompt_parked_and_resumed(Dk, Dv, kind, limit):
    """Prefill, park, restore into other slots (one of them twice: a fork), decode on; against
    the oracle on the whole sequence. The restored state is off by the codes' rounding, which
    for a code step of m/127 and values of m/3 rms is 1/127/sqrt(12)*3 = 0.7 % of the norm
    (int8) or at most 2^-4/sqrt(3) of each value, 2.6 % rms over a binade (e4m3)."""
    import gated_delta_rule_recurrent_b200 as gdr

    gen = torch.Generator().manual_seed(5)
    B, H, T, n = 2, 2, 180, 3

    def bf(*shape, by=1.0):
        return (by * torch.randn(*shape, generator=gen)).to(torch.bfloat16)

    q, k, v = bf(B, H, T + n, Dk), bf(B, H, T + n, Dk, by=Dk ** -0.5), bf(B, H, T + n, Dv)
    decay = torch.tensor([-0.01, -0.2])
    pool = torch.zeros(6, H, Dk, Dv, dtype=torch.bfloat16)
    whole = linear_oracle.linear_attention(f64(q), f64(k), f64(v), f64(decay), f64(pool),
                                           [T + n] * B, [0, 1], scale=0.125)[0]
    pool = pool.cuda()
    cache = torch.zeros(4, H, Dk, Dv, dtype=torch.int8, device="cuda").view(KINDS[kind])
    scales = torch.zeros(4, H, Dk, Dv // 64, device="cuda")

    def part(x, a, b, items):
        return x[items, :, a:b].contiguous().cuda()

    gdr.linear_attention_prefill(*(part(x, 0, T, [0, 1]) for x in (q, k, v)), decay.cuda(), pool,
                                 i32([T, T]), i32([0, 1]), 0.125)
    gdr.state_quantize(pool, i32([0, 1]), cache, scales, i32([3, 1]))
    gdr.state_dequantize(cache, scales, i32([3, 1, 3]), pool, i32([4, 2, 5]))
    items = [0, 1, 0]
    out, _ = gdr.linear_attention_decode(*(part(x, T, T + n, items) for x in (q, k, v)),
                                         decay.cuda(), pool, i32([n] * 3), i32([4, 2, 5]), None,
                                         0.125)
    assert torch.equal(out[0], out[2])
    ref = whole[items][:, :, T:]
    assert np.linalg.norm(f64(out) - ref) <= limit * np.linalg.norm(ref)
