"""Timing cases of the operators around a linear-attention layer with one decay per
head, and around the state pool that its layers share with the gated delta rule.

Three operators, each with a plain form (elementary torch operations in float32) and the
package's own call:

* ``prefill``: linear attention with a decay for each head over prompts,
  S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t, from and into the
  slots of a bf16 state pool.
* ``decode``: the same recurrence for one to eight new tokens of each sequence, with the
  committed count of speculative decoding.
* ``park`` / ``restore``: slots of the pool written to an 8-bit cache (one float32 scale
  for each 64 values) and read back into slots, as a prefix cache or a swapped-out
  sequence needs.

``own`` selects the side: False runs the plain forms, True the package's entry points.
"""
import math

import torch

own = False

_GROUP = 64  # values that share one scale of the 8-bit cache
_FLOOR = 2.0 ** -100  # a group whose largest magnitude is below this is held as zeros


def listed():
    return [
        # one sequence, one token: the latency of a chat with a single user
        dict(name="decode one sequence", kind="decode", B=1, Hq=64, Hv=64, T=1, Dk=64, Dv=512,
             pool=1),
        # a small batch with grouped heads out of a larger pool
        dict(name="decode grouped heads", kind="decode", B=64, Hq=16, Hv=32, T=1, Dk=128, Dv=128,
             pool=256),
        # speculative decoding: up to eight draft tokens, some of them accepted
        dict(name="decode eight drafts", kind="decode", B=128, Hq=32, Hv=32, T=8, Dk=128, Dv=128,
             pool=128),
        # the large-batch serving step, bound by the state's traffic
        dict(name="decode large batch", kind="decode", B=512, Hq=64, Hv=64, T=1, Dk=64, Dv=512,
             pool=512),
        # one short question
        dict(name="prefill short prompt", kind="prefill", B=1, Hq=16, Hv=32, T=97, Dk=128,
             Dv=128, pool=4),
        # a ragged batch of prompts with grouped heads
        dict(name="prefill ragged batch", kind="prefill", B=8, Hq=16, Hv=32, T=2048, Dk=128,
             Dv=128, pool=16),
        # one long document on one GPU of a tensor-parallel group: few heads, a long axis
        dict(name="prefill long document", kind="prefill", B=1, Hq=8, Hv=8, T=32768, Dk=128,
             Dv=128, pool=2),
        # narrow keys and wide values, a length that fills no whole block
        dict(name="prefill wide values", kind="prefill", B=4, Hq=16, Hv=16, T=4001, Dk=64,
             Dv=512, pool=8),
        # one sequence swapped out and back in
        dict(name="park one sequence", kind="park", n=1, H=64, R=64, C=512, pool=4, entries=2,
             bits="e4m3"),
        # a batch of sequences out of a larger pool, integer codes
        dict(name="park a batch", kind="park", n=64, H=32, R=128, C=128, pool=256, entries=100,
             bits="int8"),
        # half of a large pool
        dict(name="park half a pool", kind="park", n=256, H=64, R=64, C=512, pool=512,
             entries=256, bits="e4m3"),
        # a prefix cache's hits copied into the slots of new sequences
        dict(name="restore cached prefixes", kind="restore", n=96, H=64, R=64, C=512, pool=128,
             entries=60, bits="int8"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "park", "restore"])
    if kind in ("decode", "prefill"):
        Dk = rng.choice([64, 128])
        Dv = 64 * rng.randint(1, 8)
        group = rng.choice([1, 1, 2, 4])
        Hq = _log_int(rng, 1, 64 // group)
        Hv = Hq * group
        slot = Hv * Dk * Dv
        if kind == "decode":
            B = _log_int(rng, 1, max(1, min(512, (1 << 29) // slot)))
            T = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
            return dict(kind=kind, B=B, Hq=Hq, Hv=Hv, T=T, Dk=Dk, Dv=Dv,
                        pool=B + rng.randint(0, B))
        T = _log_int(rng, 1, max(2, min(32768, (1 << 25) // (Hv * Dv))))
        B = _log_int(rng, 1, max(1, min(16, (1 << 25) // (Hv * Dv * T))))
        return dict(kind=kind, B=B, Hq=Hq, Hv=Hv, T=T, Dk=Dk, Dv=Dv, pool=B + rng.randint(0, 4))
    R, C = rng.choice([(64, 64 * rng.randint(1, 8)), (128, 64 * rng.randint(1, 4)),
                       (64 * rng.randint(1, 8), 128)])
    H = _log_int(rng, 1, 64)
    n = _log_int(rng, 1, max(1, min(256, (1 << 28) // (H * R * C))))
    entries = n + rng.randint(0, n) if kind == "park" else rng.randint(max(1, n // 2), 2 * n)
    return dict(kind=kind, n=n, H=H, R=R, C=C, pool=2 * n + rng.randint(0, 3), entries=entries,
                bits=rng.choice(["e4m3", "int8"]))


def _cache_dtype(bits):
    return torch.float8_e4m3fn if bits == "e4m3" else torch.int8


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = case

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def perm(n, k):
        return torch.randperm(n, generator=gen, device=dev)[:k].to(torch.int32)

    def state(P, H, R, C):  # drawn a slot at a time: a large pool in float32 would not fit
        pool = torch.empty(P, H, R, C, dtype=torch.bfloat16, device=dev)
        for s in range(P):
            pool[s] = 0.1 * randn(H, R, C)
        return pool

    if c["kind"] in ("decode", "prefill"):
        B, Hq, Hv, T, Dk, Dv, P = (c[k] for k in ("B", "Hq", "Hv", "T", "Dk", "Dv", "pool"))

        def unit(x):
            return (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)

        low = 1 if c["kind"] == "decode" else (T + 1) // 2
        lengths = torch.randint(low, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        if B == 1:
            lengths.fill_(T)
        accepted = (torch.rand(B, generator=gen, device=dev) * (lengths + 1)).to(torch.int32)
        spread = torch.rand(Hv, generator=gen, device=dev)
        return dict(kind=c["kind"], query=unit(randn(B, Hq, T, Dk)), key=unit(randn(B, Hq, T, Dk)),
                    value=randn(B, Hv, T, Dv).to(torch.bfloat16),
                    # memories of 1 to 512 tokens, a different one for each head
                    log_decay=-torch.exp(-spread * math.log(512.0)),
                    state_pool=state(P, Hv, Dk, Dv), lengths=lengths, indices=perm(P, B),
                    accepted=accepted if c["kind"] == "decode" and T > 1 else None,
                    scale=Dk ** -0.5)
    n, H, R, C, P, N = (c[k] for k in ("n", "H", "R", "C", "pool", "entries"))
    kind = _cache_dtype(c["bits"])
    s = dict(kind=c["kind"], state_pool=state(P, H, R, C), slots=perm(P, P)[:n].contiguous())
    if c["kind"] == "park":
        s["back"] = perm(P, n)
        s["entries"] = perm(N, n)
        s["cache"] = torch.zeros(N, H, R, C, dtype=torch.int8, device=dev).view(kind)
        s["scales"] = torch.zeros(N, H, R, C // _GROUP, device=dev)
    else:  # several new sequences may start from the same cached prefix
        s["entries"] = torch.randint(0, N, (n,), generator=gen, device=dev, dtype=torch.int32)
        s["cache"] = torch.empty(N, H, R, C, dtype=torch.int8, device=dev).view(kind)
        s["scales"] = torch.empty(N, H, R, C // _GROUP, device=dev)
        for e in range(N):
            codes, scale = _quantize(0.1 * randn(H, R, C), kind)
            s["cache"].view(torch.int8)[e] = codes.view(torch.int8)
            s["scales"][e] = scale
    return s


# ------------------------------------------------------------------ plain forms


def _quantize(x, kind):
    """8-bit codes and float32 scales of float32 values, one scale for each 64 of a row."""
    top = 448.0 if kind == torch.float8_e4m3fn else 127.0
    g = x.unflatten(-1, (-1, _GROUP))
    most = g.abs().amax(-1)
    some = most >= _FLOOR
    factor = torch.where(some, top / most, torch.zeros_like(most))
    scale = torch.where(some, most / top, torch.zeros_like(most))
    y = g * factor[..., None]
    codes = y.to(kind) if kind == torch.float8_e4m3fn else y.round().to(kind)
    return codes.flatten(-2), scale


def _dequantize(codes, scale):
    x = codes.float().unflatten(-1, (-1, _GROUP)) * scale[..., None]
    return x.flatten(-2).to(torch.bfloat16)


def _plain_decode(s):
    q, k, v, pool = s["query"], s["key"], s["value"].float(), s["state_pool"]
    group = v.shape[1] // q.shape[1]
    q = q.float().repeat_interleave(group, 1)
    k = k.float().repeat_interleave(group, 1)
    T = q.shape[2]
    t = torch.arange(T, device=q.device)
    length = s["lengths"][:, None]
    kept = length if s["accepted"] is None else torch.minimum(s["accepted"][:, None], length)
    g = s["log_decay"][:, None]
    live = (t < length)[:, None, :, None]
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    apart = t[:, None] - t[None, :]
    mask = torch.where(apart >= 0, torch.exp(g[:, :, None] * apart.clamp(min=0)), 0.0)
    start = pool[s["indices"]].float()
    out = (q @ k.transpose(-1, -2) * mask) @ v
    out += torch.exp(g * (t + 1))[..., None] * (q @ start)
    weight = torch.exp(g * (kept - 1 - t).clamp(min=0)[:, None, :]) * (t < kept)[:, None, :]
    start *= torch.exp(g * kept[:, None, :])[..., None]
    start += (k * weight[..., None]).transpose(-1, -2) @ v
    pool[s["indices"]] = start.to(torch.bfloat16)
    return torch.where(live, out * s["scale"], 0.0).to(torch.bfloat16), pool


def _plain_prefill(s):
    """The recurrence in blocks of 64 tokens: products inside a block, and one matrix over
    the blocks for what each of them starts from."""
    q, k, v, pool = s["query"], s["key"], s["value"].float(), s["state_pool"]
    group = v.shape[1] // q.shape[1]
    B, H, T, Dv = v.shape
    Dk = q.shape[3]
    W = 64
    N = -(-T // W)
    t = torch.arange(T, device=q.device)
    length = s["lengths"][:, None]
    live = (t < length)[:, None, :, None]
    v = torch.where(live, v, 0.0)
    k = torch.where(live, k.float().repeat_interleave(group, 1), 0.0)
    q = q.float().repeat_interleave(group, 1)
    g = s["log_decay"]
    start = pool[s["indices"]].float()
    weight = torch.exp(g[:, None] * (length - 1 - t).clamp(min=0)[:, None, :])
    final = torch.exp(g[:, None, None] * length[:, None, None]) * start
    final += (k * weight[..., None]).transpose(-1, -2) @ v

    def blocks(x):
        return torch.nn.functional.pad(x, (0, 0, 0, N * W - T)).unflatten(2, (N, W))

    q, k, v = blocks(q), blocks(k), blocks(v)
    i = torch.arange(W, device=q.device)
    apart = i[:, None] - i[None, :]
    mask = torch.where(apart >= 0, torch.exp(g[:, None, None] * apart.clamp(min=0)), 0.0)
    out = (q @ k.transpose(-1, -2) * mask[:, None]) @ v
    fall = torch.exp(g[:, None] * (W - 1 - i))[:, None, :, None]
    added = (k * fall).transpose(-1, -2) @ v
    begun = torch.cat([start[:, :, None], added[:, :, :-1]], 2).flatten(3)
    n = torch.arange(N, device=q.device)
    over = (n[:, None] - n[None, :]) * W
    carry = torch.where(over >= 0, torch.exp(g[:, None, None] * over.clamp(min=0)), 0.0)
    begun = (carry @ begun).unflatten(3, (Dk, Dv))
    out += torch.exp(g[:, None] * (i + 1))[:, None, :, None] * (q @ begun)
    out = out.flatten(2, 3)[:, :, :T]
    pool[s["indices"]] = final.to(torch.bfloat16)
    return torch.where(live, out * s["scale"], 0.0).to(torch.bfloat16), pool


def _plain_park(s):
    kind = s["cache"].dtype
    codes, scale = _quantize(s["state_pool"][s["slots"]].float(), kind)
    s["cache"].view(torch.int8)[s["entries"]] = codes.view(torch.int8)
    s["scales"][s["entries"]] = scale


def _plain_restore(s, slots):
    codes = s["cache"].view(torch.int8)[s["entries"]].view(s["cache"].dtype)
    s["state_pool"][slots] = _dequantize(codes, s["scales"][s["entries"]])


def run(state):
    s = state
    if own:
        import gated_delta_rule_recurrent_b200 as gdr

        if s["kind"] == "decode":
            return gdr.linear_attention_decode(
                s["query"], s["key"], s["value"], s["log_decay"], s["state_pool"], s["lengths"],
                s["indices"], s["accepted"], s["scale"])
        if s["kind"] == "prefill":
            return gdr.linear_attention_prefill(
                s["query"], s["key"], s["value"], s["log_decay"], s["state_pool"], s["lengths"],
                s["indices"], s["scale"])
        if s["kind"] == "park":
            gdr.state_quantize(s["state_pool"], s["slots"], s["cache"], s["scales"], s["entries"])
            gdr.state_dequantize(s["cache"], s["scales"], s["entries"], s["state_pool"],
                                 s["back"])
            return s["state_pool"], s["scales"]
        return gdr.state_dequantize(s["cache"], s["scales"], s["entries"], s["state_pool"],
                                    s["slots"])
    if s["kind"] == "decode":
        return _plain_decode(s)
    if s["kind"] == "prefill":
        return _plain_prefill(s)
    if s["kind"] == "park":
        _plain_park(s)
        _plain_restore(s, s["back"])
        return s["state_pool"], s["scales"]
    _plain_restore(s, s["slots"])
    return s["state_pool"]


def work(case):
    c = case
    if c["kind"] in ("decode", "prefill"):
        B, Hq, Hv, T, Dk, Dv = (c[k] for k in ("B", "Hq", "Hv", "T", "Dk", "Dv"))
        # mean valid tokens of a sequence; the padding of the output is written as zeros
        full = float(T)
        if B > 1:
            full = (T + 1) / 2 if c["kind"] == "decode" else 0.75 * T
        rows = 2 * (2 * Hq * Dk + Hv * Dv) * full + 2 * Hv * Dv * T
        states = 2 * 2 * Hv * Dk * Dv
        # the state's update and its product with the query, for each token
        return {"bytes": B * (rows + states) + 4.0 * Hv + 12.0 * B,
                "flops": 4.0 * B * Hv * full * Dk * Dv}
    values = float(c["n"] * c["H"] * c["R"] * c["C"])
    packed = values * (1 + 4 / _GROUP)
    if c["kind"] == "park":
        return {"bytes": 2 * (2 * values + packed), "flops": 4 * values}
    return {"bytes": min(1.0, c["entries"] / c["n"]) * packed + 2 * values, "flops": values}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] in ("decode", "prefill"):
        pool = s["state_pool"]
        q, k, v = (s[n].double() for n in ("query", "key", "value"))
        B, H, T, Dv = v.shape
        head = torch.arange(H, device=v.device) // (H // q.shape[1])
        q, k = q[:, head] * s["scale"], k[:, head]
        decay = torch.exp(s["log_decay"].double())[None, :, None, None]
        live = pool[s["indices"]].double()
        kept = live.clone()
        length, count = s["lengths"], s["lengths"] if s["accepted"] is None else s["accepted"]
        out = torch.zeros(B, H, T, Dv, dtype=torch.float64, device=v.device)
        # a token at a time, as the recurrence is written; past an item's length nothing moves
        every = bool((length == T).all()) and s["accepted"] is None
        for t in range(T):
            if every:
                live.mul_(decay)
                live.add_(k[:, :, t, :, None] * v[:, :, t, None, :])
                out[:, :, t] = (q[:, :, t, None, :] @ live)[:, :, 0]
                continue
            on = (t < length).view(B, 1, 1, 1)
            live = torch.where(on, decay * live + k[:, :, t, :, None] * v[:, :, t, None, :], live)
            out[:, :, t] = torch.where(on[..., 0], (q[:, :, t, None, :] @ live)[:, :, 0], 0.0)
            if s["accepted"] is not None:
                kept = torch.where((t < torch.minimum(count, length)).view(B, 1, 1, 1), live, kept)
        del q, k, v
        if s["accepted"] is None:
            kept = live
        whole = pool.double()
        whole[s["indices"]] = kept
        return out, whole
    kind = s["cache"].dtype
    top, dense = (448.0, True) if kind == torch.float8_e4m3fn else (127.0, False)
    pool = s["state_pool"].double()
    if s["kind"] == "restore":
        codes = s["cache"].float().double()
        values = codes * s["scales"].double().repeat_interleave(_GROUP, -1)
        pool[s["slots"]] = values[s["entries"]]
        return pool
    scales = s["scales"].double()
    x = pool[s["slots"]]
    shape = x.shape
    x = x.view(*shape[:-1], shape[-1] // _GROUP, _GROUP)
    scale = x.abs().max(-1, keepdim=True).values / top
    x = x / torch.where(scale > 0, scale, torch.ones_like(scale))
    if dense:  # three bits behind the leading one, down to a step of 2^-9
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        x = torch.round(x / step) * step
    else:
        x = torch.round(x)
    scales[s["entries"]] = scale[..., 0]
    pool[s["back"]] = (x * scale).view(shape)
    return pool, scales
