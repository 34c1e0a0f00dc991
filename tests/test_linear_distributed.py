"""One linear-attention call split over ranks by item and by value head (CPU, gloo): each rank
runs the oracle on its share, and the gathered results equal the whole call's bit for bit."""
import os

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from oracle.linear_oracle import linear_attention
from test_distributed_gloo import _free_port


def _whole_call():
    """A ragged call: grouped heads, a decay of its own for each, an empty item, a slot outside
    the pool, committed counts below the lengths."""
    gen = torch.Generator().manual_seed(31)
    B, H_qk, H_v, T, D_k, D_v, P = 5, 2, 4, 6, 8, 8, 7
    r = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(query=r(B, H_qk, T, D_k), key=r(B, H_qk, T, D_k), value=r(B, H_v, T, D_v),
                log_decay=-torch.rand(H_v, generator=gen), state_pool=r(P, H_v, D_k, D_v),
                actual_seq_lengths=i32(6, 0, 3, 1, 5), ssm_state_indices=i32(4, 1, 99, 0, 6),
                num_accepted_tokens=i32(4, 0, 1, 1, 2), scale_value=0.3)


def _oracle(x):
    f = lambda t: t.to(torch.float64).numpy()  # noqa: E731
    return linear_attention(f(x["query"]), f(x["key"]), f(x["value"]), f(x["log_decay"]),
                            f(x["state_pool"]), x["actual_seq_lengths"].numpy(),
                            x["ssm_state_indices"].numpy(), x["num_accepted_tokens"].numpy(),
                            x["scale_value"])


def test_a_head_shard_has_its_heads_decays():
    from gated_delta_rule_recurrent_b200 import distributed as D

    x = _whole_call()
    for rank in range(2):
        share, shard = D.shard_call(x, 2, rank, by="head")
        assert torch.equal(share["log_decay"], x["log_decay"][shard.lo:shard.hi])
        assert share["log_decay"].is_contiguous()
        assert share["value"].shape[1] == share["log_decay"].shape[0]


@pytest.mark.parametrize("world", [1, 2])
def test_shares_of_a_call_put_together(world):
    from gated_delta_rule_recurrent_b200 import distributed as D

    x = _whole_call()
    want = _oracle(x)
    for by in ("item", "head"):
        outs, pools, shards = [], [], []
        for rank in range(world):
            share, shard = D.shard_call(x, world, rank, by=by)
            out, pool = _oracle(share)
            outs.append(torch.from_numpy(out))
            pools.append(torch.from_numpy(pool))
            shards.append(shard)
        out, pool = D.gather_call(outs, pools, shards, x["state_pool"].double())
        assert np.array_equal(out.numpy(), want[0]) and np.array_equal(pool.numpy(), want[1]), by


def _worker(rank, world, port, out_dir):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), WORLD_SIZE=str(world),
                      RANK=str(rank), LOCAL_RANK=str(rank))
    from datetime import timedelta

    from gated_delta_rule_recurrent_b200 import distributed as D

    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))
    try:
        x = _whole_call()
        results = {}
        for by in ("item", "head"):
            share, shard = D.shard_call(x, world, rank, by=by)
            out, pool = _oracle(share)
            parts = [None] * world
            dist.all_gather_object(parts, (torch.from_numpy(out), torch.from_numpy(pool), shard))
            results[by] = D.gather_call([p[0] for p in parts], [p[1] for p in parts],
                                        [p[2] for p in parts], x["state_pool"].double())
        torch.save(results, os.path.join(out_dir, f"linear{rank}.pt"))
        dist.barrier()
    finally:
        dist.destroy_process_group()


@pytest.mark.timeout(180)
def test_one_call_over_two_gloo_ranks(tmp_path):
    world = 2
    mp.start_processes(_worker, args=(world, _free_port(), str(tmp_path)), nprocs=world,
                       join=True, start_method="spawn")
    want = _oracle(_whole_call())
    for rank in range(world):
        for by, (out, pool) in torch.load(tmp_path / f"linear{rank}.pt").items():
            assert np.array_equal(out.numpy(), want[0]), by
            assert np.array_equal(pool.numpy(), want[1]), by
