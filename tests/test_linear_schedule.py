"""How a linear-attention prefill spreads its chunks over the SMs, on the CPU.

Compiles tests/native/linear_schedule.cu against the kernel's headers as a host program:
the plan of a call and every block's stretches of chunks come from the code that the host
and the kernel run. Checked: each chunk of each tile is worked on once; a state goes from
block to block in order, so that no two blocks wait for one another; and which of the ways
through the equal-shares mode a call takes, so that the GPU tests below reach all of them.
"""
import collections
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "gated_delta_rule_recurrent_b200")
SMS = 148
CHUNK = 128

Stretch = collections.namedtuple("Stretch", "block bh col0 c0 n L whole_start whole_end slot_row")
Plan = collections.namedtuple("Plan", "stream segments team grid seg_chunks")


@pytest.fixture(scope="session")
def schedule(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("schedule") / "linear_schedule")
    done = subprocess.run([nvcc, "-std=c++17", "-arch=sm_100a", "--expt-relaxed-constexpr",
                           "-I", os.path.join(PKG, "csrc"), "-I", os.path.join(ROOT, "include"),
                           "-o", exe, os.path.join(ROOT, "tests", "native", "linear_schedule.cu")],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr

    def run(shape, lengths=None, slots=None, sms=SMS):
        """(plan, stretches of every block in its order) of a call's shape
        (B, H_qk, H_v, T, D_k, D_v, pool) as in the GPU tests."""
        B, Hq, Hv, T, Dk, Dv, P = shape
        lengths = [T] * B if lengths is None else lengths
        slots = list(range(B)) if slots is None else slots
        args = [sms, B, Hq, Hv, Dk, Dv, T, P, *lengths, *slots]
        out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True)
        assert out.returncode == 0, out.stderr
        rows = [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
        return Plan(*rows[0]), [Stretch(*r) for r in rows[1:]]

    return run


def by_block(stretches):
    blocks = collections.defaultdict(list)
    for s in stretches:
        blocks[s.block].append(s)
    return blocks


def ways(stretches):
    """How often a block of the shares mode takes each of the orders that differ in what its
    state group has to wait for."""
    count = collections.Counter()
    for work in by_block(stretches).values():
        for k, s in enumerate(work):
            if not s.whole_start and not s.whole_end:
                count["receives and hands on"] += 1
            if k:
                if work[k - 1].whole_end and not s.whole_start:
                    count["stores a slot, then receives"] += 1
                if not work[k - 1].whole_end and not s.whole_start:
                    count["hands on, then receives"] += 1
                if not work[k - 1].whole_end and s.whole_start:
                    count["hands on, then starts from a slot"] += 1
    return count


# One item many chunks long, the others of no chunk or one: shares that lie inside one tile,
# whose block receives a state and hands it on.
SKEWED = [
    ((40, 2, 4, 3000, 64, 64, 41), [3000] + [(37 * b) % 129 for b in range(1, 40)]),
    ((20, 4, 8, 2600, 128, 128, 20), [100, 2600] + [b % 3 for b in range(2, 20)]),
    ((151, 1, 1, 20000, 128, 64, 151), [20000] + [b % 2 for b in range(1, 151)]),
    ((150, 1, 1, 15000, 64, 128, 150), [b % 2 for b in range(149)] + [15000]),
]
# Slightly more tiles than SMs: blocks that hand a state on and then receive one.
CHAINS = [((1, 150, 150, 1152, 64, 64, 1), [1152]), ((2, 76, 76, 1100, 128, 64, 3), [1100, 1024])]


def check(plan, stretches, shape, lengths):
    B, Hq, Hv, T, Dk, Dv, P = shape
    tiles = collections.defaultdict(list)
    for s in stretches:
        # from the slot: a tile's first stretch; of a tile in segments only where the block
        # has all of it, since nothing orders its load and another block's store
        assert s.n > 0
        assert s.whole_start == (s.c0 == 0 and (plan.segments == 1 or bool(s.whole_end)))
        tiles[s.bh, s.col0].append(s)
    for b, L in enumerate(lengths):
        L = min(max(L, 0), T)
        chunks = -(-L // CHUNK)
        for h in range(Hv):
            for col0 in range(0, Dv, 128):
                parts = sorted(tiles.pop((b * Hv + h, col0), []), key=lambda s: s.c0)
                # every chunk once, the parts in the order of the blocks
                at = 0
                for s in parts:
                    assert s.c0 == at and s.L == L - CHUNK * at
                    at += s.n
                    assert s.whole_end == (at == chunks)
                assert at == chunks
                step = plan.team if plan.stream else 1
                assert [s.block - parts[0].block for s in parts] == \
                    list(range(0, step * len(parts), step))
    assert not tiles
    for work in by_block(stretches).values():
        # a state is received by a block's last stretch and handed on by its first one: each
        # has one place for it, and nobody waits for a block that waits for it
        assert all(s.whole_start for s in work[:-1])
        assert all(s.whole_end for s in work[1:])


CASES = SKEWED + CHAINS + [
    ((8, 16, 32, 2048, 128, 128, 16), [2048, 1100, 1337, 1999, 1024, 1500, 1800, 1250]),
    ((4, 16, 16, 4001, 64, 512, 8), [4001, 2001, 3000, 3500]),
    ((9, 10, 20, 13, 128, 64, 9), [13, 0, -3, 18, 1, 2, 3, 4, 5]),
    ((4, 40, 40, 140, 128, 64, 4), [0, 0, 0, 0]),
    ((300, 1, 1, 10, 64, 64, 300), [10] * 300),
    ((2, 1, 2, 1700, 128, 192, 3), [1700, 900]),
    ((1, 8, 8, 32768, 128, 128, 2), [32768]),
    ((3, 1, 1, 2900, 64, 320, 3), [2900, 90, 0]),
]


@pytest.mark.parametrize("shape,lengths", CASES, ids=lambda v: str(v) if isinstance(v, tuple) else "")
def test_every_chunk_once_and_states_in_order(schedule, shape, lengths):
    plan, stretches = schedule(shape, lengths)
    check(plan, stretches, shape, lengths)


@pytest.mark.parametrize("team", [1, 2, 4, 8])
def test_shares_of_any_number_of_sms(schedule, team):
    lengths = [700, 1, 0, 129, 2000]
    shape = (5, 4, 4 * team, 2000, 64, 64, 5)
    for sms in (7, 20, 33, 64, 132, 148):
        plan, stretches = schedule(shape, lengths, sms=sms)
        check(plan, stretches, shape, lengths)


def test_the_cases_reach_every_way_through_the_shares(schedule):
    count = collections.Counter()
    for shape, lengths in SKEWED + CHAINS:
        plan, stretches = schedule(shape, lengths)
        assert plan.stream
        found = ways(stretches)
        if (shape, lengths) in SKEWED:
            assert found["receives and hands on"] > 0, shape
        count += found
    assert count["stores a slot, then receives"] >= 10
    assert count["hands on, then receives"] >= 100
    assert count["hands on, then starts from a slot"] > 0
