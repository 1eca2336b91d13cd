"""Randomized checks of the per-channel product's mbarrier protocol (CPU only):
both blocks of a pair under random interleavings and orders of completion
(pair_model), and the same protocol with one of its rules taken out, which the
checks must see."""
import re

import pytest

import pair_model as pm
from w4a16_linear_layers_gb300 import build as qbuild

# K steps of a pair's segments: whole tiles, cut ones in front, chunks that end
# with the segment, one-step tiles, a single segment
SEGMENTS = [[40], [9, 40], [1], [1, 1, 1, 1, 1, 1, 1], [8, 8, 8], [3, 17, 17], [5, 31, 2], [16], [33, 1, 8]]


def failures(T, seeds, warps=1, segments=SEGMENTS, **change):
    out = {}
    for seg in segments:
        for seed in range(seeds):
            r = pm.run(T, seg, seed, warps=warps, **change)
            if r:
                out[tuple(seg)] = (seed, r)
                break
    return out


@pytest.mark.parametrize("T", sorted(pm.CONFIGS))
def test_no_deadlock_or_hazard(T):
    assert failures(T, 30) == {}


@pytest.mark.parametrize("T", [64, 192])
def test_no_deadlock_or_hazard_with_all_warps(T):
    assert failures(T, 2, warps=4, segments=[[9, 20], [3, 17, 2]]) == {}


@pytest.mark.parametrize("T", [64, 192])
@pytest.mark.parametrize("change", ["no_consumed", "no_dempty", "commit_to_one", "early_release"])
def test_a_missing_wait_or_commit_or_an_early_release_is_seen(T, change):
    assert failures(T, 30, segments=[[40], [3, 17, 17]], **{change: True}) != {}


def test_fewer_token_slots_than_a_buffers_break_the_protocol():
    """The wait for an A buffer is on the token slot's barrier, by parity: it
    would pass when the barrier is two phases behind."""
    assert failures(64, 30, segments=[[40]], kx=2) != {}


def test_the_counts_are_the_kernels():
    """What the kernel's source says of its rings."""
    with open(f"{qbuild.CSRC}/gemm_channel_pair.cuh") as f:
        text = f.read()

    def value(name):
        return re.search(rf"constexpr (?:int|uint32_t) {name} = ([^;]*);", text)[1]
    assert int(value("kA")) == pm.KA and int(value("kND")) == pm.ND
    assert int(value("kChunkK")) == 128 * pm.CHUNK
    assert value("kX") == "T == 192 ? 8 : 4" and value("kUnit") == "T == 192 ? 64 : 128"
    room = int(value("kSmemMax")) - 1024 - int(value("kCtrl"))
    for T, c in pm.CONFIGS.items():
        unit = T // 2 * (64 if T == 192 else 128) * 2
        assert c["nw"] == min(int(value("kMaxW")), (room - c["kx"] * unit) // (32 * 128 * 4) & ~1)
    for bar, count in (("ready", "9"), ("consumed", "1"), ("d_full", "1"), ("d_empty", "16"), ("wempty", "4")):
        assert re.search(rf"mbar_init\(smem_u32\(&ctrl->{bar}\[i\]\), {count}\);", text)
