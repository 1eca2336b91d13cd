"""csrc/channel_plan.h on the host (CPU only): the sizes that the tests of the
per-channel product list take the forms they are listed for, every form has
one, and the model of the division of work restates what the code does."""
import random

import pytest

import channel_plan as cp
import test_channel_plan_model as model
from channel_forms import FORMS


@pytest.mark.parametrize("size", list(FORMS), ids=lambda s: "x".join(map(str, s)))
def test_listed_sizes_take_their_forms(size):
    """A constant of the rules that changes moves sizes to other forms: list
    others then, so that none of the forms loses its test."""
    assert cp.form(*size) == FORMS[size]


def test_every_form_is_listed():
    hows = ("direct", "sums", "shared2", "shared3", "shared4", "parts", "across")
    assert {("pair", T, how) for T in (64, 96, 128, 192) for how in hows} <= set(FORMS.values())
    assert {f[1:3] for f in FORMS.values() if f[0] == "stream"} == {(32, 8), (64, 8), (32, 16)}


@pytest.mark.parametrize("seed", range(4))
def test_the_model_is_the_code(seed):
    rng = random.Random(seed)
    for _ in range(500):
        M, N, K = int(2 ** rng.uniform(0, 12)), 8 * int(2 ** rng.uniform(0, 13)), 128 * int(2 ** rng.uniform(0, 10))
        p, m = cp.pair_plan(M, N, K), model.plan(M, N, K, 152)
        assert [p[k] for k in ("T", "TT", "F2", "G", "pairs", "band", "sk_tiles", "cost")] == \
            [m[k] for k in ("T", "TT", "F2", "G", "pairs", "band", "sk_tiles", "cost")]
        assert p["parts"] == m["cluster"] and (p["sk_pairs"] or 1) == m["sk_pairs"]
        assert p["part_bytes"] == m["parts"] * p["T"] * 128 * 4


@pytest.mark.parametrize("seed", range(4))
def test_workspace(seed):
    """Small batches and streamed ones need none; cut tiles their partials, and
    int8 codes in tiles their fp16 image."""
    rng = random.Random(seed)
    for _ in range(500):
        M, N, K = int(2 ** rng.uniform(0, 12)), 8 * int(2 ** rng.uniform(0, 13)), 128 * int(2 ** rng.uniform(0, 8))
        i8, c16 = cp.workspace_bytes(M, N, K, False), cp.workspace_bytes(M, N, K, True)
        if cp.streams(M, N, K):
            assert i8 == c16 == 0
            continue
        p = cp.pair_plan(M, N, K)
        assert c16 == (1024 + p["part_bytes"] if p["cut"] else 0) and i8 == c16 + 2 * M * K
    assert all(cp.streams(M, 248320, 17408) for M in range(1, 9))
