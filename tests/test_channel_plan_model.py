"""The per-channel product's division of work, modelled on the host: the plan of
csrc/gemm_channel.cu (plan_pair) and the segments each pair of blocks derives
from it (struct Work in csrc/gemm_channel_pair.cuh), restated here.  Checked
for many shapes: every K step of every tile belongs to exactly one pair, a pair
shares at most two tiles with others, the contributors that a finishing block
expects are those that exist, their partials' slots differ, and every counter
and partial lies inside the workspace."""
import random

import pytest

SIZES = [(64, 38, 170, 330), (96, 43, 210, 400), (128, 47, 250, 450), (192, 56, 320, 560)]
MIN_SHARE = 8
COUNTERS = 256
ROOM = {2: 36, 3: 23, 4: 15}     # clusters of so many pairs on 152 SMs


def plan_tiles(size, M, N, K, sm_count):
    T, step, out, base = size
    slots, F2, TT, G = sm_count // 2, -(-N // 256), -(-M // T), K // 128
    tiles = TT * F2
    rounds, rest = divmod(tiles, slots)
    p = dict(T=T, TT=TT, F2=F2, G=G, pairs=min(tiles, slots), band=min(TT, 8), sk_tiles=0, sk_pairs=1, parts=0,
             cluster=1)
    whole = max(step * G, out)
    last = whole if rest else 0
    if rest and rest * 8 < slots * 7:
        most = slots // rest
        n = rest * min(most, G // MIN_SHARE) if most >= 2 else slots
        if n * MIN_SHARE > rest * G:
            n = rest * G // MIN_SHARE
        if n > rest:
            cut = step * -(-rest * G // n) + (150 if rounds else 480 + 45 * -(-n // rest) * T // 64)
            if cut < last:
                p.update(sk_tiles=rest, sk_pairs=n, parts=n * 4, pairs=max(p["pairs"], n))
                last = cut
    for c, room in ROOM.items():
        shared = step * -(-G // c) + 200
        if c * MIN_SHARE <= G and tiles * 152 <= room * sm_count and shared < last:
            p.update(cluster=c, sk_tiles=tiles, sk_pairs=tiles * c, pairs=tiles * c, parts=0)
            last = shared
    p["cost"] = base + whole * rounds + last
    return p


def plan(M, N, K, sm_count):
    return min((plan_tiles(size, M, N, K, sm_count) for size in SIZES), key=lambda p: p["cost"])


def segments(p, pair):
    """(tile of the whole order, g0, g1, cut tile or None) of one pair."""
    W, n, G = p["sk_tiles"] * p["G"], p["sk_pairs"], p["G"]
    whole = p["F2"] * p["TT"] - p["sk_tiles"]
    s, s1 = (pair * W // n, (pair + 1) * W // n) if pair < n else (0, 0)
    out = []
    while s < s1:
        tile = s // G
        g0 = s - tile * G
        g1 = min(G, g0 + s1 - s)
        s += g1 - g0
        out.append((whole + tile, g0, g1, tile if g1 - g0 != G else None))
    out += [(q, 0, G, None) for q in range(pair, whole, p["pairs"])]
    return out


def place(p, i):
    b, r = divmod(i, p["band"] * p["F2"])
    rows = min(p["TT"] - b * p["band"], p["band"])
    return r // rows, b * p["band"] + r % rows


def check(M, N, K, sm_count=152):
    p = plan(M, N, K, sm_count)
    G, tiles, W, n = p["G"], p["F2"] * p["TT"], p["sk_tiles"] * p["G"], p["sk_pairs"]
    seen, contributors = set(), {}
    for pair in range(p["pairs"]):
        cut = 0
        for tile, g0, g1, shared in segments(p, pair):
            for g in range(g0, g1):
                assert (tile, g) not in seen
                seen.add((tile, g))
            if shared is not None:
                cut += 1
                if p["cluster"] > 1:     # its one segment, of the cluster's tile
                    assert shared == pair // p["cluster"] and cut == 1
                    continue
                first = pair * W // n // G
                slot = pair * 2 + (0 if first == shared else 1)
                assert 0 <= slot * 2 + 1 < p["parts"]
                contributors.setdefault(shared, []).append((pair, slot))
        assert cut <= 2
    assert len(seen) == tiles * G

    if p["cluster"] > 1:
        assert all(len(segments(p, pair)) == 1 for pair in range(p["pairs"]))
        return p

    def pair_of_step(i):
        return ((i + 1) * n + W - 1) // W - 1
    slots = [c[1] for cs in contributors.values() for c in cs]
    assert len(set(slots)) == len(slots)
    for tile in range(p["sk_tiles"]):
        c0, c1 = pair_of_step(tile * G), pair_of_step(tile * G + G - 1)
        expect = list(range(c0, c1 + 1)) if c1 > c0 else []
        assert [c[0] for c in contributors.get(tile, [])] == expect
    assert p["sk_tiles"] * 2 <= COUNTERS
    assert {place(p, i) for i in range(tiles)} == {(f, t) for f in range(p["F2"]) for t in range(p["TT"])}
    return p


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(seed):
    rng = random.Random(seed)
    for _ in range(60):
        M = int(2 ** rng.uniform(0, 11.5))
        N = 8 * int(2 ** rng.uniform(0, 11))
        K = 128 * int(2 ** rng.uniform(0, 7.5))
        check(M, N, K, rng.choice([152, 152, 148, 160]))


@pytest.mark.parametrize("M,N,K", [(96, 248320, 5120), (509, 5120, 17408), (8192, 34816, 5120), (96, 1024, 5120),
                                   (9, 8, 128), (200, 19456, 1152), (77, 12800, 1280), (1, 256, 130944)])
def test_named_shapes(M, N, K):
    p = check(M, N, K)
    assert p["pairs"] <= 76
