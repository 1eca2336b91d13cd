"""The operators around the paged cache at the ends of their contract: value
scales over fp32's whole range, long tails of small weights, scales that are not
finite, heads whose squares vanish, capped scores of either sign, and calls that
follow one another closely.

The attention's tolerance is that of tests/test_paged_cache.py, all of whose terms
hold here (n: the tokens of a row; a weight below fp16's normal range is at most a
step of 2^-24 off where the row's largest is 1 or more), and, for values near
fp32's end, half a step of a subnormal bf16, 2^-134, besides."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from helpers import from_dev_bits, to_dev, to_dev_bits
from test_paged_cache import Attn, Batch, D, attn_of, gpu, needs_gpu, random_cache, step_state, tolerance  # noqa: F401
from w4a16_linear_layers_gb300 import qlin

PAGE = 64


def one_head(x, vcodes, vs):
    """A cache of one head and consecutive pages, whose token j has the score x[j] under
    first() (exactly: its key's first code is 64, its scale x / 64) and codes and scale of
    its value."""
    n = len(x)
    pages = -(-n // PAGE)
    kcodes = np.full((pages * PAGE, D), 128, np.uint8)
    kcodes[:n, 0] = 128 + 64
    codes = np.full((pages * PAGE, D), 128, np.uint8)
    codes[:n] = vcodes + 128
    scales = np.zeros((2, pages * PAGE), np.float32)
    scales[0, :n], scales[1, :n] = np.asarray(x, np.float32) / 64, vs
    raw = np.zeros((pages * PAGE // 16, ref.BLOCK), np.uint8)
    for w, c in enumerate((kcodes, codes)):
        part = raw[:, 2048 * w:2048 * w + 2048]
        for r in range(16):
            part[:, ref.PLACES[r]] = c[r::16]
        raw[:, 4096 + 64 * w:4160 + 64 * w] = scales[w].reshape(-1, 16).view(np.uint8)
    return raw.reshape(pages, 1, PAGE // 16, ref.BLOCK)


def first(rows=1):
    """q whose only component, the first, is 1."""
    q = np.zeros((rows, D))
    q[:, 0] = 1.0
    return ref.bf16(q)


def expected(x, vcodes, vs):
    """(out, A, big) of a row that sees all."""
    x = np.asarray(x, np.float32).astype(np.float64)
    v = vcodes.astype(np.float64) * np.asarray(vs, np.float32).astype(np.float64)[:, None]
    p = np.exp(x - x.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), np.abs(v).max()


def attend(raw, n, B=1, **kw):
    """Rows of B sequences that all have the same pages."""
    table = np.broadcast_to(np.arange(raw.shape[0], dtype=np.int32), (B, raw.shape[0])).copy()
    out = qlin.paged_attn_i8(to_dev_bits(first(B), torch.bfloat16), to_dev(raw), to_dev(table), to_dev(np.full(B, n, np.int32)),
                             **{"scale": 1.0, **kw})
    return ref.bf16_to_f64(from_dev_bits(out))


def check_one_head(x, vcodes, vs, B=1):
    out = attend(one_head(x, vcodes, vs), len(x), B)
    o64, A, big = expected(x, vcodes, vs)
    bound = tolerance(o64, A, np.abs(x).max(), big, len(x)) + 2.0 ** -134
    bad = ~(np.abs(out - o64) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], out[bad][:4], np.broadcast_to(o64, out.shape)[bad][:4])


# ------------------------------------------------ value scales of every size

@needs_gpu
@pytest.mark.parametrize("B", [1, 40, 320])
@pytest.mark.parametrize("e", [-140, -120, -60, 0, 60, 96, 104, 110, 116, 120])
def test_value_scales_of_one_size(gpu, e, B):
    """One token of weight 2^13 among 8191 of weight 1, with the other sign, at the
    beginning, within and at the end."""
    rng = np.random.default_rng(e + 200)
    n = 8192
    for at in (0, 5000, n - 1):
        x = np.zeros(n)
        x[at] = 13 * np.log(2.0)
        codes = np.full((n, D), -100)
        codes[at] = 100
        codes[:, 64:] = rng.integers(-127, 128, (n, 64))
        check_one_head(x, codes, np.full(n, 2.0 ** e), B)


@needs_gpu
@pytest.mark.parametrize("order", ["random", "rising", "falling"])
@pytest.mark.parametrize("B", [1, 320])
def test_value_scales_of_all_sizes(gpu, B, order):
    """Small values count in the denominator beside large ones, in whatever order they come."""
    rng = np.random.default_rng(7)
    for n, low, high in ((3000, -110, 110), (700, -126, 120), (1500, -20, 118), (900, -120, 10), (129, -149, 60)):
        e = rng.uniform(low, high, n)
        if order != "random":
            e = np.sort(e) if order == "rising" else -np.sort(-e)
        check_one_head(3 * rng.standard_normal(n), rng.integers(-127, 128, (n, D)), 2.0 ** e, B)


@needs_gpu
@pytest.mark.parametrize("B", [1, 320])
@pytest.mark.parametrize("big", [1.0, 2.0 ** 60, 2.0 ** 120])
def test_values_of_zero_beside_large_ones(gpu, B, big):
    """Most tokens have values of zero (a scale of 0): they count in the denominator alone."""
    rng = np.random.default_rng(8)
    n = 2000
    for at in (0, 900, n - 1):
        vs = np.zeros(n)
        vs[at] = big
        check_one_head(rng.standard_normal(n), rng.integers(-127, 128, (n, D)), vs, B)


@needs_gpu
def test_values_written_and_read_by_attention_near_the_largest(gpu):
    """Heads that the write accepts at 2e37 give scales that the attention takes."""
    rng = np.random.default_rng(9)
    T, Hq, Hkv = 40, 4, 2
    x = rng.standard_normal((T, Hq + 2 * Hkv, D))
    x[:, Hq + Hkv:] = (x[:, Hq + Hkv:] * 2e37).clip(-3e38, 3e38)
    batch = Batch(10, 1, T, Hq, Hkv, 16, 3, [T], qkv=ref.bf16(x).reshape(T, -1))
    q = batch.run()
    batch.check(q)
    a = Attn(11, 1, T, Hq, Hkv, 16, 3, [T])
    a.raw, a.table, a.q = batch.cache.cpu().numpy(), batch.table, from_dev_bits(q)
    a.check(a.run())


@needs_gpu
@pytest.mark.parametrize("B", [1, 320])
@pytest.mark.parametrize("rise", [0.5, 0.9, 1.5])
def test_small_values_under_rising_scores(gpu, rise, B):
    """Two rows of a head.  The first one's scores rise by 16 powers of two every 128 tokens.
    The second sees tokens of values of ordinary size at a score of 0 all along, and others,
    whose scores rise slowly and whose values are 2^-100 of those: they count in its
    denominator alone, and the products of the others, the largest, keep their precision."""
    rng = np.random.default_rng(21)
    n = 60 * 128
    tile = np.arange(n) // 128
    slow = rng.random(n) < 0.3
    vs = np.where(slow, 2.0 ** -100, 1.0) / 64
    codes = rng.integers(-127, 128, (n, D))
    raw = one_head(np.full(n, 64 * 16 * np.log(2.0)), codes, vs)
    flat = raw.reshape(-1, ref.BLOCK)
    for d, c in ((0, tile), (1, np.where(slow, tile, 0))):
        for r in range(16):
            flat[:, ref.PLACES[r][d]] = 128 + c[r::16]
    q = np.zeros((B, 2, D))
    q[:, 0, 0], q[:, 1, 1] = 1.0, rise / 16
    q = ref.bf16(q.reshape(B, -1))
    table = np.broadcast_to(np.arange(raw.shape[0], dtype=np.int32), (B, raw.shape[0])).copy()
    out = qlin.paged_attn_i8(to_dev_bits(q, torch.bfloat16), to_dev(raw), to_dev(table), to_dev(np.full(B, n, np.int32)), scale=1.0)
    out = ref.bf16_to_f64(from_dev_bits(out)).reshape(B, 2, D)
    step = float(np.float32(16 * np.log(2.0)))
    q64 = ref.bf16_to_f64(q).reshape(B, 2, D)[0]
    for row, x in ((0, tile * step), (1, np.where(slow, tile, 0) * step * q64[1, 1])):
        o64, A, _ = expected(x, codes, vs)
        # (of what is rounded to steps each is 2^-24 of the largest product with a scale)
        p = np.exp(x - x.max())
        big = 127 * (p / p.sum() * vs).max()
        assert (np.abs(out[:, row] - o64) <= tolerance(o64, A, np.abs(x).max(), big, n)).all(), (row, out[0, row, :4], o64[:4])


# ------------------------------------------------------- small weights, many

@needs_gpu
@pytest.mark.parametrize("n,B", [(130, 1), (2657, 1), (2657, 320), (40001, 320), (131072, 320)])
def test_a_tail_of_small_weights(gpu, n, B):
    """A token that outweighs each of many alike by 2^gap, at the beginning: their sum
    is what components have in which that token has nothing, or the tail one sign."""
    rng = np.random.default_rng(n)
    for gap in (12.5, 15.3, 18.4, 20.7, 22.2, 24.0, 24.9, 25.5, 27.0):
        x = np.zeros(n)
        x[0] = gap * np.log(2.0)
        codes = np.full((n, D), 127)
        codes[0, :100] = 0
        codes[:, 20:40] = rng.integers(0, 128, (n, 20))
        codes[1:, 40:60] = rng.integers(0, 2, (n - 1, 1)) * 127
        for i, step in enumerate((2, 4, 8, 16, 32, 64)):       # few of the tokens, at regular places
            codes[1:, 60 + i] = 0
            codes[1 + i::step, 60 + i] = 127
        codes[1:, 66:100] *= -1
        codes[0, :100] = 0
        check_one_head(x, codes, np.full(n, 0.01), B)


@needs_gpu
@pytest.mark.parametrize("B", [1, 320])
def test_a_tail_that_falls_and_one_that_rises(gpu, B):
    """Weights over forty powers of two, the largest first or last."""
    n = 20000
    for slope in (1.0, -1.0):
        x = np.linspace(0, 40 * slope, n) * np.log(2.0)
        codes = np.full((n, D), 127)
        codes[:, 64:] = np.arange(n)[:, None] % 128
        codes[-1 if slope > 0 else 0, :32] = 0
        check_one_head(x, codes, np.full(n, 0.3), B)


# -------------------------------------------------- scales that are not finite

@needs_gpu
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("total", [100, 700])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_scales_that_are_not_finite_reach_the_rows_that_see_them(gpu, which, value, total, softcap):
    """A key's (0) or value's (1) at the third last token: the last three rows see it."""
    for seed in (1, 2, 3):
        a = Attn(seed, 1, 8, 4, 2, 16, 45, [total], softcap=softcap)
        clean = a.raw.copy()
        cache = ref.Cache(a.raw)
        codes, s = cache.get(a.table, 0, total - 3)
        s = s.copy()
        s[which] = value
        cache.put(a.table, 0, total - 3, codes, s)
        o = ref.bf16_to_f64(from_dev_bits(a.run()))
        assert not np.isfinite(o[5:]).any()
        o64, A, X, big, _ = ref.attention(ref.bf16_to_f64(a.q), ref.Cache(clean), a.table, a.total, a.T, softcap=softcap)
        assert (np.abs(o - o64) <= tolerance(o64, A, X, big, total))[:5].all()


# ------------------------------------------------------- heads of small numbers

@needs_gpu
@pytest.mark.parametrize("size", [2.0 ** -72, 2.0 ** -76, 2.0 ** -90, 2.0 ** -120])
def test_write_normed_heads_whose_squares_vanish(gpu, size):
    """eps alone is left under the root: 1 / sqrt(eps) for such heads."""
    rng = np.random.default_rng(12)
    for R in (0, 128):
        x = rng.standard_normal((8, 6 * D)) * size
        batch = Batch(13, 1, 8, 2, 2, 16, 2, [8], R=R, norm=True, eps=1e-6, qkv=ref.bf16(x))
        batch.check(batch.run())


@needs_gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("R", [0, 64, 128])
def test_query_heads_that_are_not_finite(gpu, R, value, norm):
    """NaN everywhere under a norm; else the component, with its partner in the rotation, and no other."""
    rng = np.random.default_rng(16)
    T, Hq = 6, 2
    x = rng.standard_normal((T, Hq + 2, D))
    at = [0, 31, 40, 64, 100, 127]
    x[np.arange(T), 0, at] = value
    batch = Batch(17, 1, T, Hq, 1, 16, 1, [T], R=R, norm=norm, qkv=ref.bf16(x).reshape(T, -1))
    q = ref.bf16_to_f64(from_dev_bits(batch.run())).reshape(T, Hq, D)
    with np.errstate(invalid="ignore"):
        want = list(batch.expect())
    for row, _, _, q64, S, _, _ in want:
        hit = np.zeros((Hq, D), bool)
        hit[0, at[row]] = True
        if at[row] < R:
            hit[0, (at[row] + R // 2) % R] = True
        if norm:
            hit[0] = True
        assert np.isnan(q[row][hit]).all() if norm else not np.isfinite(q[row][hit]).any()
        with np.errstate(invalid="ignore"):
            assert (np.abs(q[row] - q64) <= 2.0 ** -8 * np.abs(q64) + 2.0 ** -20 * S)[~hit].all()


# ---------------------------------------------------------------- capped scores

@needs_gpu
def test_capped_scores_are_odd(gpu):
    """Two tokens of opposite values under scores of either sign: the tanh of both signs
    is the same but for its sign, so outputs of q and -q are too, up to the roundings of
    the weights (at most 2^-11) and of the outputs."""
    rng = np.random.default_rng(14)
    B, cap = 4000, 2.0 ** 17
    x = -cap * rng.uniform(0.4, 1.5, B)
    raw = np.concatenate([one_head([s, s + d], np.array([[100] * D, [-100] * D]), [0.01, 0.01])[:, :, :1]
                          for s, d in zip(x, rng.uniform(-1.5, 1.5, B))])
    table = to_dev(np.arange(B, dtype=np.int32)[:, None])
    q = to_dev_bits(first(B), torch.bfloat16)
    o = [ref.bf16_to_f64(from_dev_bits(qlin.paged_attn_i8(t, to_dev(raw), table, to_dev(np.full(B, 2, np.int32)), scale=1.0, softcap=cap)))
         for t in (q, -q)]
    assert (np.abs(o[0]) < 0.9).any() and (np.abs(o[0]) > 0.1).any()
    bound = 2.0 ** -11 + 2.0 ** -8 * np.abs(o[0])
    assert (np.abs(o[0] + o[1]) <= bound).all(), np.abs(o[0] + o[1]).max()


@needs_gpu
def test_a_softcap_that_fp32_does_not_hold(gpu):
    """One below fp32's smallest number is refused and not taken as none."""
    s = attn_of(step_state(5))
    for cap in (1e-46, 1e-300):
        with pytest.raises(ValueError, match="softcap"):
            qlin.paged_attn_i8(s["q"], s["cache"], s["table"], s["total"], softcap=cap)
    qlin.paged_attn_i8(s["q"], s["cache"], s["table"], s["total"], softcap=1.5e-45)


# ------------------------------------------------- calls close behind one another

@needs_gpu
@pytest.mark.parametrize("before,T", [(512, 512), (512, 1), (4096, 64), (20000, 512)])
def test_reads_around_a_write(gpu, before, T):
    """A read, a write of tokens that it read and a read of those, one close behind the
    other: the last one gives what was written, whatever the first left in caches."""
    rng = np.random.default_rng(15)
    Hkv, page = 8, 64
    per = -(-before // page)
    cache = to_dev(random_cache(rng, per, Hkv, page))
    table = to_dev(rng.permutation(per).astype(np.int32)[None])
    total = to_dev(np.array([before], np.int32))
    start = total - T
    rows = [to_dev_bits(ref.bf16(rng.standard_normal((T, 2 * Hkv * D))), torch.bfloat16) for _ in range(2)]
    want = []
    for x in rows:
        qlin.kv_write_i8(x, cache, table, total, 0)
        torch.cuda.synchronize()
        want.append([t.clone() for t in qlin.kv_read_bf16(cache, table, total, T, start=start)])
        torch.cuda.synchronize()
    k, v = (torch.empty((1, before, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        if i % 10 == 0:
            torch.cuda._sleep(200_000)
        qlin.kv_read_bf16(cache, table, total, before, k=k, v=v)
        qlin.kv_write_i8(rows[i % 2], cache, table, total, 0)
        got = qlin.kv_read_bf16(cache, table, total, T, start=start)
        for g, w in zip(got, want[i % 2]):
            wrong += (g != w).any()
    assert int(wrong) == 0

# ------------------------------------------------ the ends of what scales may be

@needs_gpu
@pytest.mark.parametrize("B", [1, 320])
@pytest.mark.parametrize("size", [3.3e38, 2.0 ** 124, 2.0 ** -126])
def test_value_scales_at_the_very_ends(gpu, size, B):
    """Products that leave fp32's range where weights stand above 1: scores rise all along."""
    rng = np.random.default_rng(18)
    n = 4000
    check_one_head(np.linspace(0, 40, n), rng.integers(-1, 2, (n, D)), np.full(n, size), B)
    check_one_head(rng.standard_normal(n), rng.integers(-1, 2, (n, D)), np.where(rng.random(n) < 0.3, size, 1.0), B)


@needs_gpu
@pytest.mark.parametrize("B", [1, 320])
def test_negative_scales(gpu, B):
    """As the formula has them, although no write makes them."""
    rng = np.random.default_rng(19)
    n = 3000
    vs = np.exp(rng.standard_normal(n)) * rng.choice([-1.0, 1.0], n) / 90
    check_one_head(-4 + 3 * rng.standard_normal(n), rng.integers(-127, 128, (n, D)), vs, B)


@needs_gpu
@pytest.mark.parametrize("B", [1, 320])
@pytest.mark.parametrize("size", [1e28, 1e31, 1e36])
def test_scores_far_below_zero(gpu, size, B):
    """The largest is all that counts, however low it is: its value comes out."""
    rng = np.random.default_rng(20)
    for n in (3, 200, 5000):
        x = -size * (1.0 + 1e-3 * rng.permutation(n))
        codes = rng.integers(-127, 128, (n, D))
        out = attend(one_head(x, codes, np.full(n, 0.01)), n, B)
        want = codes[x.argmax()] * float(np.float32(0.01))
        assert (np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all()


# --------------------------------------------------------------- many new tokens

@needs_gpu
@pytest.mark.parametrize("T,Hq,Hkv,total,new,wide,kw", [
    # a prompt; one behind a prefix and padded; in a window, both ways
    (2000, 8, 2, 2000, 2000, 0, {}), (1500, 6, 2, 3300, 1471, 0, {}), (1500, 8, 2, 1700, 1500, 0, {"window": 300, "causal": False}),
    # row tiles past 2^16, with tables of any width
    (4100, 512, 1, 4100, 4100, 0, {"window": 500}), (4100, 512, 1, 1200, 1200, 60000, {}),
    # rows of a segment past 2^24
    (1100, 16384, 1, 1100, 1100, 0, {"window": 16})])
def test_many_new_tokens(gpu, T, Hq, Hkv, total, new, wide, kw):
    """Rows at both ends, at random and around every power of two of row tiles against
    binary64; padding as it was."""
    rng = np.random.default_rng(T + Hq)
    page = 64
    per = -(-total // page)
    raw = random_cache(rng, per, Hkv, page)
    table = rng.permutation(per).astype(np.int32)[None]
    cache = ref.Cache(raw)
    if wide:
        table = np.concatenate([table, np.full((1, wide), -1, np.int32)], 1)
    g = torch.Generator("cuda").manual_seed(T)
    q = torch.randn((T, Hq * D), generator=g, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(q, 7.0)
    qlin.paged_attn_i8(q, to_dev(raw), to_dev(table), to_dev(np.array([total], np.int32)), new_len=to_dev(np.array([new], np.int32)),
                       out=out, **kw)
    k, v, _ = cache.values(table, 0, 0, total)
    G = Hq // Hkv
    at = [0, new * G - 1] + [r + d for i in range(25) for r in (32 << i,) for d in (-1, 0) if r + d < new * G]
    at += list(rng.integers(0, new * G, 60))
    for r in at:
        t, h = r // G, int(rng.integers(0, Hkv)) * G + r % G
        i = total - new + t
        j = np.arange(total)
        see = (j <= i) | (not kw.get("causal", True))
        if kw.get("window"):
            see &= np.abs(i - j) < kw["window"]
        kk, vv = k[see, h // G], v[see, h // G]
        qr = q[t, h * D:(h + 1) * D].double().cpu().numpy()
        x = D ** -0.5 * (kk @ qr)
        p = np.exp(x - x.max())
        p /= p.sum()
        o64 = p @ vv
        X = D ** -0.5 * (np.abs(kk) @ np.abs(qr)).max()
        o = out[t, h * D:(h + 1) * D].double().cpu().numpy()
        assert (np.abs(o - o64) <= tolerance(o64, p @ np.abs(vv), X, np.abs(vv).max(), int(see.sum()))).all(), (r, t, h)
    assert bool((out[new:] == 7.0).all())
