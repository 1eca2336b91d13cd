"""The operators around the paged INT8 key/value cache, against their
definitions in binary64 (tests/paged_ref.py).

Tolerances, from the definitions of include/qlin.h:
  * codes: equal.  The binary64 quotient 127 y / a is off by less than 2^-44; a
    quotient nearer than that to a half-integer without being one does not
    occur by chance.
  * scales: a * rho / 127 in fp32: y two products and a sum (2.42 half steps of
    a, the products of a rotation being at most sqrt(2) a), the mean of 128
    squares plus eps under rho (half of at most 13 half steps), its root (two
    ulps: 4), two products (2, and 1/127 in fp32 is 2^-28 off): below 15 half
    steps of 2^-24, held to 2^-20; subnormal ones are half a step of 2^-149 off
    besides.
  * q: the same sums, whose terms' magnitudes S = |u c| + |u' s| (times rho)
    carry them, then the rounding to bf16 (2^-8 of the value):
    |q - q64| <= 2^-8 |q64| + 2^-20 S + 2^-134 (half a step of subnormal bf16).
  * cache values read: bf16 of the fp32 product: equal.
  * attention, with A = sum_j p_j |V_j|, X = the largest sum of a score's terms'
    magnitudes and n tokens: a score's 128 exact products are added in fp32
    (at most 128 * 2^-23 X = 2^-16 X off, the tensor cores truncate), its
    factors and the exponent's argument add 2^-21 X, the exponential 2^-21 of
    its value; the weight's rounding to fp16 2^-11 of it; numerator and
    denominator each carry that, and sums of n terms in fp32, 4 sqrt(n) 2^-23
    of A (Higham and Mary, as in tests/helpers.py); a row's largest weight is
    2^-1 or more in fp16's units (its reference puts a power of two above it at
    2^0), so the weights below its normal range (2^-14), off by half a step of
    2^-24, are off by at most 2^-24 of the largest, times a code of at most 127
    by 2^-24 of the largest |V|, n of them by n of that at most and, as roundings
    of either sign, by 4 sqrt(n) of it; then bf16's rounding:
    |o - o64| <= 2^-8 |o64| + (2^-11 + 2 (2^-16 X + 2^-20) + 4 sqrt(n) 2^-23) A
                 + min(n, 4 sqrt(n)) 2^-24 max|V|, all but the first term times 1.05."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import paged_ref as ref
from helpers import from_dev_bits, to_dev, to_dev_bits
from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin, synth

needs_gpu = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qlin.load()
    assert qlin.device_status() == qlin.QLIN_OK
    yield torch.device("cuda")
    torch.cuda.synchronize()
    assert qlin.device_status() == qlin.QLIN_OK


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qlin.load()


# ----------------------------------------------------------------- batches

def make_table(rng, B, per, pages):
    """int32 [B, per]: different pages in random order."""
    assert B * per <= pages
    return rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)


def random_cache(rng, pages, kv_heads, page, spread=0.5):
    """Codes of all values, scales of unequal size."""
    raw = np.empty((pages, kv_heads, page // 16, ref.BLOCK), np.uint8)
    raw[..., :4096] = rng.integers(1, 256, raw[..., :4096].shape)
    s = np.exp(spread * rng.standard_normal((pages, kv_heads, page // 16, 32))) / 90.0
    raw[..., 4096:] = s.astype(np.float32).view(np.uint8)
    return raw


def cos_sin(P, R, theta=1e4):
    angle = np.arange(P)[:, None] * theta ** (-np.arange(0, R, 2) / R)[None, :]
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


class Batch:
    """A batch of rows for kv_write, on the host and on the device."""

    def __init__(self, seed, B, T, Hq, Hkv, page, per, total, new=None, R=128, A=0, norm=True, eps=1e-6, qkv=None, P=None):
        rng = np.random.default_rng(seed)
        self.B, self.T, self.Hq, self.Hkv, self.page = B, T, Hq, Hkv, page
        self.total, self.new = np.asarray(total, np.int32), None if new is None else np.asarray(new, np.int32)
        pages = B * per + 2
        self.table = make_table(rng, B, per, pages)
        self.raw = random_cache(rng, pages, Hkv, page)
        x = rng.standard_normal((B * T, (Hq + 2 * Hkv) * D)) * np.exp(0.5 * rng.standard_normal((Hq + 2 * Hkv) * D))
        self.qkv = ref.bf16(x) if qkv is None else qkv
        self.kw = {"eps": eps}
        if norm:
            self.kw["q_gamma"] = ref.bf16(1.0 + 0.2 * rng.standard_normal(D))
            self.kw["k_gamma"] = ref.bf16(1.0 + 0.2 * rng.standard_normal(D))
        if R:
            self.kw["cos_sin"] = cos_sin(per * page if P is None else P, R)
            if A:
                self.kw["positions"] = rng.integers(-3, self.kw["cos_sin"].shape[0] + 3, (A, B * T)).astype(np.int32)
                if A > 1:
                    self.kw["axes"] = rng.integers(0, A + 2, R // 2).astype(np.uint8)

    def run(self, q=None, **more):
        kw = {k: to_dev_bits(v, torch.bfloat16) if k.endswith("gamma") else to_dev(v) if isinstance(v, np.ndarray) else v
              for k, v in self.kw.items()}
        self.cache = to_dev(self.raw)
        if q is None:
            q = torch.full((self.B * self.T, self.Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
        got = qlin.kv_write_i8(to_dev_bits(self.qkv, torch.bfloat16), self.cache, to_dev(self.table), to_dev(self.total),
                               self.Hq, new_len=None if self.new is None else to_dev(self.new), q=q, **kw, **more)
        assert got.data_ptr() == q.data_ptr()
        torch.cuda.synchronize()
        return q

    def expect(self):
        kw = {k: ref.bf16_to_f64(v) if k.endswith("gamma") else v for k, v in self.kw.items()}
        kw["eps"] = float(np.float32(kw["eps"]))
        return ref.write(ref.bf16_to_f64(self.qkv), ref.Cache(self.raw.copy()), self.table, self.total, self.Hq, self.T,
                         new=self.new, **kw)

    def check(self, q):
        q = ref.bf16_to_f64(from_dev_bits(q)).reshape(self.B * self.T, self.Hq, D)
        after = ref.Cache(self.cache.cpu().numpy().copy())
        padding = np.ones(self.B * self.T, bool)
        n = 0
        for row, b, pos, q64, size, codes, scales in self.expect():
            padding[row] = False
            n += 1
            if self.Hq:
                assert (np.abs(q[row] - q64) <= 2.0 ** -8 * np.abs(q64) + 2.0 ** -20 * size + 2.0 ** -134).all(), (row, "q")
            got = after.get(self.table, b, pos)
            if got is None:
                continue
            assert np.array_equal(got[0], codes), (row, np.argwhere(got[0] != codes)[:4])
            assert (np.abs(got[1] - scales) <= 2.0 ** -20 * scales + 2.0 ** -149).all(), (row, "scale")
            # put back what was there: everything else is as it was
            before = ref.Cache(self.raw).get(self.table, b, pos)
            after.put(self.table, b, pos, *before)
        assert np.array_equal(after.raw, self.raw)
        assert (q[padding] == 7.0).all()
        return n


# ------------------------------------------------------------------- write

@needs_gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,page,R,A,norm", [
    (1, 1, 32, 8, 16, 128, 0, True), (1, 1, 1, 1, 16, 0, 0, False), (2, 3, 5, 1, 16, 16, 1, True), (3, 8, 4, 2, 32, 64, 0, False),
    (1, 17, 0, 3, 48, 128, 0, True), (2, 5, 7, 7, 64, 96, 3, True), (12, 8, 32, 8, 16, 128, 0, True), (1, 40, 2, 1, 16, 32, 2, False),
    (5, 1, 28, 4, 1024, 112, 4, True), (1, 300, 6, 2, 16, 128, 0, True), (40, 9, 16, 8, 16, 128, 0, True), (2, 200, 40, 8, 16, 48, 0, True)])
def test_write(gpu, B, T, Hq, Hkv, page, R, A, norm):
    per = -(-(T + 40) // page)
    rng = np.random.default_rng(B * T)
    total = T + rng.integers(0, 41, B)
    batch = Batch(B + T + R, B, T, Hq, Hkv, page, per, total, R=R, A=A, norm=norm)
    assert batch.check(batch.run()) == B * T


@needs_gpu
@pytest.mark.parametrize("T,Hq,Hkv,R,norm", [
    # heads as they come, many ties, heads of a kind that leave lanes without one
    (200, 3, 5, 0, False), (90, 2, 6, 0, True), (60, 5, 3, 16, False),
    # a warp through several groups of a row: of one kind, of two, of all three
    (1300, 7, 5, 128, True), (2600, 9, 1, 64, True), (5200, 6, 2, 0, False)])
def test_write_long(gpu, T, Hq, Hkv, R, norm):
    batch = Batch(T, 1, T, Hq, Hkv, 64, -(-T // 64), [T], R=R, norm=norm)
    assert batch.check(batch.run()) == T


@needs_gpu
def test_write_padded_rows_and_lengths_outside_the_table(gpu):
    """new_len below 0, above T and above the sequence; total_len below 0 and above the table."""
    total = [20, 5, 3, 70, -4, 64, 2 ** 31 - 1, 9, 0]
    new = [4, 0, 6, 6, 3, -1, 2, 2 ** 31 - 1, 1]
    batch = Batch(3, 9, 6, 4, 2, 16, 4, total, new=new)
    assert batch.check(batch.run()) == 4 + 0 + 3 + 6 + 0 + 0 + 2 + 6 + 0
    batch = Batch(4, 9, 6, 4, 2, 16, 4, total)
    assert batch.check(batch.run()) == 6 + 5 + 3 + 6 + 0 + 6 + 6 + 6 + 0


@needs_gpu
def test_write_drops_what_is_on_no_page(gpu):
    batch = Batch(5, 4, 20, 2, 2, 16, 3, [20, 40, 36, 48])
    pages = batch.raw.shape[0]
    batch.table[0, 0], batch.table[1, 1], batch.table[2, 2], batch.table[3, 1] = -1, pages, 2 ** 31 - 1, -2 ** 31
    assert batch.check(batch.run()) == 80


@needs_gpu
def test_write_codes_at_ties(gpu):
    """Halves of the largest component are ties between 63 and 64: the even one,
    under a norm and where a rotation by nothing leaves them."""
    rng = np.random.default_rng(6)
    B, T, Hq, Hkv = 1, 64, 2, 4
    x = rng.standard_normal((T, (Hq + 2 * Hkv), D))
    x[..., 5] = 4.0 * np.sign(x[..., 5])
    x[..., 40:60] = rng.choice([-2.0, 2.0, 1.0], x[..., 40:60].shape)
    x[..., 100] = 4.0 * 61 / 254          # near one, not on it
    for R, norm in ((0, False), (0, True), (16, True), (128, False)):
        batch = Batch(7, B, T, Hq, Hkv, 16, 8, [T], R=R, norm=norm, qkv=ref.bf16(x).reshape(T, -1))
        if norm:
            batch.kw["k_gamma"] = ref.bf16(np.full(D, 1.5))
        if R:
            batch.kw["cos_sin"] = np.concatenate([np.ones((128, R // 2)), np.zeros((128, R // 2))], 1).astype(np.float32)
        batch.check(batch.run())


@needs_gpu
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-15, 1e15, 1e30, 2e37])
def test_write_small_and_large_heads(gpu, size):
    rng = np.random.default_rng(8)
    x = (rng.standard_normal((8, 6 * D)) * size).clip(-3e38, 3e38)
    batch = Batch(9, 1, 8, 2, 2, 16, 2, [8], R=128, norm=False, qkv=ref.bf16(x))
    batch.check(batch.run())


@needs_gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_write_zero_and_non_finite_heads(gpu, norm, eps):
    """Zero heads give zeros; a NaN or an infinity gives its own head a NaN scale and no other."""
    rng = np.random.default_rng(10)
    Hq, Hkv, T = 3, 3, 6
    x = rng.standard_normal((T, Hq + 2 * Hkv, D))
    x[0, [0, 3, 6]] = 0.0
    x[1, [1, 4, 7], 77] = np.nan
    x[2, [2, 5, 8], 3] = np.inf
    x[3, [0, 5, 6], 127] = -np.inf
    x[4, :, :64] = 0.0
    batch = Batch(11, 1, T, Hq, Hkv, 16, 1, [T], R=64, norm=norm, eps=eps, qkv=ref.bf16(x).reshape(T, -1))
    q = ref.bf16_to_f64(from_dev_bits(batch.run())).reshape(T, Hq, D)
    after = ref.Cache(batch.cache.cpu().numpy())
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(invalid="ignore"):
        want = list(batch.expect())
    for row, b, pos, q64, S, codes, scales in want:
        got, s = after.get(batch.table, b, pos)
        for h in range(Hq):
            if bad[row, h]:
                assert not np.isfinite(q[row, h]).all()
            else:
                assert (np.abs(q[row, h] - q64[h]) <= 2.0 ** -8 * np.abs(q64[h]) + 2.0 ** -20 * S[h]).all()
        for w in range(2):
            for h in range(Hkv):
                if bad[row, Hq + w * Hkv + h]:
                    assert np.isnan(s[w, h])
                else:
                    assert np.array_equal(got[w, h], codes[w, h])
                    assert abs(s[w, h] - scales[w, h]) <= 2.0 ** -20 * scales[w, h]


@needs_gpu
def test_write_the_same_place_twice(gpu):
    """Two rows at one place: each byte there is one of theirs, all else is as ever."""
    batch = Batch(12, 2, 4, 2, 2, 16, 1, [16, 16])
    batch.table[1] = batch.table[0]
    batch.run()
    got = batch.cache.cpu().numpy().copy()
    ones = []
    for b in range(2):
        alone = Batch(12, 2, 4, 2, 2, 16, 1, [16, 16])
        alone.table[1] = alone.table[0]
        alone.new = np.array([4, 0] if b == 0 else [0, 4], np.int32)
        alone.run()
        ones.append(alone.cache.cpu().numpy().copy())
    assert ((got == ones[0]) | (got == ones[1])).all()


# -------------------------------------------------------------------- read

def check_read(raw, table, total, L, start, k, v):
    cache = ref.Cache(raw)
    B = table.shape[0]
    total, _ = ref.lengths(total, None, 1, table.shape[1] * cache.page)
    k, v = from_dev_bits(k), from_dev_bits(v)
    for b in range(B):
        first = 0 if start is None else int(np.clip(start[b], 0, total[b]))
        for i in range(L):
            j = first + i
            got = cache.get(table, b, j) if j < total[b] else None
            for w, out in ((0, k), (1, v)):
                want = np.zeros((cache.kv_heads, D), np.uint16) if got is None else \
                    ref.bf16(got[0][w].astype(np.float32) * got[1][w][:, None])
                assert np.array_equal(out[b, i], want), (b, i, w)


@needs_gpu
@pytest.mark.parametrize("B,L,Hkv,page,start", [
    (1, 1, 1, 16, False), (3, 50, 2, 16, False), (2, 17, 3, 32, True), (4, 33, 8, 48, True), (1, 515, 4, 64, False), (2, 2, 1, 16, True),
    (5, 16, 1, 16, True)])
def test_read(gpu, B, L, Hkv, page, start):
    rng = np.random.default_rng(L)
    per = -(-(L + 20) // page)
    raw = random_cache(rng, B * per + 1, Hkv, page)
    table = make_table(rng, B, per, raw.shape[0])
    table[0, -1] = -1
    total = rng.integers(0, per * page + 1, B).astype(np.int32)
    total[-1] = per * page + 5
    first = rng.integers(-2, per * page, B).astype(np.int32) if start else None
    k, v = qlin.kv_read_bf16(to_dev(raw), to_dev(table), to_dev(total), L, start=to_dev(first) if start else None)
    check_read(raw, table, total, L, first, k, v)


@needs_gpu
def test_read_one_of_the_two(gpu, lib):
    rng = np.random.default_rng(1)
    raw, table = random_cache(rng, 4, 2, 16), np.array([[2, 0], [3, 1]], np.int32)
    total = np.array([20, 32], np.int32)
    raw_d, table_d, total_d = to_dev(raw), to_dev(table), to_dev(total)
    k, v = qlin.kv_read_bf16(raw_d, table_d, total_d, 32)
    for which in range(2):
        out = torch.full((2, 32, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
        to = [None, None]
        to[which] = out.data_ptr()
        assert lib.qlin_kv_read_bf16(raw_d.data_ptr(), 4, 16, 2, table_d.data_ptr(), 2, 2, total_d.data_ptr(), None, 32,
                                     to[0], to[1], None) == qlin.QLIN_OK
        torch.cuda.synchronize()
        assert torch.equal(out, (k, v)[which])


# --------------------------------------------------------------- attention

def tolerance(o64, A, X, big, n):
    return 2.0 ** -8 * np.abs(o64) + 1.05 * ((2.0 ** -11 + 2 * (2.0 ** -16 * X + 2.0 ** -20) + 4 * np.sqrt(n) * 2.0 ** -23) * A
                                             + min(n, 4 * np.sqrt(n)) * 2.0 ** -24 * big)


class Attn:
    def __init__(self, seed, B, T, Hq, Hkv, page, per, total, new=None, spread=0.5, size=1.0, **kw):
        rng = np.random.default_rng(seed)
        self.T, self.kw = T, kw
        pages = B * per + 2
        self.raw = random_cache(rng, pages, Hkv, page, spread)
        self.table = make_table(rng, B, per, pages)
        self.total = np.asarray(total, np.int32)
        self.new = None if new is None else np.asarray(new, np.int32)
        self.q = ref.bf16(size * rng.standard_normal((B * T, Hq * D)))

    def args(self):
        return (to_dev_bits(self.q, torch.bfloat16), to_dev(self.raw), to_dev(self.table), to_dev(self.total))

    def run(self, **more):
        out = torch.full((self.q.shape[0], self.q.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
        got = qlin.paged_attn_i8(*self.args(), new_len=None if self.new is None else to_dev(self.new), out=out, **self.kw, **more)
        assert got.data_ptr() == out.data_ptr()
        return out

    def check(self, out):
        o = ref.bf16_to_f64(from_dev_bits(out))
        o64, A, X, big, rows = ref.attention(ref.bf16_to_f64(self.q), ref.Cache(self.raw), self.table, self.total, self.T,
                                             new=self.new, **self.kw)
        n = max(1, int(self.total.max(initial=1)))
        n = min(n, self.table.shape[1] * ref.Cache(self.raw).page)
        bad = rows[:, None] & ~(np.abs(o - o64) <= tolerance(o64, A, X, big, n))
        assert not bad.any(), (np.argwhere(bad)[:4], o[bad][:4], o64[bad][:4])
        assert (o[~rows] == 7.0).all()


@needs_gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,page,total,kw", [
    # the lengths around a block, a tile and a cut
    (1, 1, 1, 1, 16, [1], {}), (3, 1, 4, 1, 16, [15, 16, 17], {}), (4, 1, 8, 2, 16, [127, 128, 129, 1], {}),
    (2, 1, 32, 8, 16, [515, 300], {}), (1, 1, 32, 8, 32, [2500], {}), (5, 1, 6, 6, 48, [1, 700, 2, 333, 48], {}),
    # groups of 1 to 16 query heads, odd ones too
    (2, 1, 3, 1, 16, [100, 40], {}), (2, 1, 5, 1, 16, [100, 40], {}), (1, 1, 9, 1, 16, [200], {}), (1, 1, 16, 1, 16, [333], {}),
    (1, 1, 14, 2, 64, [200], {}), (2, 1, 300, 1, 16, [40, 3], {}), (1, 2, 130, 2, 32, [60], {"window": 20}),
    # drafted blocks: rows of 8 to 128 a key/value head
    (2, 8, 4, 1, 16, [8, 140], {}), (2, 8, 16, 4, 16, [40, 300], {}), (1, 3, 30, 6, 48, [1000], {}), (2, 8, 8, 1, 16, [90, 9], {}),
    (2, 5, 4, 1, 16, [300, 20], {}), (3, 3, 16, 2, 16, [150, 3, 70], {}), (1, 10, 8, 2, 16, [280], {"causal": False}),
    (2, 9, 8, 1, 16, [200, 33], {"window": 70}), (1, 16, 8, 1, 16, [200], {}), (1, 9, 7, 1, 16, [70], {}), (1, 33, 2, 1, 16, [100], {}), (1, 1, 65, 1, 16, [50], {}),
    # masks
    (2, 8, 4, 1, 16, [8, 300], {"causal": False}), (2, 8, 4, 2, 16, [20, 300], {"window": 1}), (2, 8, 4, 2, 16, [20, 300], {"window": 5}),
    (2, 8, 4, 2, 16, [20, 300], {"window": 5, "causal": False}), (2, 1, 4, 1, 16, [300, 299], {"window": 128}),
    (3, 1, 4, 1, 16, [300, 12, 140], {"window": 131}), (2, 4, 4, 2, 16, [400, 20], {"window": 100, "causal": False}),
    (1, 1, 4, 1, 16, [200], {"window": 2 ** 40}),
    # scores
    (2, 2, 4, 2, 16, [90, 200], {"softcap": 5.0}), (1, 3, 6, 2, 16, [150], {"softcap": 1e5}), (1, 2, 4, 2, 16, [150], {"softcap": 0.01}),
    (1, 2, 4, 2, 16, [150], {"softcap": 2.0 ** -140}), (1, 2, 4, 2, 16, [150], {"softcap": 3e38}),
    (1, 2, 4, 2, 16, [150], {"window": 2 ** 63 - 1, "causal": False}), (1, 8, 8, 2, 16, [200], {"softcap": 30.0, "causal": False, "window": 60}),
    (1, 1, 4, 1, 16, [200], {"scale": 0.0}), (1, 1, 4, 1, 16, [200], {"scale": -0.3})])
def test_attention(gpu, B, T, Hq, Hkv, page, total, kw):
    per = -(-max(total) // page) + 1
    a = Attn(B + T + Hq + page, B, T, Hq, Hkv, page, per, total, **kw)
    a.check(a.run())


@needs_gpu
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (4, 8, 2), (8, 8, 1)])
def test_attention_padded_and_ragged(gpu, T, Hq, Hkv):
    """Lengths of zero, outside the table, new_len of all kinds: padding rows stay as they were."""
    total = [0, 1, 5, 400, -3, 2 ** 31 - 1, 129, 2]
    for new in (None, [1, 1, 0, T, 1, 2, -5, 2 ** 31 - 1]):
        a = Attn(T, 8, T, Hq, Hkv, 16, 26, total, new=new)
        a.check(a.run())


@needs_gpu
@pytest.mark.parametrize("T,window", [(1, 0), (8, 0), (8, 3)])
def test_attention_leaves_out_what_is_on_no_page(gpu, T, window):
    a = Attn(20 + T, 4, T, 4, 2, 16, 12, [190, 16, 40, 150], window=window)
    a.table[0, 3:7], a.table[1, 0], a.table[2, 2], a.table[3, :] = -1, a.raw.shape[0], 2 ** 31 - 1, -2 ** 31
    o = a.run()
    a.check(o)
    assert (o[3 * T:] == 0).all() and (o[T:2 * T] == 0).all()       # rows that see nothing


@needs_gpu
@pytest.mark.parametrize("T,causal,window", [(1, True, 0), (8, True, 0), (8, True, 20), (4, False, 30)])
def test_attention_ignores_what_no_row_sees(gpu, T, causal, window):
    """NaN, infinite and huge scales, and any codes, behind the end, before the window and on other pages."""
    a = Attn(31, 2, T, 4, 2, 16, 10, [100, 139], causal=causal, window=window)
    want = a.run()
    a.check(want)
    cache = ref.Cache(a.raw)
    poison = np.array([np.nan, np.inf, -np.inf, 3e38], np.float32)
    seen = np.zeros((a.raw.shape[0], 160), bool)
    for b, n in enumerate(a.total):
        for j in range(n):
            if not window or j > n - T - window:
                seen[a.table[b, j // 16], j % 16] = True
    for p in range(a.raw.shape[0]):
        for r in range(16):
            if not seen[p, r]:
                one = np.full((1, 1), p, np.int32)
                cache.put(one, 0, r, np.full((2, 2, D), 127), np.full((2, 2), poison[(p + r) % 4]))
    assert np.array_equal(from_dev_bits(a.run()), from_dev_bits(want))


@needs_gpu
def test_attention_non_finite_tokens_reach_only_rows_that_see_them(gpu):
    """The last of the drafted tokens has a NaN value scale, the one before a NaN key scale."""
    a = Attn(33, 1, 8, 4, 2, 16, 10, [100])
    want = ref.bf16_to_f64(from_dev_bits(a.run()))
    cache = ref.Cache(a.raw)
    for j, w in ((99, 1), (98, 0)):
        codes, s = cache.get(a.table, 0, j)
        s = s.copy()
        s[w] = np.nan
        cache.put(a.table, 0, j, codes, s)
    got = ref.bf16_to_f64(from_dev_bits(a.run()))
    assert np.isnan(got[6:]).all()
    assert np.array_equal(got[:6], want[:6])


@needs_gpu
def test_attention_large_and_small_scores_and_values(gpu):
    """Scores that leave one token, all alike; value scales over forty powers of two."""
    for seed, kw in ((1, {"size": 60.0}), (2, {"size": 0.0}), (3, {"spread": 6.0}), (4, {"size": 1e-30}), (5, {"size": 300.0, "spread": 0.0}),
                     (6, {"spread": 9.0, "size": 0.01})):
        a = Attn(40 + seed, 2, 2, 8, 2, 16, 20, [310, 200], **kw)
        a.check(a.run())


@needs_gpu
def test_attention_long_context(gpu):
    """One long and several short sequences, cut at different places; and twice the same."""
    for T, Hq, Hkv in ((1, 8, 2), (8, 8, 2)):
        a = Attn(50 + T, 4, T, Hq, Hkv, 64, 320, [20000, 9, 4000, 77])
        first = a.run()
        a.check(first)
        for _ in range(3):
            assert torch.equal(a.run(), first)


@needs_gpu
@pytest.mark.parametrize("seed,B,T,Hq,Hkv,longest", [
    # few segments, each cut into parts; as many as thread blocks; more
    (1, 1, 1, 4, 1, 9000), (2, 2, 3, 8, 2, 5000), (3, 7, 8, 16, 4, 900), (4, 31, 2, 16, 8, 700), (5, 32, 1, 6, 6, 1500),
    # a sequence more than a warp has lanes
    (6, 33, 1, 6, 6, 1500), (7, 33, 5, 4, 2, 600), (8, 40, 1, 8, 8, 200), (9, 12, 8, 8, 2, 2500)])
def test_attention_however_the_work_is_shared_out(gpu, seed, B, T, Hq, Hkv, longest):
    """Lengths alike, of all sizes, and one long among short ones."""
    rng = np.random.default_rng(100 + seed)
    for total in (np.full(B, longest // 3), rng.integers(0, longest + 1, B), np.where(np.arange(B) == B // 2, longest, 20)):
        a = Attn(110 + seed, B, T, Hq, Hkv, 16, -(-longest // 16), total, window=int(rng.integers(0, 2)) * 333)
        a.check(a.run())
        # tables with room for much longer sequences
        a.table = np.concatenate([a.table, np.full((B, 16000), -1, np.int32)], 1)
        a.check(a.run())


@needs_gpu
def test_attention_many_sequences(gpu):
    """More sequences than threads of a block, most of them short."""
    rng = np.random.default_rng(60)
    total = rng.integers(0, 40, 700)
    total[5], total[600] = 900, 333
    a = Attn(61, 700, 1, 2, 1, 16, 57, total)
    a.check(a.run())
    a = Attn(62, 300, 2, 4, 2, 16, 57, total[:300], new=rng.integers(0, 3, 300))
    a.check(a.run())


# ----------------------------------------------------- together, as in a step

@needs_gpu
def test_a_layer_between_its_linears(gpu):
    """The q/k/v linear, the cache, attention, quantization and the o linear over
    a prompt and three drafted blocks: each step from the step before's own
    output, against the definitions."""
    rng = np.random.default_rng(70)
    B, Hq, Hkv, page, per, K = 2, 4, 2, 16, 6, 512
    raw = random_cache(rng, B * per, Hkv, page)
    table = make_table(rng, B, per, B * per)
    cache = to_dev(raw)
    g = torch.Generator("cuda").manual_seed(71)

    def weights(K, N):
        w = torch.empty((K // 4, N), dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
        return w, 2e-4 * (1.0 + torch.rand(N, generator=g, device="cuda"))
    qkv_w, o_w = weights(K, (Hq + 2 * Hkv) * D), weights(Hq * D, K)
    gamma = to_dev_bits(ref.bf16(1.0 + 0.1 * rng.standard_normal(K)), torch.bfloat16)
    head = {k: ref.bf16(1.0 + 0.1 * rng.standard_normal(D)) for k in ("q_gamma", "k_gamma")}
    head_d = {k: to_dev_bits(v, torch.bfloat16) for k, v in head.items()}
    turn = cos_sin(per * page, D)
    total = np.zeros(B, np.int32)
    for T, new in ((33, [33, 20]), (8, None), (8, [8, 3]), (1, None)):
        total = (total + (T if new is None else np.array(new))).astype(np.int32)
        new_d = None if new is None else to_dev(np.array(new, np.int32))
        x = torch.randn((B * T, K), generator=g, device="cuda").bfloat16()
        q8, s, _ = qlin.add_rmsnorm_act_quant_i8(x, torch.zeros_like(x), gamma, 1e-6)
        qkv = qlin.gemm_w8a8_ch(q8, s, *qkv_w)
        q = qlin.kv_write_i8(qkv, cache, to_dev(table), to_dev(total), Hq, new_len=new_d, cos_sin=to_dev(turn), **head_d,
                             q=torch.zeros((B * T, Hq * D), dtype=torch.bfloat16, device="cuda"))
        out = qlin.paged_attn_i8(q, cache, to_dev(table), to_dev(total), new_len=new_d, out=torch.zeros_like(q))
        codes, s_o = qlin.act_quant_i8(out)
        y = qlin.gemm_w8a8_ch(codes, s_o, *o_w)
        torch.cuda.synchronize()
        after = ref.Cache(cache.cpu().numpy())
        for row, b, pos, q64, size, want, scales in ref.write(
                ref.bf16_to_f64(from_dev_bits(qkv)), after, table, total, Hq, T, new=new, cos_sin=turn, eps=float(np.float32(1e-6)),
                **{k: ref.bf16_to_f64(v) for k, v in head.items()}):
            got, gs = after.get(table, b, pos)
            assert np.array_equal(got, want) and (np.abs(gs - scales) <= 2.0 ** -20 * scales).all()
            assert (np.abs(ref.bf16_to_f64(from_dev_bits(q[row])).reshape(Hq, D) - q64) <= 2.0 ** -8 * np.abs(q64) + 2.0 ** -20 * size + 2.0 ** -134).all()
        o64, A, X, big, rows = ref.attention(ref.bf16_to_f64(from_dev_bits(q)), after, table, total, T, new=new)
        o = ref.bf16_to_f64(from_dev_bits(out))
        assert (np.abs(o - o64) <= tolerance(o64, A, X, big, int(total.max())))[rows].all()
        assert (o[~rows] == 0).all()
        P = codes.double().cpu().numpy() @ (torch.stack([((o_w[0] >> (8 * i)) & 255) - 128 for i in range(4)], 1)
                                            .reshape(Hq * D, K).double().cpu().numpy())
        y64 = P * o_w[1].double().cpu().numpy()[None] * s_o.double().cpu().numpy()[:, None]
        assert (np.abs(ref.bf16_to_f64(from_dev_bits(y)) - y64) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(y64)).all()
    back = qlin.kv_read_bf16(cache, to_dev(table), to_dev(total), int(total.max()))
    check_read(cache.cpu().numpy(), table, total, int(total.max()), None, *back)


# --------------------------------------------------- streams, graphs, threads

def decoding_step(state, **kw):
    q = qlin.kv_write_i8(state["qkv"], state["cache"], state["table"], state["total"], state["Hq"], cos_sin=state["turn"], **kw)
    out = qlin.paged_attn_i8(q, state["cache"], state["table"], state["total"], window=state.get("window", 0), **kw)
    k, v = qlin.kv_read_bf16(state["cache"], state["table"], state["total"], 40, **kw)
    return q, out, k, v


def step_state(seed, B=3, T=2, Hq=8, Hkv=2, per=40):
    rng = np.random.default_rng(seed)
    raw = random_cache(rng, B * per, Hkv, 16)
    return {"qkv": to_dev_bits(ref.bf16(rng.standard_normal((B * T, (Hq + 2 * Hkv) * D))), torch.bfloat16), "cache": to_dev(raw),
            "table": to_dev(make_table(rng, B, per, B * per)), "total": to_dev(np.array([600, 35, 200][:B], np.int32)), "Hq": Hq,
            "turn": to_dev(cos_sin(per * 16, D))}


@needs_gpu
def test_step_in_a_graph_beside_eager_calls(gpu):
    """A captured step with its lengths moved between replays, eager steps of
    other states in between, on another stream too."""
    a, b = step_state(1), step_state(2)
    want = {}
    fresh = a["cache"].clone()
    for n in (35, 60, 16 * 40):
        a["cache"].copy_(fresh)
        a["total"].fill_(n)
        want[n] = [t.clone() for t in decoding_step(a)]
    want_b = [t.clone() for t in decoding_step(b)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decoding_step(a)
    for n in (60, 35, 16 * 40, 60):
        a["cache"].copy_(fresh)
        a["total"].fill_(n)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        other = decoding_step(b, stream=side)
        torch.cuda.synchronize()
        for x, y in zip(got, want[n]):
            assert torch.equal(x, y), n
        for x, y in zip(other, want_b):
            assert torch.equal(x, y)


def attn_of(state):
    """The state behind its step's write, with the queries."""
    q = qlin.kv_write_i8(state["qkv"], state["cache"], state["table"], state["total"], state["Hq"], cos_sin=state["turn"])
    return {**state, "q": q}


@needs_gpu
def test_two_captured_steps_in_one_workspace(gpu):
    """Replayed one behind the other, in either order."""
    room = torch.empty(qlin.paged_attn_workspace_bytes(3, 2, 8, 2), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    states = [attn_of(step_state(3)), attn_of(step_state(4))]
    for s in states:
        out = torch.empty_like(s["q"])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            qlin.paged_attn_i8(s["q"], s["cache"], s["table"], s["total"], out=out, workspace=room)
        outs.append(out)
        graphs.append(graph)
    alone = []
    for i in (0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        alone.append(outs[i].clone())
    assert not torch.equal(alone[0], alone[1])
    for order in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0, 1)):
        for out in outs:
            out.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


@needs_gpu
def test_calls_on_the_null_stream_by_its_handle(gpu):
    s = attn_of(step_state(5))
    want = qlin.paged_attn_i8(s["q"], s["cache"], s["table"], s["total"])
    k, v = qlin.kv_read_bf16(s["cache"], s["table"], s["total"], 30)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = qlin.paged_attn_i8(s["q"], s["cache"], s["table"], s["total"], stream=0)
        k0, v0 = qlin.kv_read_bf16(s["cache"], s["table"], s["total"], 30, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(k0, k) and torch.equal(v0, v)


@needs_gpu
def test_steps_of_several_threads(gpu):
    states = [step_state(10 + i) for i in range(4)]
    want = [[t.clone() for t in decoding_step(s)] for s in states]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(20):
            got = decoding_step(states[i], stream=stream)
            stream.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


@needs_gpu
def test_step_follows_late_inputs(gpu):
    """Inputs that the kernels in front write late on the same stream."""
    s = step_state(20)
    want = [t.clone() for t in decoding_step(s)]
    late = {k: torch.zeros_like(v) for k, v in s.items() if isinstance(v, torch.Tensor)}
    torch.cuda.synchronize()
    for _ in range(3):
        for t in late.values():
            t.zero_()
        torch.cuda._sleep(5_000_000)
        for k, t in late.items():
            t.copy_(s[k])
        got = decoding_step({**s, **late})
        copies = [t.clone() for t in got]
        torch.cuda.synchronize()
        for x, y in zip(copies, want):
            assert torch.equal(x, y)


@needs_gpu
def test_attention_with_a_dirty_guarded_workspace(gpu):
    for T, Hq, Hkv, total in ((1, 8, 2, [700, 33]), (8, 8, 2, [300, 90])):
        a = Attn(80 + T, 2, T, Hq, Hkv, 16, 50, total)
        need = qlin.paged_attn_workspace_bytes(2, T, Hq, Hkv)
        buf = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")      # NaN everywhere
        want = a.run()
        for _ in range(2):
            assert torch.equal(a.run(workspace=buf[256:256 + need]), want)
        assert (buf[:256] == 255).all() and (buf[256 + need:] == 255).all()
        if need:
            with pytest.raises(qlin.QlinError) as e:
                a.run(workspace=buf[:need - 16])
            assert e.value.status == qlin.QLIN_ERR_WORKSPACE


@needs_gpu
def test_cache_past_32_bits(gpu):
    """Pages and rows whose bytes lie past 2^32."""
    Hkv, page = 8, 64
    pages = (2 ** 32 + 2 ** 28) // (Hkv * page // 16 * ref.BLOCK)
    g = torch.Generator("cuda").manual_seed(3)
    cache = torch.zeros((pages, Hkv, page // 16, ref.BLOCK), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, pages - 2], [3, 1], [pages // 2, pages - 3]], dtype=torch.int32, device="cuda")
    total = torch.tensor([100, 70, 128], dtype=torch.int32, device="cuda")
    qkv = torch.randn((3 * 70, 3 * Hkv * D), generator=g, device="cuda").bfloat16()
    q = qlin.kv_write_i8(qkv, cache, table, total, Hkv)
    low = torch.zeros((6, Hkv, page // 16, ref.BLOCK), dtype=torch.uint8, device="cuda")
    small = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    assert torch.equal(qlin.kv_write_i8(qkv, low, small, total, Hkv), q)
    assert torch.equal(cache[table.view(-1).long()], low)
    assert int(cache.view(-1)[:table[1, 1] * Hkv * page // 16 * ref.BLOCK].any()) == 0
    assert torch.equal(qlin.paged_attn_i8(q, cache, table, total), qlin.paged_attn_i8(q, low, small, total))
    for x, y in zip(qlin.kv_read_bf16(cache, table, total, 128), qlin.kv_read_bf16(low, small, total, 128)):
        assert torch.equal(x, y)


@needs_gpu
def test_read_output_past_32_bits(gpu):
    B, L, Hkv = 3, 2 ** 20, 8
    raw = to_dev(random_cache(np.random.default_rng(4), 2, Hkv, 16))
    table = torch.zeros((B, L // 16), dtype=torch.int32, device="cuda")
    table[:, ::2] = 1
    k, v = qlin.kv_read_bf16(raw, table, torch.full((B,), L, dtype=torch.int32, device="cuda"), L)
    assert B * L * Hkv * D > 2 ** 31
    for t in (k, v):
        assert torch.equal(t[:, 32:].view(B, -1, 32, Hkv, D), t[:, :32].unsqueeze(1).expand(B, L // 32 - 1, 32, Hkv, D))
    check_read(raw.cpu().numpy(), table[:, :2].cpu().numpy(), np.full(B, 32), 32, None, k[:, :32], v[:, :32])


# ---------------------------------------------------------------- refusals

@needs_gpu
def test_empty_batches(gpu):
    cache = qlin.kv_cache(2, 2, 16)
    none = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = qlin.kv_write_i8(torch.zeros((0, 8 * D), dtype=torch.bfloat16, device="cuda"), cache, none, lens, 4)
    assert q.shape == (0, 4 * D)
    assert qlin.paged_attn_i8(q, cache, none, lens).shape == (0, 4 * D)
    k, v = qlin.kv_read_bf16(cache, none, lens, 5)
    assert k.shape == v.shape == (0, 5, 2, D)
    one = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    k, v = qlin.kv_read_bf16(cache, one, torch.ones(1, dtype=torch.int32, device="cuda"), 0)
    assert k.shape == (1, 0, 2, D)
    rows = torch.zeros((0, 8 * D), dtype=torch.bfloat16, device="cuda")
    assert qlin.kv_write_i8(rows, cache, one, torch.ones(1, dtype=torch.int32, device="cuda"), 4).shape == (0, 4 * D)


@needs_gpu
def test_refused_tensors(gpu):
    cache = qlin.kv_cache(4, 2, 16)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    total = torch.ones(2, dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 8 * D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((4, 4 * D), dtype=torch.bfloat16, device="cuda")
    turn = torch.zeros((8, 64), device="cuda")
    pos = torch.zeros((2, 4), dtype=torch.int32, device="cuda")

    def write(x=x, cache=cache, table=table, total=total, heads=4, **kw):
        return qlin.kv_write_i8(x, cache, table, total, heads, **kw)
    write()
    for error, kw in ((TypeError, {"x": x.half()}), (ValueError, {"x": x[:3].contiguous()}), (ValueError, {"x": x[:, ::2]}),
                      (ValueError, {"heads": 5}), (ValueError, {"heads": -1}), (TypeError, {"heads": "4"}),
                      (TypeError, {"cache": cache.char()}), (ValueError, {"cache": cache[..., :4096].contiguous()}),
                      (ValueError, {"cache": cache[0]}), (ValueError, {"cache": cache.cpu()}), (TypeError, {"table": table.long()}),
                      (ValueError, {"table": table[0]}), (ValueError, {"total": total[:1]}), (TypeError, {"total": total.long()}),
                      (ValueError, {"new_len": total[:1]}), (ValueError, {"q_gamma": x[0, :64].contiguous()}),
                      (TypeError, {"k_gamma": turn[0]}), (TypeError, {"cos_sin": turn.double()}), (ValueError, {"cos_sin": turn[:0]}),
                      (ValueError, {"positions": pos}), (ValueError, {"cos_sin": turn, "positions": pos}),
                      (ValueError, {"cos_sin": turn, "positions": pos[:, :3].contiguous()}),
                      (TypeError, {"cos_sin": turn, "positions": pos, "axes": pos[0]}),
                      (ValueError, {"cos_sin": turn, "positions": pos, "axes": torch.zeros(64, dtype=torch.uint8, device="cuda")}),
                      (ValueError, {"q": q[:2]}), (TypeError, {"q": q.float()})):
        with pytest.raises(error):
            write(**kw)
    for kw in ({"cos_sin": turn[:, :40].contiguous()}, {"eps": float("nan")}, {"eps": -1.0}):
        with pytest.raises(qlin.QlinError) as e:
            write(**kw)
        assert e.value.status == qlin.QLIN_ERR_SHAPE

    def attn(q=q, cache=cache, table=table, total=total, **kw):
        return qlin.paged_attn_i8(q, cache, table, total, **kw)
    attn()
    for error, kw in ((TypeError, {"q": q.half()}), (ValueError, {"q": q[:, :3 * D].contiguous()}), (ValueError, {"q": q[:3].contiguous()}),
                      (ValueError, {"q": q[:, :0].contiguous()}), (ValueError, {"out": q[:2]}), (TypeError, {"workspace": q}),
                      (TypeError, {"window": 1.5}), (TypeError, {"softcap": "a"}), (ValueError, {"new_len": total[:1]})):
        with pytest.raises(error):
            attn(**kw)
    for kw in ({"window": -1}, {"softcap": -1.0}, {"softcap": float("inf")}, {"scale": float("nan")}):
        with pytest.raises(qlin.QlinError) as e:
            attn(**kw)
        assert e.value.status == qlin.QLIN_ERR_SHAPE

    def read(cache=cache, table=table, total=total, length=4, **kw):
        return qlin.kv_read_bf16(cache, table, total, length, **kw)
    read()
    for error, kw in ((ValueError, {"length": -1}), (ValueError, {"start": total[:1]}), (ValueError, {"k": q}),
                      (TypeError, {"start": total.long()}), (TypeError, {"total": total.float()})):
        with pytest.raises(error):
            read(**kw)
    with pytest.raises(ValueError):
        qlin.kv_cache(2, 2, 24)


OK, ODD = 0x1000, 0x1008      # never dereferenced: every call below is refused


def _p(n):
    return ctypes.c_void_p(n)


def test_write_refusals(lib):
    def call(x=OK, B=2, T=3, Hq=4, Hkv=2, qg=None, kg=None, eps=1e-6, cs=None, P=0, R=0, pos=None, A=0, ax=None, cache=OK, pages=4,
             page=16, tab=OK, per=2, tot=OK, new=None, q=OK):
        return int(lib.qlin_kv_write_i8(_p(x), B, T, Hq, Hkv, _p(qg), _p(kg), eps, _p(cs), P, R, _p(pos), A, _p(ax), _p(cache), pages,
                                        page, _p(tab), per, _p(tot), _p(new), _p(q), None))
    turn = {"cs": OK, "P": 8, "R": 64}
    for kw in ({"x": None}, {"cache": None}, {"tab": None}, {"tot": None}, {"q": None}, {"P": 8, "R": 64}, {"cs": OK},
               {**turn, "A": 1}, {**turn, "A": 2, "pos": OK}):
        assert call(**kw) == qlin.QLIN_ERR_NULL, kw
    for kw in ({"B": -1}, {"T": -1}, {"B": 2 ** 16, "T": 2 ** 16}, {"Hq": -1}, {"Hq": 65536}, {"Hkv": 0}, {"Hkv": 65536}, {"eps": -1.0},
               {"eps": float("nan")}, {"eps": float("inf")}, {**turn, "R": 40}, {**turn, "R": 144}, {**turn, "R": -16}, {**turn, "P": 0},
               {**turn, "P": 2 ** 31}, {**turn, "A": -1, "pos": OK}, {**turn, "A": 256, "pos": OK, "ax": OK}, {"pages": 0},
               {"pages": 2 ** 31}, {"page": 0}, {"page": 24}, {"page": 65552}, {"per": 0}, {"per": 2 ** 26 + 1}):
        assert call(**kw) == qlin.QLIN_ERR_SHAPE, kw
    for kw in ({"x": ODD}, {"q": ODD}, {"qg": ODD}, {"kg": ODD}, {**turn, "cs": ODD}, {**turn, "A": 1, "pos": 0x1002},
               {**turn, "A": 2, "pos": OK, "ax": 0x1002}, {"cache": 0x1040}, {"tab": 0x1002}, {"tot": 0x1002}, {"new": 0x1002}):
        assert call(**kw) == qlin.QLIN_ERR_ALIGN, kw
    if not torch.cuda.is_available():
        for kw in ({}, {"Hq": 0, "q": None}, {**turn, "A": 1, "pos": OK}, {"B": 0, "x": None, "cache": None, "tab": None, "tot": None, "q": None}):
            assert call(**kw) == qlin.QLIN_ERR_DEVICE, kw


def test_read_refusals(lib):
    def call(cache=OK, pages=4, page=16, Hkv=2, tab=OK, B=2, per=2, tot=OK, st=None, L=5, k=OK, v=OK):
        return int(lib.qlin_kv_read_bf16(_p(cache), pages, page, Hkv, _p(tab), B, per, _p(tot), _p(st), L, _p(k), _p(v), None))
    for kw in ({"cache": None}, {"tab": None}, {"tot": None}, {"k": None, "v": None}):
        assert call(**kw) == qlin.QLIN_ERR_NULL, kw
    for kw in ({"B": -1}, {"L": -1}, {"L": 2 ** 30 + 1}, {"pages": 0}, {"page": 8}, {"Hkv": 0}, {"per": 0}):
        assert call(**kw) == qlin.QLIN_ERR_SHAPE, kw
    for kw in ({"cache": 0x1010}, {"tab": 0x1002}, {"tot": 0x1002}, {"st": 0x1002}, {"k": ODD}, {"v": ODD}):
        assert call(**kw) == qlin.QLIN_ERR_ALIGN, kw
    if not torch.cuda.is_available():
        for kw in ({}, {"k": None}, {"L": 0, "cache": None, "tab": None, "tot": None, "k": None, "v": None}):
            assert call(**kw) == qlin.QLIN_ERR_DEVICE, kw


def test_attention_refusals(lib):
    def call(q=OK, B=2, T=3, Hq=4, Hkv=2, cache=OK, pages=4, page=16, tab=OK, per=2, tot=OK, new=None, scale=0.1, cap=0.0, window=0,
             causal=1, out=OK, ws=OK, n=1 << 40):
        return int(lib.qlin_paged_attn_i8(_p(q), B, T, Hq, Hkv, _p(cache), pages, page, _p(tab), per, _p(tot), _p(new), scale, cap, window,
                                          causal, _p(out), _p(ws), n, None))
    for kw in ({"q": None}, {"cache": None}, {"tab": None}, {"tot": None}, {"out": None}):
        assert call(**kw) == qlin.QLIN_ERR_NULL, kw
    for kw in ({"B": -1}, {"T": -1}, {"B": 2 ** 16, "T": 2 ** 16}, {"Hq": 0}, {"Hq": 5}, {"Hkv": 0}, {"Hq": 65536}, {"pages": 0}, {"page": 17},
               {"per": 0}, {"scale": float("inf")}, {"scale": float("nan")}, {"cap": -1.0}, {"cap": float("nan")}, {"window": -1}):
        assert call(**kw) == qlin.QLIN_ERR_SHAPE, kw
    for kw in ({"q": ODD}, {"out": ODD}, {"ws": ODD}, {"cache": 0x1008}, {"tab": 0x1002}, {"tot": 0x1002}, {"new": 0x1002}):
        assert call(**kw) == qlin.QLIN_ERR_ALIGN, kw
    for B, T, Hq, Hkv in ((-1, 1, 4, 2), (1, -1, 4, 2), (1, 1, 5, 2), (1, 1, 0, 2), (1, 1, 4, 0), (0, 1, 4, 2), (1, 0, 4, 2)):
        assert qlin.paged_attn_workspace_bytes(B, T, Hq, Hkv) == 0
    if not torch.cuda.is_available():
        assert call() == qlin.QLIN_ERR_DEVICE
        assert qlin.paged_attn_workspace_bytes(1, 1, 4, 2) == 0


def test_cache_bytes(lib):
    assert qlin.kv_cache_bytes(3, 2, 16) == 3 * 2 * 4224
    assert qlin.kv_cache_bytes(5, 8, 64) == 5 * 8 * 4 * 4224
    for pages, heads, page in ((0, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 24), (1, 1, 65552), (2 ** 31, 1, 16), (-1, 1, 16), (1, 65536, 16),
                               (2 ** 31 - 1, 65535, 65536)):
        assert qlin.kv_cache_bytes(pages, heads, page) == 0


def test_cpu_tensors_are_refused(lib):
    x = torch.zeros((2, 4 * D), dtype=torch.bfloat16)
    cache = torch.zeros((2, 1, 1, 4224), dtype=torch.uint8)
    table, total = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: qlin.kv_write_i8(x, cache, table, total, 2), lambda: qlin.paged_attn_i8(x, cache, table, total),
                 lambda: qlin.kv_read_bf16(cache, table, total, 3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_places_of_codes():
    """Every byte of a token's row is used once, a block's parts are 4224 bytes."""
    p = ref.code_places()
    assert (np.sort(p, 1) == 128 * np.arange(16)[:, None] + np.arange(128)[None, :]).all()
    assert 2 * 2048 + 2 * 64 == ref.BLOCK
