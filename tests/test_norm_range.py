"""Residual addition + RMSNorm + act-quant at the ends of its range: rows of very
large and very small values, and rows that hold no finite result.

The references are exact where the definition is: the sum is one bf16 rounding,
and the oracle forms the norm in binary64 (relative error of its 1 / sqrt about
2^-52), rounded once to bf16.  So the checks are equalities."""
import numpy as np
import pytest
import torch

import oracle
from helpers import from_dev_bits, to_dev_bits
from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    oracle.build()
    qlin.load()


def bits(v):
    return synth.bf16_bits(np.asarray(v, np.float64))


def run(xb, rb, gb, eps, c16=False):
    x, r, g = (to_dev_bits(a, torch.bfloat16) for a in (xb, rb, gb))
    y = torch.empty_like(x)
    call = qlin.add_rmsnorm_act_quant_c16 if c16 else qlin.add_rmsnorm_act_quant_i8
    q, s, h = call(x, r, g, eps, y=y)
    return q, s, h, y


# the mean of h^2 is about 2^e; one block a row in each of the kernel's forms, rows of
# several blocks, and rows longer than registers hold
@pytest.mark.parametrize("M,K", [(3, 640), (60000, 128), (2000, 2560), (8, 17408), (700, 5120), (2, 33024)])
@pytest.mark.parametrize("e", [-98, -62, -58, 0, 58, 62, 112, "top"])
def test_rows_of_large_and_small_values(M, K, e):
    if e == "top":      # sums between 2^126 and 2^128
        e = 126 - int(np.log2(K))
    rng = np.random.default_rng(K + e)
    amp = 2.0 ** (e / 2) * (1.0 + 0.2 * rng.random((M, 1)))
    h = rng.uniform(-1.7, 1.7, (M, K)) * amp
    part = rng.uniform(0.2, 0.8, (M, K))
    xb, rb = bits(h * part), bits(h * (1 - part))
    gb = bits(1.0 + 0.1 * rng.standard_normal(K))
    hb = bits(synth.bf16_values(xb).astype(np.float64) + synth.bf16_values(rb).astype(np.float64))
    h64 = synth.bf16_values(hb).astype(np.float64)
    assert (h64 * h64).sum(1).max() < 2.0 ** 128 and ((h64 * h64).mean(1)).min() >= 2.0 ** -100
    for eps in (0.0, 1e-6):
        # the call takes eps in fp32, and here it is most of the norm of small rows
        q0, s0, z0 = oracle.rmsnorm_act_quant_i8(hb, gb, float(np.float32(eps)))
        q, s, h, y = run(xb, rb, gb, eps)
        assert np.array_equal(from_dev_bits(h), hb)
        assert np.array_equal(from_dev_bits(y), z0)
        assert np.array_equal(s.cpu().numpy(), s0) and np.array_equal(q.cpu().numpy(), q0)


def near_ties(rows, K, keep):
    """`keep` rows of K bf16 values about 1 in size, each with an element whose
    product with 1 / rms lies next to the middle between two bf16 values: the
    nearest ones of `rows` rows with each of 384 values in front."""
    rng = np.random.default_rng(5)
    body = synth.bf16_values(bits(rng.uniform(-1.7, 1.7, (rows, K - 1)))).astype(np.float64)
    first = np.outer([0.25, 0.5, 1.0], np.arange(128, 256) / 128.0).reshape(1, -1)
    t = first / np.sqrt(((body * body).sum(1)[:, None] + first * first) / K)
    u = np.frexp(t)[0] * 256.0          # bf16 values are the integers from 128 to 256
    away = np.abs(u - np.floor(u) - 0.5)
    row, col = np.unravel_index(np.argsort(away, axis=None)[:keep], away.shape)
    assert away[row, col].max() < 2.0 ** -19
    return np.concatenate([first[0, col][:, None], body[row]], 1)


def test_products_next_to_the_middle_at_the_largest_sums():
    """Sums of h^2 of about 2^127: 1 / rms has to be as exact there as elsewhere."""
    K = 128
    h = near_ties(100000, K, 64)
    gb = bits(np.ones(K))
    zero = bits(np.zeros_like(h))
    for scale in (2.0 ** 60, 1.0, 2.0 ** -49):
        hb = bits(h * scale)
        _, _, z0 = oracle.rmsnorm_act_quant_i8(hb, gb, 0.0)
        _, _, _, y = run(hb, zero, gb, 0.0)
        assert np.array_equal(from_dev_bits(y), z0)


BAD = ["nan", "inf", "both infinities", "the sum overflows bf16", "the squares overflow", "large and nan"]


@pytest.mark.parametrize("M,K", [(8, 256), (300, 640), (12, 17408), (9, 33024)])
@pytest.mark.parametrize("c16", [False, True], ids=["i8", "c16"])
def test_rows_without_a_finite_result_are_nan(M, K, c16):
    """Not zeros: the product after them is NaN too, and the other rows are as ever."""
    rng = np.random.default_rng(K)
    x, r = rng.standard_normal((M, K)), rng.standard_normal((M, K))
    xb, rb = bits(x), bits(r)
    at = {name: i + 1 for i, name in enumerate(BAD)}
    nan, inf = 0x7FC0, 0x7F80
    xb[at["nan"], K // 3] = nan
    rb[at["inf"], 5] = inf
    xb[at["both infinities"], [0, K - 1]] = inf
    rb[at["both infinities"], K - 1] = inf | 0x8000
    xb[at["the sum overflows bf16"], K // 2] = rb[at["the sum overflows bf16"], K // 2] = 0x7F7F
    xb[at["the squares overflow"], :] = bits(2.0 ** 62)
    rb[at["the squares overflow"], :] = bits(2.0 ** 62)
    xb[at["large and nan"], :] = bits(2.0 ** 62)
    xb[at["large and nan"], K - 2] = nan | 0x8000
    gb = bits(1.0 + 0.1 * rng.standard_normal(K))
    bad = np.zeros(M, bool)
    bad[list(at.values())] = True
    q, s, h, y = run(xb, rb, gb, 1e-6, c16)
    assert torch.isnan(s).cpu().numpy().tolist() == bad.tolist()
    assert torch.isnan(y).all(1).cpu().numpy().tolist() == bad.tolist()
    fine = ~bad
    hb = bits(synth.bf16_values(xb[fine]).astype(np.float64) + synth.bf16_values(rb[fine]).astype(np.float64))
    q0, s0, z0 = oracle.rmsnorm_act_quant_i8(hb, gb, 1e-6)
    assert np.array_equal(from_dev_bits(h)[fine], hb) and np.array_equal(from_dev_bits(y)[fine], z0)
    assert np.array_equal(s.cpu().numpy()[fine], s0)
    assert np.array_equal(q.float().cpu().numpy()[fine], q0.astype(np.float32))
    # the product: few channels (streamed) and many (in tiles)
    for N in (64, 20488) if K == 640 else (64,):
        w = torch.randint(-2 ** 31, 2 ** 31, (K // 4, N), device="cuda").to(torch.int32)
        s_w = torch.ones(N, device="cuda")
        out = (qlin.gemm_w8a8_ch_c16 if c16 else qlin.gemm_w8a8_ch)(q, s, w, s_w)
        assert torch.isnan(out).all(1).cpu().numpy().tolist() == bad.tolist()
        assert not torch.isnan(out[torch.from_numpy(fine).cuda()]).any()


def test_a_bad_row_written_in_place():
    K = 640
    xb, rb = bits(np.ones((4, K))), bits(np.full((4, K), 2.0))
    xb[2, 7] = 0x7FC0
    x, r, g = (to_dev_bits(a, torch.bfloat16) for a in (xb, rb, bits(np.ones(K))))
    _, s, h = qlin.add_rmsnorm_act_quant_i8(x, r, g, 1e-6, residual_out=r)
    assert h.data_ptr() == r.data_ptr()
    assert torch.isnan(s).tolist() == [False, False, True, False]
    assert torch.isnan(r).sum() == 1 and torch.isnan(r[2, 7])
    keep = torch.ones_like(r, dtype=torch.bool)
    keep[2, 7] = False
    assert (r[keep] == 3).all()
