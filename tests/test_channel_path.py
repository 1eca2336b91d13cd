"""The operators around a per-channel W8A8 linear: the residual addition fused
with RMSNorm and act-quant, the product with one scale per token and one per
output channel, and the adjusted logits.

The definitions round at stated places only (include/qlin.h), so most checks
are equalities: h, t, z, the scales and the codes with the oracle's chain, y
with the exact integer product (binary64 sums of integers below 2^53) put
through the definition's two fp32 products, the logits with the definition's
fp32 steps.  Each is also held to an unrounded binary64 evaluation:
  * y: float(P) and two products, each off by at most 2^-24 of its value, then
    the rounding to bf16, at most 2^-8 of the value (half a step next to a
    power of two): |y - y64| <= (3 * 2^-24 * 1.01 + 2^-8) |y64|;
  * logits: at most five fp32 roundings (quotient, frequency * n, + presence,
    the difference, + bias), each 2^-24 of a value at most S = |x| max(rep,
    1 / rep) + frequency n + presence + |bias|, then the rounding to the
    logits' type: |o - o64| <= 5 * 2^-24 S + e |o64|, e = 2^-8 (bf16) or 0."""
import ctypes

import threading

import numpy as np
import pytest
import torch

import oracle
from helpers import from_dev_bits, to_dev, to_dev_bits
from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin, synth

needs_gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qlin.load()
    oracle.build()
    assert qlin.device_status() == qlin.QLIN_OK
    yield torch.device("cuda")
    torch.cuda.synchronize()
    assert qlin.device_status() == qlin.QLIN_OK


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qlin.load()


# --------------------------------------------- references (numpy, binary64)

def ref_add_rmsnorm(xb, rb, gb, eps):
    """(q, s, z bits, h bits): the exact bf16 sum, then the oracle's chain."""
    h = synth.bf16_bits(synth.bf16_values(xb).astype(np.float64) + synth.bf16_values(rb).astype(np.float64))
    q, s, z = oracle.rmsnorm_act_quant_i8(h, gb, eps)
    return q, s, z, h


def ref_channel(q_a, s_a, q_w, s_w):
    """(y bf16 bits, y in binary64 unrounded)."""
    P = q_a.astype(np.float64) @ q_w.astype(np.float64)
    y = (P.astype(np.float32) * s_w[None, :].astype(np.float32)) * s_a[:, None].astype(np.float32)
    return synth.bf16_bits(y), P * s_w[None, :].astype(np.float64) * s_a[:, None].astype(np.float64)


def ref_logits(x, bf16, tokens=None, prompt=None, total=None, rep=None, pres=None, freq=None,
               bias_ids=None, bias=None, allowed=None, dtype=np.float32):
    """The definition row by row, in `dtype`; for binary32 also rounded to the
    logits' type.  Returns (values, S of the module docstring, argmax)."""
    M, V = x.shape
    out = x.astype(dtype).copy()
    S = np.abs(np.where(np.isfinite(x), x, 0)).astype(np.float64)
    for m in range(M):
        row = out[m]
        if tokens is not None:
            L = tokens.shape[1]
            tot = L if total is None else min(max(int(total[m]), 0), L)
            pr = 0 if prompt is None else int(prompt[m])
            made, seen = {}, set()
            for i, v in enumerate(tokens[m, :tot].tolist()):
                if 0 <= v < V:
                    seen.add(v)
                    if i >= pr:
                        made[v] = made.get(v, 0) + 1
            r = dtype(1 if rep is None else rep[m])
            p = dtype(0 if pres is None else pres[m])
            f = dtype(0 if freq is None else freq[m])
            for v in seen:
                row[v] = row[v] / r if row[v] > 0 else row[v] * r
                S[m, v] *= max(float(r), 1.0 / float(r))
            for v, n in made.items():
                row[v] = row[v] - (f * dtype(n) + p)
                S[m, v] += abs(float(f)) * n + abs(float(p))
        if bias_ids is not None:
            last = {}
            for j, v in enumerate(bias_ids[m].tolist()):
                if 0 <= v < V:
                    last[v] = j
            for v, j in last.items():
                row[v] = row[v] + dtype(bias[m, j])
                S[m, v] += abs(float(bias[m, j]))
        if allowed is not None:
            words = allowed[m].view(np.uint32)
            bits = (words[:, None] >> np.arange(32, dtype=np.uint32)[None, :]) & 1
            row[bits.reshape(-1)[:V] == 0] = -np.inf
    if dtype == np.float32 and bf16:
        out = synth.bf16_values(synth.bf16_bits(out)).astype(np.float32)
    arg = np.empty(M, np.int32)
    for m in range(M):
        v = np.where(np.isnan(out[m]), -np.inf, out[m])
        arg[m] = int(np.argmax(v)) if v.max() > -np.inf else -1
    return out, S, arg


# ------------------------------------------------------------ add + RMSNorm

def _norm_inputs(M, K, seed=0):
    rng = np.random.default_rng(1000 * M + K + seed)
    x = rng.standard_normal((M, K))
    r = rng.standard_normal((M, K))
    r[:, rng.integers(0, K, 8)] *= 20.0
    if M > 2:
        r[1] = -synth.bf16_values(synth.bf16_bits(x[1]))   # sums to zero
        x[1] = -r[1]
        x[2] *= 1e-4                      # far smaller than the stream
    return synth.bf16_bits(x), synth.bf16_bits(r), synth.bf16_bits(1.0 + 0.1 * rng.standard_normal(K))


@needs_gpu
@pytest.mark.parametrize("M,K,eps", [
    (1, 128, 1e-6), (1, 5120, 1e-6), (3, 5120, 1e-5), (8, 8192, 1e-6), (5, 8320, 1e-6), (7, 17408, 1e-6),
    (2, 25600, 1e-6), (2, 32768, 1e-6), (3, 33024, 1e-6), (160, 640, 1e-6), (153, 4096, 1e-6),
    (300, 1280, 1e-6), (200, 5120, 0.0), (400, 128, 1e-3),
    # rows in four, two blocks and one
    (38, 8320, 1e-6), (39, 8320, 1e-6), (60, 17408, 0.0), (152, 18432, 1e-6), (20, 18560, 1e-6), (19, 32768, 1e-6), (154, 12288, 1e-6)])
def test_add_rmsnorm_equals_the_oracle_chain(gpu, M, K, eps):
    xb, rb, gb = _norm_inputs(M, K)
    if eps == 0.0:
        rb[1] = xb[1]                     # no zero row: the oracle's rstd would be infinite
    q0, s0, z0, h0 = ref_add_rmsnorm(xb, rb, gb, eps)
    x, r, g = (to_dev_bits(a, torch.bfloat16) for a in (xb, rb, gb))
    y = torch.empty_like(x)
    q, s, h = qlin.add_rmsnorm_act_quant_i8(x, r, g, eps, y=y)
    q16, s16, h16 = qlin.add_rmsnorm_act_quant_c16(x, r, g, eps)
    torch.cuda.synchronize()
    assert np.array_equal(from_dev_bits(h), h0) and np.array_equal(from_dev_bits(h16), h0)
    assert np.array_equal(from_dev_bits(y), z0)
    assert np.array_equal(s.cpu().numpy(), s0) and np.array_equal(s16.cpu().numpy(), s0)
    assert np.array_equal(q.cpu().numpy(), q0)
    assert np.array_equal(q16.float().cpu().numpy(), q0.astype(np.float32))
    assert not torch.signbit(q16[q16 == 0]).any()


@needs_gpu
@pytest.mark.parametrize("M,K", [(2, 640), (170, 5120), (1, 33024), (6, 17408), (40, 9088)])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_add_rmsnorm_in_place(gpu, M, K, into):
    xb, rb, gb = _norm_inputs(M, K, 1)
    q0, s0, _, h0 = ref_add_rmsnorm(xb, rb, gb, 1e-6)
    x, r, g = (to_dev_bits(a, torch.bfloat16) for a in (xb, rb, gb))
    target = x if into == "x" else r
    q, s, h = qlin.add_rmsnorm_act_quant_i8(x, r, g, 1e-6, residual_out=target)
    assert h.data_ptr() == target.data_ptr()
    assert np.array_equal(from_dev_bits(target), h0)
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)


@needs_gpu
def test_add_rmsnorm_zero_rows_and_tiny_scales(gpu):
    K = 256
    xb = synth.bf16_bits(np.zeros((3, K)))
    rb = xb.copy()
    rb[1, 5] = 0x8000                                     # -0
    rb[2] = synth.bf16_bits(np.full(K, 3.0))
    gb = synth.bf16_bits(np.full(K, 2.0 ** -126))         # scales of the smallest normal size
    x, r, g = (to_dev_bits(a, torch.bfloat16) for a in (xb, rb, gb))
    q, s, h = qlin.add_rmsnorm_act_quant_i8(x, r, g, 0.0)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert not q[:2].any() and not s[:2].any()
    # t = 1, z = 2^-126, s = z / 127 (a subnormal, so rounded coarsely), q = rint(z / s)
    z = np.float32(2.0 ** -126)
    s2 = z / np.float32(127.0)
    assert s[2] == s2 and (q[2] == min(127, int(np.rint(z / s2)))).all()


@needs_gpu
def test_add_rmsnorm_dense_code_borders(gpu):
    """Rows that sweep [-amax, amax]: quotients next to half-integers."""
    M, K = 64, 4096
    rng = np.random.default_rng(3)
    amp = np.exp(rng.uniform(np.log(1e-2), np.log(1e2), M))
    xb = synth.bf16_bits(np.linspace(-1, 1, K)[None, :] * amp[:, None])
    rb = synth.bf16_bits(0.25 * np.linspace(1, -1, K)[None, :] * amp[:, None])
    gb = synth.bf16_bits(np.ones(K))
    q0, s0, _, _ = ref_add_rmsnorm(xb, rb, gb, 1e-6)
    q, s, _ = qlin.add_rmsnorm_act_quant_i8(*(to_dev_bits(a, torch.bfloat16) for a in (xb, rb, gb)), 1e-6)
    assert np.array_equal(s.cpu().numpy(), s0) and np.array_equal(q.cpu().numpy(), q0)


# ------------------------------------------------------ per-channel product

def _channel_inputs(M, K, N, kind, seed=0):
    rng = np.random.default_rng(7 * M + 3 * K + N + seed)
    if kind == "random":
        q_a = rng.integers(-127, 128, (M, K)).astype(np.int8)
        q_w = rng.integers(-128, 128, (K, N)).astype(np.int8)
    else:   # every product of the largest size, all of one sign in half the columns
        q_a = np.full((M, K), 127, np.int8)
        q_w = np.full((K, N), -128, np.int8)
        q_w[:, 1::2] = 127
        q_w[::3, 3::4] = -127
    s_a = np.exp(rng.uniform(-6, 0, M)).astype(np.float32)
    s_w = np.exp(rng.uniform(-9, -4, N)).astype(np.float32)
    return q_a, s_a, q_w, s_w


def _channel_run(q_a, s_a, q_w, s_w, c16):
    words, _, _ = oracle.pack_gptq(q_w, 8)
    if c16:
        return qlin.gemm_w8a8_ch_c16(to_dev(q_a.astype(np.float16)), to_dev(s_a), to_dev(words), to_dev(s_w))
    return qlin.gemm_w8a8_ch(to_dev(q_a), to_dev(s_a), to_dev(words), to_dev(s_w))


CHANNEL_SHAPES = [
    (1, 128, 8), (1, 5120, 1024), (3, 384, 40), (7, 256, 200), (8, 640, 64), (8, 1152, 136), (9, 128, 72),
    (16, 1280, 1000), (17, 512, 264), (31, 2176, 328), (33, 1024, 128), (40, 1152, 264), (63, 384, 512),
    (64, 5120, 256), (65, 2048, 520), (96, 17408, 264), (97, 256, 8), (128, 1024, 136), (129, 640, 1288),
    (9, 5120, 5120), (20, 17408, 1032), (130, 5120, 1032), (33, 1152, 3208), (513, 130944, 8), (1030, 128, 8),
    (200, 3200, 392), (255, 128, 256), (257, 2304, 264), (300, 5120, 520), (513, 1152, 776), (1030, 256, 264)]


@needs_gpu
@pytest.mark.parametrize("M,K,N", CHANNEL_SHAPES)
@pytest.mark.parametrize("c16", [False, True], ids=["i8", "c16"])
def test_channel_product_is_exact(gpu, M, K, N, c16):
    args = _channel_inputs(M, K, N, "random")
    y0, y64 = ref_channel(*args)
    y = from_dev_bits(_channel_run(*args, c16))
    assert np.array_equal(y, y0)
    v = synth.bf16_values(y).astype(np.float64)
    assert (np.abs(v - y64) <= (3.03 * 2.0 ** -24 + 2.0 ** -8) * np.abs(y64)).all()


@needs_gpu
@pytest.mark.parametrize("M,K,N", [(1, 1024, 64), (5, 130944, 8), (8, 17408, 136), (20, 9344, 72), (96, 17408, 264),
                                   (130, 4096, 264), (300, 9344, 264)])
@pytest.mark.parametrize("c16", [False, True], ids=["i8", "c16"])
def test_channel_product_is_exact_at_the_largest_sums(gpu, M, K, N, c16):
    args = _channel_inputs(M, K, N, "extreme")
    y0, _ = ref_channel(*args)
    assert np.array_equal(from_dev_bits(_channel_run(*args, c16)), y0)


@needs_gpu
def test_channel_rows_do_not_depend_on_the_batch(gpu):
    q_a, s_a, q_w, s_w = _channel_inputs(300, 2304, 520, "random", 1)
    full = _channel_run(q_a, s_a, q_w, s_w, True)
    for M in (1, 8, 16, 33, 96, 128, 200):
        part = _channel_run(q_a[:M], s_a[:M], q_w, s_w, True)
        assert torch.equal(part, full[:M])


@needs_gpu
def test_channel_int8_minimum_code(gpu):
    """Int8 activation codes of -128 are taken as they are."""
    for M in (4, 70, 100, 150, 700):
        q_a = np.full((M, 1024), -128, np.int8)
        q_w = np.full((1024, 16), -128, np.int8)
        y = _channel_run(q_a, np.ones(M, np.float32), q_w, np.ones(16, np.float32), False)
        assert (y.float() == 128 * 128 * 1024).all()


@needs_gpu
@pytest.mark.parametrize("M,K,N", [(3000, 256, 520), (2500, 1152, 264), (700, 8320, 520), (1000, 2176, 2056)])
def test_channel_product_of_many_tiles(gpu, M, K, N):
    """Several token tiles a pair, bands, a last round cut along K, ragged edges."""
    args = _channel_inputs(M, K, N, "random", 3)
    y0, _ = ref_channel(*args)
    for c16 in (False, True):
        assert np.array_equal(from_dev_bits(_channel_run(*args, c16)), y0)


# Every token tile (64, 96, 128, 192), in whole tiles, in equal parts of K and in
# shares that cross tiles; ragged channel and token tiles.
TILED_SHAPES = [
    (16, 5120, 10248), (40, 2304, 8200), (64, 1280, 20488), (24, 10240, 4104), (90, 8192, 2056), (96, 2304, 8200),
    (100, 1152, 20488), (128, 5120, 4104), (120, 17408, 1544), (130, 9344, 2056), (150, 4224, 5128),
    (200, 17408, 1032), (192, 1152, 10248), (600, 1152, 5128), (300, 65536, 264),
    (24, 5120, 10248), (96, 5120, 10248), (96, 3200, 20488), (160, 10240, 10248), (128, 10240, 10248), (700, 8320, 2568),
    # few codes
    (9, 5120, 20488), (12, 5120, 12296), (40, 1536, 20488), (57, 1152, 20488)]


@needs_gpu
@pytest.mark.parametrize("M,K,N", TILED_SHAPES)
@pytest.mark.parametrize("kind", ["random", "extreme"])
def test_channel_product_in_tiles(gpu, M, K, N, kind):
    assert qlin.gemm_w8a8_ch_workspace_bytes(M, N, K) > 0
    args = _channel_inputs(M, K, N, kind, 4)
    y0, _ = ref_channel(*args)
    for c16 in (False, True):
        assert np.array_equal(from_dev_bits(_channel_run(*args, c16)), y0)


@needs_gpu
@pytest.mark.parametrize("M,K,N", [(24, 10240, 10248), (96, 10240, 10248), (128, 10240, 10248), (700, 8320, 2568)])
def test_channel_product_in_cut_tiles_again_and_again(gpu, M, K, N):
    """A captured call with one workspace, replayed over a dirty workspace, and
    four streams at once with a workspace each: guard bytes stay, y is the same."""
    args = _channel_inputs(M, K, N, "random", 6)
    y0, _ = ref_channel(*args)
    words, _, _ = oracle.pack_gptq(args[2], 8)
    q, s_a, w, s_w = to_dev(args[0].astype(np.float16)), to_dev(args[1]), to_dev(words), to_dev(args[3])
    need = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K, True)
    assert need > 0
    want = torch.from_numpy(y0.astype(np.int16)).cuda()
    streams = [torch.cuda.Stream() for _ in range(4)]
    ws = [torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda") for _ in streams]
    bufs = [torch.full((M * N + 512,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in streams]
    ys = [b[256:256 + M * N].view(M, N) for b in bufs]
    torch.cuda.synchronize()
    for i in range(12):
        with torch.cuda.stream(streams[i % 4]):
            ys[i % 4].zero_()
            qlin.gemm_w8a8_ch_c16(q, s_a, w, s_w, y=ys[i % 4], workspace=ws[i % 4][256:256 + need])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qlin.gemm_w8a8_ch_c16(q, s_a, w, s_w, y=ys[0], workspace=ws[0][256:256 + need])
    for fill in (0xFF, 0x01):
        ws[0][256:256 + need].fill_(fill)
        ys[0].zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0].view(torch.int16), want)
    for b, t in zip(bufs, ws):
        assert torch.equal(b[256:256 + M * N].view(M, N).view(torch.int16), want)
        assert (b[:256] == 7).all() and (b[256 + M * N:] == 7).all()
        assert (t[:256] == 0x5A).all() and (t[256 + need:] == 0x5A).all()


@needs_gpu
def test_channel_workspace_refusals(gpu):
    M, K, N = 24, 10240, 10248
    q = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    s, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    w = torch.zeros((K // 4, N), dtype=torch.int32, device="cuda")
    need = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K)
    need16 = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K, True)
    assert need == need16 + 2 * M * K and need16 > 0
    for call, codes, n in ((qlin.gemm_w8a8_ch, q, need), (qlin.gemm_w8a8_ch_c16, q.half(), need16)):
        with pytest.raises(qlin.QlinError) as e:
            call(codes, s, w, sw, workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
        assert e.value.status == qlin.QLIN_ERR_WORKSPACE
        with pytest.raises(ValueError):
            call(codes, s, w, sw, workspace=torch.empty(n, dtype=torch.uint8))
        with pytest.raises(TypeError):
            call(codes, s, w, sw, workspace=n)
        with pytest.raises(TypeError):
            call(codes, s, w, sw, workspace=torch.empty(n, device="cuda"))
        assert (call(codes, s, w, sw, workspace=torch.empty(n, dtype=torch.uint8, device="cuda")) == 0).all()


@needs_gpu
@pytest.mark.parametrize("M", [1, 8, 24, 96, 300])
def test_channel_writes_only_its_output(gpu, M):
    K, N = 640, 136
    args = _channel_inputs(M, K, N, "random", 2)
    y0, _ = ref_channel(*args)
    words, _, _ = oracle.pack_gptq(args[2], 8)
    buf = torch.full((M * N + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[256:256 + M * N].view(M, N)
    need = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    qlin.gemm_w8a8_ch(to_dev(args[0]), to_dev(args[1]), to_dev(words), to_dev(args[3]), y=y,
                      workspace=ws[256:256 + need] if need else None)
    assert np.array_equal(from_dev_bits(y), y0)
    assert (buf[:256] == 7).all() and (buf[256 + M * N:] == 7).all()
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()


# ----------------------------------------------------------- adjusted logits

def _logit_inputs(M, V, L, B, mask, seed):
    rng = np.random.default_rng(seed + 31 * M + V)
    x = (4.0 * rng.standard_normal((M, V))).astype(np.float32)
    kw = {}
    if L is not None:
        few = rng.integers(0, V, (M, 5))
        tok = np.where(rng.random((M, L)) < 0.6, np.take_along_axis(few, rng.integers(0, 5, (M, L)), 1),
                       rng.integers(-2, V + 3, (M, L)))
        kw["tokens"] = tok.astype(np.int32)
        kw["total"] = rng.integers(-1, L + 3, M).astype(np.int32)
        kw["prompt"] = rng.integers(-1, L + 2, M).astype(np.int32)
        kw["rep"] = rng.uniform(0.7, 1.6, M).astype(np.float32)
        kw["pres"] = rng.uniform(-0.5, 1.0, M).astype(np.float32)
        kw["freq"] = rng.uniform(-0.1, 0.3, M).astype(np.float32)
    if B is not None:
        kw["bias_ids"] = rng.integers(-2, V + 2, (M, B)).astype(np.int32)
        if B > 3:
            kw["bias_ids"][:, B // 2:] = kw["bias_ids"][:, : B - B // 2]   # every id at least twice
            if L:
                kw["bias_ids"][:, 0] = kw["tokens"][:, 0]
        kw["bias"] = (5 * rng.standard_normal((M, B))).astype(np.float32)
    if mask:
        kw["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (M, (V + 31) // 32)).astype(np.int32)
        if M > 1:
            kw["allowed"][1] = 0          # a row that allows nothing
    return x, kw


_NAMES = {"prompt": "prompt_len", "total": "total_len", "rep": "repetition", "pres": "presence", "freq": "frequency"}


def _check_logits(x, kw, bf16, in_place=False):
    dt = torch.bfloat16 if bf16 else torch.float32
    if bf16:
        x = synth.bf16_values(synth.bf16_bits(x)).astype(np.float32)
    dev = to_dev(x).to(dt)
    args = {_NAMES.get(k, k): to_dev(v) for k, v in kw.items()}
    o32, _, arg = ref_logits(x, bf16, **kw)
    o64, S, _ = ref_logits(x, bf16, dtype=np.float64, **kw)
    only = qlin.adjust_logits_argmax(dev, **args)
    assert np.array_equal(only.cpu().numpy(), arg)
    out = dev if in_place else torch.empty_like(dev)
    token = qlin.adjust_logits_argmax(dev, **args, out=out)
    got = out.float().cpu().numpy()
    assert np.array_equal(got, o32, equal_nan=True)
    assert np.array_equal(token.cpu().numpy(), arg)
    fine = np.isfinite(o64)
    off = np.abs(got[fine].astype(np.float64) - o64[fine])
    assert (off <= 5 * 2.0 ** -24 * S[fine] + (2.0 ** -8 if bf16 else 0.0) * np.abs(o64[fine])).all()


@needs_gpu
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,V,L,B,mask", [
    (1, 8, 3, 2, True), (1, 1000, None, None, False), (2, 1000, 0, 0, True), (3, 4104, 1, 1, False),
    (5, 8200, 700, 9, True), (2, 50264, 300, 600, True), (1, 248320, 2000, 16, True), (33, 50264, 515, None, False),
    (3, 151936, None, 40, True), (160, 2056, 64, 5, True), (400, 4096, 20, 3, True), (2, 400008, 3000, 30, True),
    # more touched tokens than the table takes: windows of them; many bias entries
    (2, 9000, 30000, 1700, True), (330, 6000, 5000, 3, False), (1, 4096, 20000, 9000, True), (3, 40000, 60000, 0, False),
    # slices of several parts
    (10, 700008, 900, 20, True)])
def test_adjusted_logits(gpu, M, V, L, B, mask, bf16):
    x, kw = _logit_inputs(M, V, L, B, mask, 5)
    _check_logits(x, kw, bf16)


@needs_gpu
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_adjusted_logits_in_place_and_defaults(gpu, bf16):
    x, kw = _logit_inputs(4, 9000, 200, 12, True, 9)
    _check_logits(x, kw, bf16, in_place=True)
    for drop in (("prompt",), ("total",), ("rep",), ("pres", "freq"), ("prompt", "total", "rep", "pres", "freq")):
        _check_logits(x, {k: v for k, v in kw.items() if k not in drop}, bf16)


@needs_gpu
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_adjusted_logits_special_values(gpu, bf16):
    M, V = 6, 4160
    x, kw = _logit_inputs(M, V, 50, 8, False, 11)
    x = synth.bf16_values(synth.bf16_bits(x)).astype(np.float32)
    kw["bias_ids"][:] = -1
    kw["tokens"][:] = -1
    allowed = np.full((M, (V + 31) // 32), -1, np.int32)
    x[0, 10] = np.nan
    x[0, 40] = np.inf
    allowed[0, 0] = ~(1 << 10)                       # the NaN is masked
    allowed[0, 1] = ~(1 << 8)                        # and so is the infinity
    x[1, :] = -np.inf                                # nothing above -inf
    x[2, :] = np.nan
    x[2, 4159] = -3.0                                # NaN is never the greedy token
    x[3, :] = -1.0
    x[3, [7, 100, 4000]] = 0.0
    x[3, 7] = -0.0                                   # -0 equals +0: the lowest index
    x[4, [4100, 33, 2000]] = 500.0                   # ties
    x[5, 17] = np.inf
    kw["tokens"][5, :] = 17                          # inf through every penalty
    kw["total"][5] = 50
    kw["allowed"] = allowed
    dt = torch.bfloat16 if bf16 else torch.float32
    args = {_NAMES.get(k, k): to_dev(v) for k, v in kw.items()}
    out = torch.empty((M, V), dtype=dt, device="cuda")
    token = qlin.adjust_logits_argmax(to_dev(x).to(dt), **args, out=out).cpu().numpy()
    got = out.float().cpu().numpy()
    o32, _, _ = ref_logits(x, bf16, **kw)
    assert np.array_equal(got, o32, equal_nan=True)
    assert got[0, 10] == -np.inf and got[0, 40] == -np.inf
    assert token[1] == -1 and token[2] == 4159 and token[3] == 7 and token[4] == 33 and token[5] == 17


@needs_gpu
def test_adjusted_logits_leave_other_memory(gpu):
    M, V = 3, 5000
    x, kw = _logit_inputs(M, V, 100, 9, True, 13)
    buf = torch.full((M * V + 1024,), 3.0, dtype=torch.float32, device="cuda")
    out = buf[512:512 + M * V].view(M, V)
    args = {_NAMES.get(k, k): to_dev(v) for k, v in kw.items()}
    qlin.adjust_logits(to_dev(x), **args, out=out)
    o32, _, _ = ref_logits(x, False, **kw)
    assert np.array_equal(out.cpu().numpy(), o32)
    assert (buf[:512] == 3).all() and (buf[512 + M * V:] == 3).all()


# ------------------------------------------------------- the run of them all

def _chain_inputs(M, K, N, seed):
    rng = np.random.default_rng(seed)
    xb, rb, gb = _norm_inputs(M, K, seed)
    q_w = rng.integers(-127, 128, (K, N)).astype(np.int8)
    s_w = np.exp(rng.uniform(-9, -7, N)).astype(np.float32)
    tokens = rng.integers(0, N, (M, 40)).astype(np.int32)
    allowed = rng.integers(-2 ** 31, 2 ** 31, (M, (N + 31) // 32)).astype(np.int32)
    return xb, rb, gb, q_w, s_w, tokens, allowed


def _chain_ref(xb, rb, gb, q_w, s_w, tokens, allowed, pen):
    q, s, _, h = ref_add_rmsnorm(xb, rb, gb, 1e-6)
    y, _ = ref_channel(q, s, q_w, s_w)
    o, _, arg = ref_logits(synth.bf16_values(y).astype(np.float32), True, tokens=tokens, rep=pen, freq=pen,
                           allowed=allowed)
    return h, y, o, arg


@needs_gpu
@pytest.mark.parametrize("M", [1, 8, 40, 200])
@pytest.mark.parametrize("codes", ["i8", "c16"])
def test_step_from_the_stream_to_the_token(gpu, M, codes):
    """Residual stream -> codes -> vocabulary head -> adjusted greedy token, on
    a side stream, captured once and replayed on new inputs."""
    K, N = 640, 4104
    first = _chain_inputs(M, K, N, 21)
    second = _chain_inputs(M, K, N, 22)
    pen = np.full(M, 1.25, np.float32)
    words, _, _ = oracle.pack_gptq(first[3], 8)
    x, r, g = (to_dev_bits(a, torch.bfloat16) for a in first[:3])
    qw, sw, tok, ok, pn = to_dev(words), to_dev(first[4]), to_dev(first[5]), to_dev(first[6]), to_dev(pen)

    def step():
        if codes == "i8":
            q, s, h = qlin.add_rmsnorm_act_quant_i8(x, r, g, 1e-6)
            y = qlin.gemm_w8a8_ch(q, s, qw, sw)
        else:
            q, s, h = qlin.add_rmsnorm_act_quant_c16(x, r, g, 1e-6)
            y = qlin.gemm_w8a8_ch_c16(q, s, qw, sw)
        out = torch.empty_like(y)
        return h, y, out, qlin.adjust_logits_argmax(y, tokens=tok, repetition=pn, frequency=pn, allowed=ok, out=out)

    def check(got, inputs):
        h0, y0, o0, arg0 = _chain_ref(*inputs[:3], first[3], first[4], inputs[5], inputs[6], pen)
        h, y, o, arg = got
        assert np.array_equal(from_dev_bits(h), h0) and np.array_equal(from_dev_bits(y), y0)
        assert np.array_equal(o.float().cpu().numpy(), o0) and np.array_equal(arg.cpu().numpy(), arg0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    check(got, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for inputs in (second, first):
        for t, a in ((x, inputs[0]), (r, inputs[1]), (g, inputs[2])):
            t.copy_(to_dev_bits(a, torch.bfloat16))
        tok.copy_(to_dev(inputs[5]))
        ok.copy_(to_dev(inputs[6]))
        graph.replay()
        torch.cuda.synchronize()
        check(got, inputs)


@needs_gpu
def test_two_streams_at_once(gpu):
    """Calls with default workspaces on two streams do not meet."""
    shapes = [(8, 5120, 1032), (200, 2304, 1032)]
    inputs = [_channel_inputs(*s, "random", 5) for s in shapes]
    refs = [ref_channel(*a)[0] for a in inputs]
    dev = []
    for q_a, s_a, q_w, s_w in inputs:
        words, _, _ = oracle.pack_gptq(q_w, 8)
        dev.append((to_dev(q_a), to_dev(s_a), to_dev(words), to_dev(s_w)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 4]):
            got.append((i % 2, qlin.gemm_w8a8_ch(*dev[i % 2])))
    explicit = qlin.gemm_w8a8_ch(*dev[1], stream=streams[0])
    by_handle = qlin.gemm_w8a8_ch(*dev[1], stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(explicit, by_handle)
    for k, y in got:
        assert np.array_equal(from_dev_bits(y), refs[k])
    assert np.array_equal(from_dev_bits(explicit), refs[1])


@needs_gpu
@pytest.mark.parametrize("by_handle", [False, True], ids=["stream", "handle"])
def test_a_named_stream_leaves_freed_memory_of_the_current_one(gpu, by_handle):
    """The current stream holds work on a tensor that was freed: what a call on
    another stream allocates must not be its memory."""
    M, K, N = 64, 10240, 10248
    shape = (M, K)
    x = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    codes = torch.ones(shape, dtype=torch.float16, device="cuda")
    w, s_w = torch.zeros((K // 4, N), dtype=torch.int32, device="cuda"), torch.ones(N, device="cuda")
    s_a = torch.ones(M, device="cuda")
    logits = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    stream = side.cuda_stream if by_handle else side
    need = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K, True)
    assert need > 0
    calls = [(lambda: qlin.add_rmsnorm_act_quant_c16(x, x, g, 1e-6, stream=stream), (M * K * 2,)),
             (lambda: qlin.gemm_w8a8_ch_c16(codes, s_a, w, s_w, stream=stream), (M * N * 2, need)),
             (lambda: qlin.adjust_logits(logits, repetition=s_a, stream=stream), (M * N * 2,))]
    for call, sizes in calls:
        call()
        torch.cuda.synchronize()
        held = [torch.full((n,), 0x35, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        kept = [torch.empty_like(t) for t in held]
        torch.cuda._sleep(50_000_000)
        for k, t in zip(kept, held):
            k.copy_(t)
        del held, t
        call()
        torch.cuda.synchronize()
        for k in kept:
            assert (k == 0x35).all()


@needs_gpu
def test_threads_and_a_replay_beside_eager_calls(gpu):
    """Four threads on streams of their own, and a captured step replayed while
    another stream runs the same step eagerly: no two calls meet."""
    M, K, N = 64, 5120, 10248
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    w = torch.empty((K // 4, N), dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    s_w = torch.rand(N, generator=g, device="cuda")
    tokens = torch.randint(0, N, (M, 20), generator=g, device="cuda", dtype=torch.int32)
    rep = torch.full((M,), 1.5, device="cuda")

    def step():
        q, s, _ = qlin.add_rmsnorm_act_quant_c16(x, x, gamma, 1e-6)
        y = qlin.gemm_w8a8_ch_c16(q, s, w, s_w)
        return y, qlin.adjust_logits_argmax(y, tokens=tokens, repetition=rep)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step()
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i] = step()
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for _ in range(20):
        graph.replay()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for y, token in [replayed, *got]:
        assert torch.equal(y, want[0]) and torch.equal(token, want[1])


# --------------------------------------------- offsets of more than 32 bits

def _channel_sampled(q_a, s_a, w, s_w, y, rows, cols):
    codes = torch.stack([(w[:, cols] >> (8 * i)) & 255 for i in range(4)], 1).reshape(-1, len(cols)) - 128
    P = q_a[rows].double() @ codes.double()
    want = ((P.float() * s_w[cols]) * s_a[rows, None]).bfloat16()
    assert torch.equal(y[rows][:, cols], want)


@needs_gpu
@pytest.mark.parametrize("M,K,N", [(9000, 128, 248320), (9000, 1280, 248320), (5, 130944, 65544), (16, 130944, 65544)])
def test_channel_product_past_32_bits(gpu, M, K, N):
    """Outputs, and weights, whose last elements lie past 2^31."""
    assert max(M * N, K // 4 * N) > 2 ** 31 - 2 ** 26
    g = torch.Generator("cuda").manual_seed(M + K)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.empty((K // 4, N), dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    s_a, s_w = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = qlin.gemm_w8a8_ch(q, s_a, w, s_w)
    rows = torch.tensor(sorted({0, M // 2, M - 2, M - 1}), device="cuda")
    cols = torch.cat([torch.arange(0, 40), torch.randint(0, N, (200,)), torch.arange(N - 40, N)]).cuda()
    _channel_sampled(q, s_a, w, s_w, y, rows, cols)


@needs_gpu
def test_add_rmsnorm_past_32_bits(gpu):
    M, K = 125000, 17408
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    r = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = torch.rand(K, generator=g, device="cuda").bfloat16()
    q, s, h = qlin.add_rmsnorm_act_quant_i8(x, r, gamma, 1e-6)
    rows = torch.tensor([0, 123361, M - 1], device="cuda")     # 123361 * 17408 passes 2^31
    q0, s0, _, h0 = ref_add_rmsnorm(from_dev_bits(x[rows]), from_dev_bits(r[rows]), from_dev_bits(gamma), 1e-6)
    assert np.array_equal(from_dev_bits(h[rows]), h0) and np.array_equal(q[rows].cpu().numpy(), q0)
    assert np.array_equal(s[rows].cpu().numpy(), s0)


@needs_gpu
@pytest.mark.parametrize("rules", [False, True])
def test_adjusted_logits_past_32_bits(gpu, rules):
    M, V, L = 8800, 248320, 40
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn((M, V), generator=g, device="cuda", dtype=torch.bfloat16)
    allowed = torch.empty((M, V // 32), dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    kw = {"allowed": allowed}
    if rules:
        kw["tokens"] = torch.randint(0, V, (M, L), generator=g, device="cuda", dtype=torch.int32)
        kw["repetition"] = 1.0 + torch.rand(M, generator=g, device="cuda")
        kw["frequency"] = torch.rand(M, generator=g, device="cuda")
    out = torch.empty_like(x)
    best = qlin.adjust_logits_argmax(x, **kw, out=out)
    rows = torch.tensor([0, 8648, M - 1], device="cuda")       # 8648 * 248320 passes 2^31
    few = {"allowed": allowed[rows].cpu().numpy()}
    if rules:
        few.update(tokens=kw["tokens"][rows].cpu().numpy(), rep=kw["repetition"][rows].cpu().numpy(),
                   freq=kw["frequency"][rows].cpu().numpy())
    o0, _, arg0 = ref_logits(x[rows].float().cpu().numpy(), True, **few)
    assert np.array_equal(out[rows].float().cpu().numpy(), o0)
    assert np.array_equal(best[rows].cpu().numpy(), arg0)


@needs_gpu
def test_empty_batches(gpu):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q, s, h = qlin.add_rmsnorm_act_quant_i8(x, x, g, 1e-6)
    assert q.shape == (0, 256) and s.shape == (0,) and h.shape == (0, 256)
    w = torch.zeros((64, 16), dtype=torch.int32, device="cuda")
    y = qlin.gemm_w8a8_ch(q, s, w, torch.ones(16, device="cuda"))
    assert y.shape == (0, 16)
    assert qlin.adjust_logits_argmax(y).shape == (0,)


@needs_gpu
def test_refused_tensors(gpu):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        qlin.add_rmsnorm_act_quant_i8(x.half(), x, g, 1e-6)
    with pytest.raises(ValueError):
        qlin.add_rmsnorm_act_quant_i8(x, x[:, ::2], g, 1e-6)
    with pytest.raises(ValueError):
        qlin.add_rmsnorm_act_quant_i8(x, x.cpu(), g, 1e-6)
    with pytest.raises(ValueError):
        qlin.add_rmsnorm_act_quant_i8(x, x, g, 1e-6, q=torch.empty((3, 256), dtype=torch.int8, device="cuda"))
    with pytest.raises(qlin.QlinError) as e:
        qlin.add_rmsnorm_act_quant_i8(x, x, g, float("nan"))
    assert e.value.status == qlin.QLIN_ERR_SHAPE
    q, s, _ = qlin.add_rmsnorm_act_quant_i8(x, x, g, 1e-6)
    w = torch.zeros((64, 16), dtype=torch.int32, device="cuda")
    sw = torch.ones(16, device="cuda")
    with pytest.raises(TypeError):
        qlin.gemm_w8a8_ch(q, s, w, sw.half())
    with pytest.raises(TypeError):
        qlin.gemm_w8a8_ch_c16(q, s, w, sw)
    with pytest.raises(ValueError):
        qlin.gemm_w8a8_ch(q, s, w[:32], sw)
    with pytest.raises(ValueError):
        qlin.gemm_w8a8_ch(q, s[::2], w, sw)
    with pytest.raises(qlin.QlinError) as e:
        qlin.gemm_w8a8_ch(q, s, torch.zeros((64, 12), dtype=torch.int32, device="cuda"), sw[:12].clone())
    assert e.value.status == qlin.QLIN_ERR_SHAPE
    logits = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    ints = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        qlin.adjust_logits(logits, bias_ids=ints)
    with pytest.raises(ValueError):
        qlin.adjust_logits(logits, prompt_len=ints[:, 0].contiguous())
    with pytest.raises(ValueError):
        qlin.adjust_logits(logits, allowed=ints[:, :1].contiguous())
    with pytest.raises(TypeError):
        qlin.adjust_logits(logits, tokens=ints.long())
    with pytest.raises(TypeError):
        qlin.adjust_logits(logits.half())
    for call in (qlin.adjust_logits, qlin.adjust_logits_argmax):
        with pytest.raises(TypeError):
            call([1.0])
        with pytest.raises(ValueError):
            call(logits[0])
        with pytest.raises(ValueError):
            call(logits[:, ::2])
    with pytest.raises(ValueError):
        qlin.adjust_logits(logits, out=torch.empty((4, 128), dtype=torch.bfloat16, device="cuda")[:, ::2])


# -------------------------------------- argument checks of the C ABI (no GPU)

def _p(n):
    return ctypes.c_void_p(n)


OK, ODD = 0x1000, 0x1008      # never dereferenced: every call below is refused


def _status(lib, name, *args):
    return int(getattr(lib, name)(*args))


@pytest.mark.parametrize("name", ["qlin_add_rmsnorm_act_quant_i8", "qlin_add_rmsnorm_act_quant_c16"])
def test_add_rmsnorm_refusals(lib, name):
    def call(x=OK, r=OK, g=OK, eps=1e-6, M=4, K=256, h=OK, q=OK, s=OK, y=None):
        return _status(lib, name, _p(x), _p(r), _p(g), eps, M, K, _p(h), _p(q), _p(s), _p(y), None)
    for kw in ({"x": None}, {"r": None}, {"g": None}, {"h": None}, {"q": None}, {"s": None}):
        assert call(**kw) == qlin.QLIN_ERR_NULL
    for kw in ({"M": -1}, {"K": 0}, {"K": 200}, {"K": 2 ** 31}, {"M": 2 ** 31}, {"eps": -1e-6},
               {"eps": float("inf")}, {"eps": float("nan")}):
        assert call(**kw) == qlin.QLIN_ERR_SHAPE
    for kw in ({"x": ODD}, {"r": ODD}, {"g": ODD}, {"h": ODD}, {"q": ODD}, {"s": ODD}, {"y": ODD}):
        assert call(**kw) == qlin.QLIN_ERR_ALIGN


def test_channel_refusals(lib):
    def i8(q=OK, s=OK, w=OK, sw=OK, M=4, N=64, K=256, y=OK, ws=None, n=0):
        return _status(lib, "qlin_gemm_w8a8_ch", _p(q), _p(s), _p(w), _p(sw), M, N, K, _p(y), _p(ws), n, None)

    def c16(q=OK, s=OK, w=OK, sw=OK, M=4, N=64, K=256, y=OK, ws=None, n=0):
        return _status(lib, "qlin_gemm_w8a8_ch_c16", _p(q), _p(s), _p(w), _p(sw), M, N, K, _p(y), _p(ws), n, None)
    for call in (i8, c16):
        for kw in ({"q": None}, {"s": None}, {"w": None}, {"sw": None}, {"y": None}):
            assert call(**kw) == qlin.QLIN_ERR_NULL
        for kw in ({"M": -1}, {"N": 12}, {"N": 0}, {"K": 64}, {"K": 0}, {"K": 131072}, {"N": 2 ** 31}, {"M": 2 ** 31}):
            assert call(**kw) == qlin.QLIN_ERR_SHAPE
        for kw in ({"q": ODD}, {"s": ODD}, {"w": ODD}, {"sw": ODD}, {"y": ODD}):
            assert call(**kw) == qlin.QLIN_ERR_ALIGN
        assert call(ws=ODD, n=1 << 30) == qlin.QLIN_ERR_ALIGN
    for M, N, K in ((-1, 64, 256), (4, 12, 256), (4, 64, 100), (4, 64, 131072), (0, 64, 256)):
        assert qlin.gemm_w8a8_ch_workspace_bytes(M, N, K) == 0
        assert qlin.gemm_w8a8_ch_workspace_bytes(M, N, K, True) == 0


@pytest.mark.parametrize("name", ["qlin_adjust_logits_bf16", "qlin_adjust_logits_f32"])
def test_adjust_logits_refusals(lib, name):
    def call(x=OK, M=2, V=64, tok=None, L=0, pl=None, tl=None, rep=None, pres=None, freq=None, ids=None, b=None,
             B=0, ok=None, out=OK, arg=None):
        return _status(lib, name, _p(x), M, V, _p(tok), L, _p(pl), _p(tl), _p(rep), _p(pres), _p(freq), _p(ids),
                       _p(b), B, _p(ok), _p(out), _p(arg), None)
    for kw in ({"x": None}, {"out": None}, {"L": 3}, {"B": 2}, {"B": 2, "ids": OK}, {"B": 2, "b": OK}):
        assert call(**kw) == qlin.QLIN_ERR_NULL
    for kw in ({"M": -1}, {"V": 0}, {"V": 12}, {"V": 2 ** 31}, {"L": -1}, {"B": -1}, {"L": 2 ** 31, "tok": OK}):
        assert call(**kw) == qlin.QLIN_ERR_SHAPE
    for kw in ({"x": ODD}, {"out": ODD}, {"tok": 0x1002, "L": 2}, {"arg": 0x1002}, {"rep": 0x1001}, {"ok": 0x1002},
               {"pl": 0x1002}, {"tl": 0x1002}, {"pres": 0x1002}, {"freq": 0x1002},
               {"ids": 0x1002, "b": OK, "B": 1}, {"ids": OK, "b": 0x1002, "B": 1}):
        assert call(**kw) == qlin.QLIN_ERR_ALIGN
    if not torch.cuda.is_available():
        assert call() == qlin.QLIN_ERR_DEVICE


def test_cpu_tensors_are_refused(lib):
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    g = torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        qlin.add_rmsnorm_act_quant_i8(x, x, g, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        qlin.gemm_w8a8_ch(torch.zeros((2, 256), dtype=torch.int8), torch.ones(2),
                          torch.zeros((64, 16), dtype=torch.int32), torch.ones(16))
    with pytest.raises(ValueError, match="CUDA"):
        qlin.adjust_logits_argmax(torch.zeros((2, 64)))
