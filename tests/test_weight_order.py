"""A product directly behind the call that writes its weights, on one stream.

The products read weights before they wait for the kernel in front of them, so
the calls that write weights have to leave them complete.  Every round packs
other weights into the same memory: a word read too early is of the round
before.  All checks are equalities of integers, or with a reference product on
weights that have long been there."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin

pytestmark = pytest.mark.gpu
ROUNDS = 6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qlin.load()
    yield
    torch.cuda.synchronize()
    assert qlin.device_status() == qlin.QLIN_OK


def weights(K, N, bits, g):
    half = 1 << (bits - 1)
    return [torch.randint(-half, half, (K, N), generator=g, device="cuda", dtype=torch.int8) for _ in range(ROUNDS)]


def product(q, w, s_a, s_w):
    """The per-channel product's definition; the sums are integers below 2^53."""
    P = q.double() @ w.double()
    return ((P.float() * s_w) * s_a[:, None]).bfloat16()


# streaming kernel; pairs whose clusters share tiles; pairs with whole tiles and cut ones
@pytest.mark.parametrize("M,K,N", [(1, 512, 8192), (8, 1024, 8200), (64, 2048, 4096), (96, 1024, 20488),
                                   (200, 1280, 10248)])
@pytest.mark.parametrize("zeros", [False, True], ids=["words", "words_and_qzeros"])
def test_channel_product_behind_the_packer(M, K, N, zeros):
    g = torch.Generator("cuda").manual_seed(M + N)
    ws = weights(K, N, 8, g)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    s_a, s_w = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    words = torch.zeros((K // 4, N), dtype=torch.int32, device="cuda")
    need = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    ys = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in ws]

    def all_rounds():
        for w, y in zip(ws, ys):
            qlin.pack_gptq(w, 8, qweight=words, with_qzeros=zeros)
            qlin.gemm_w8a8_ch(q, s_a, words, s_w, y=y, workspace=scratch)

    def check():
        torch.cuda.synchronize()
        for w, y in zip(ws, ys):
            assert torch.equal(y, product(q, w, s_a, s_w))
            y.zero_()

    all_rounds()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_rounds()
    for _ in range(3):
        graph.replay()
    check()


@pytest.mark.parametrize("M", [8, 96])
def test_channel_product_behind_the_ingest(M):
    K, N = 1024, 10248
    g = torch.Generator("cuda").manual_seed(M)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    s_a, s_w = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    ws = weights(K, N, 8, g)
    packed = [qlin.pack_gptq(w, 8, with_qzeros=False)[0].t().contiguous() for w in ws]
    group = torch.ones((N, K // 128), dtype=torch.float16, device="cuda")
    qlin.ingest_nk(packed[0], group, K, 8)
    torch.cuda.synchronize()
    ys = []
    for p in packed:      # the allocator hands out the words' memory again
        words, _ = qlin.ingest_nk(p, group, K, 8)
        ys.append(qlin.gemm_w8a8_ch(q, s_a, words, s_w))
        del words
    torch.cuda.synchronize()
    for w, y in zip(ws, ys):
        assert torch.equal(y, product(q, w, s_a, s_w))


@pytest.mark.parametrize("M", [1, 8, 64])
def test_group_products_behind_the_packers(M):
    """W8A8 in both layouts and W4A16, against the same call on weights at rest."""
    K, N = 1024, 8200
    g = torch.Generator("cuda").manual_seed(M)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    s_a = torch.rand(M, generator=g, device="cuda")
    s8 = to_dev(np.full((K // 128, N), 0.01, np.float16))
    s4 = torch.full((K // 128, N), 0.02, dtype=torch.bfloat16, device="cuda")
    space = qlin.Workspace()
    ws8, ws4 = weights(K, N, 8, g), weights(K, N, 4, g)

    def calls(words8, words4):
        return (lambda: qlin.gemm_w8a8_gs128(q, s_a, words8, s8, workspace=space),
                lambda: qlin.gemm_w4a16_g128(x, words4, s4, workspace=space))

    rest = []
    for w8, w4 in zip(ws8, ws4):
        a, b = qlin.pack_gptq(w8, 8)[0], qlin.pack_gptq(w4, 4)[0]
        torch.cuda.synchronize()
        rest.append([c() for c in calls(a, b)])
        torch.cuda.synchronize()
    words8 = torch.zeros((K // 4, N), dtype=torch.int32, device="cuda")
    words4 = torch.zeros((K // 8, N), dtype=torch.int32, device="cuda")
    tiled = []
    got = []
    for w8, w4 in zip(ws8, ws4):
        f8, f4 = calls(words8, words4)
        qlin.pack_gptq(w8, 8, qweight=words8, with_qzeros=False)
        y8 = f8()
        qlin.pack_gptq(w4, 4, qweight=words4, with_qzeros=False)
        y4 = f4()
        t = qlin.pack_tiles(words8, K, 8)
        tiled.append(qlin.gemm_w8a8_gs128_tiled(q, s_a, t, s8, workspace=space))
        del t
        got.append([y8, y4])
    torch.cuda.synchronize()
    for (a8, a4), (b8, b4), t in zip(rest, got, tiled):
        assert torch.equal(a8, b8) and torch.equal(a4, b4) and torch.equal(a8, t)
