"""The stream that a call of the per-channel path runs on when one is named."""
import pytest
import torch

from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qlin.load()


def stream_of(named):
    """The handle of the stream that is current inside a call with stream=named."""
    seen = []
    lead = torch.empty(1, device="cuda")

    def call(t):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return t
    assert qlin._on(named, lead, call, lead) is lead
    return seen[0]


class Handle:
    def __init__(self, value):
        self.cuda_stream = value


@pytest.mark.parametrize("make", [int, Handle], ids=["int", "object"])
def test_handle_0_is_the_default_stream(make):
    """What torch.cuda.current_stream().cuda_stream gives where no other stream
    is current, and NULL in the C interface."""
    assert torch.cuda.default_stream().cuda_stream == 0
    side = torch.cuda.Stream()
    assert stream_of(make(0)) == 0 and stream_of(make(1)) == 0       # 1: cudaStreamLegacy
    with torch.cuda.stream(side):
        assert stream_of(make(0)) == 0
        assert stream_of(torch.cuda.default_stream()) == 0
        assert stream_of(make(side.cuda_stream)) == side.cuda_stream
    assert stream_of(make(side.cuda_stream)) == side.cuda_stream
    assert stream_of(side) == side.cuda_stream
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_calls_on_handle_0_follow_the_default_stream():
    """Inputs written on the default stream just before, behind a long wait."""
    M, K, N = 4, 1024, 512
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    w = torch.empty((K // 4, N), dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    s_w = torch.rand(N, generator=g, device="cuda")

    def step(x, **kw):
        q, s, h = qlin.add_rmsnorm_act_quant_i8(x, x, gamma, 1e-6, **kw)
        y = qlin.gemm_w8a8_ch(q, s, w, s_w, **kw)
        return h, q, s, y, qlin.adjust_logits_argmax(y, **kw)

    want = step(x)
    torch.cuda.synchronize()
    for _ in range(4):
        late = torch.zeros_like(x)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
        got = step(late, stream=0)
        copies = [t.clone() for t in got]      # on the default stream again
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, copies):
            assert torch.equal(a, b) and torch.equal(a, c)
