"""The per-channel product in every form that it takes (channel_forms), bit for
bit: random codes, int8 ones down to -128, and codes whose sums are the largest
there are, with guarded outputs and guarded, dirty workspaces.  P is summed in
binary64, exact below 2^53, and put through the definition's two fp32 products."""
import pytest
import torch

import channel_plan as cp
from channel_forms import FORMS
from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin

pytestmark = pytest.mark.gpu
GUARD = 256


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qlin.load()
    yield
    torch.cuda.synchronize()
    assert qlin.device_status() == qlin.QLIN_OK


def inputs(M, K, N, kind):
    g = torch.Generator("cuda").manual_seed(M * 7 + K + N)
    if kind == "random":
        q = torch.randint(-128, 128, (M, K), generator=g, device="cuda")
        w = torch.randint(-128, 128, (K, N), generator=g, device="cuda")
    else:                 # products of -128 and of one sign: sums of 2^14 K
        q = torch.full((M, K), -128, device="cuda")
        w = torch.full((K, N), -128, device="cuda")
        w[:, 1::2] = 127
        w[::3, 3::4] = -127
    words = torch.zeros((K // 4, N), dtype=torch.int64, device="cuda")
    for i in range(4):
        words |= (w[i::4] + 128) << (8 * i)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    s_a = torch.exp(torch.rand(M, generator=g, device="cuda") * 6 - 6)
    s_w = torch.exp(torch.rand(N, generator=g, device="cuda") * 5 - 9)
    return q, s_a, w, words, s_w


@pytest.mark.parametrize("size", list(FORMS), ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", ["random", "extreme"])
def test_every_form_bit_for_bit(size, kind):
    M, K, N = size
    q, s_a, w, words, s_w = inputs(M, K, N, kind)
    for c16 in (False, True):
        codes = q.clamp(min=-127).half() if c16 else q.to(torch.int8)
        P = codes.double() @ w.double()
        want = ((P.float() * s_w) * s_a[:, None]).bfloat16()
        need = qlin.gemm_w8a8_ch_workspace_bytes(M, N, K, c16)
        # a tile's kernel reads int8 codes through the workspace, so it has one
        assert (need > 0) == (FORMS[size][0] == "pair") or c16
        space = torch.full((need + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((M * N + 2 * GUARD,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = out[GUARD:GUARD + M * N].view(M, N)
        call = qlin.gemm_w8a8_ch_c16 if c16 else qlin.gemm_w8a8_ch
        for fill in (0xA5, 0xFF):       # what the workspace holds before the call
            space[GUARD:GUARD + need].fill_(fill)
            y.fill_(3.0)
            call(codes, s_a, words, s_w, y=y, workspace=space[GUARD:GUARD + need] if need else None)
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        assert (out[:GUARD] == 7).all() and (out[GUARD + M * N:] == 7).all()
        assert (space[:GUARD] == 0xA5).all() and (space[GUARD + need:] == 0xA5).all()


def test_rows_are_the_same_in_every_form():
    """A row of y does not depend on the rows beside it: one batch in pieces
    that stream, in tiles of every size, whole and cut."""
    K, N = 1152, 12152
    sizes = (1, 8, 9, 40, 72, 100, 140, 300, 700)
    assert {cp.form(M, K, N)[0] for M in sizes} == {"stream", "pair"}
    assert len({cp.form(M, K, N)[1:2] for M in sizes if M > 8}) >= 3
    q, s_a, _, words, s_w = inputs(max(sizes), K, N, "random")
    codes = q.to(torch.int8)
    whole = qlin.gemm_w8a8_ch(codes, s_a, words, s_w)
    for M in sizes:
        assert torch.equal(qlin.gemm_w8a8_ch(codes[:M], s_a[:M], words, s_w).view(torch.int16), whole[:M].view(torch.int16))


# Tiles that wait behind cut ones, whose sums take long to meet: the rings run
# full there, as they seldom do elsewhere.
BEHIND_CUT = [(259, 6400, 15888), (393, 14080, 10744), (986, 10496, 5744), (343, 9472, 14768), (700, 8320, 2568)]


@pytest.mark.parametrize("size", [s for s in FORMS if FORMS[s][0] == "pair"] + BEHIND_CUT,
                         ids=lambda s: "x".join(map(str, s)))
def test_the_same_call_again_and_again(size):
    """200 runs, some of them back to back: all bit for bit the definition's."""
    M, K, N = size
    q, s_a, w, words, s_w = inputs(M, K, N, "random")
    codes = q.clamp(min=-127).half()
    want = (((codes.double() @ w.double()).float() * s_w) * s_a[:, None]).bfloat16().view(torch.int16)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(200):
        qlin.gemm_w8a8_ch_c16(codes, s_a, words, s_w, y=y)
        wrong += (y.view(torch.int16) != want).any()
        if i % 3 == 0:
            torch.cuda.synchronize()
    assert int(wrong) == 0
