"""The bound that the header gives for qll_token_logprobs, on every float output:
2^-18 (1 + |value|).  Rows of all kinds that the sums' references go through:
flat ones (the weight lies far below the largest logit), steps that start up to
the reference's slack of 16 below the rest, a lane whose reference moves a little
in every step because its neighbour's moves a lot, rising and masked ones."""
import pytest
import torch

import quantized_linear_layer_amd as qll
from gpu_util import DEV, empty

pytestmark = pytest.mark.gpu

CODE = {torch.float32: qll.QLL_DTYPE_F32, torch.bfloat16: qll.QLL_DTYPE_BF16, torch.float16: qll.QLL_DTYPE_F16}
BOUND = 2.0 ** -18


def assert_published_bound(x, top=5, given=8):
    m, v = x.shape
    g = torch.Generator(device=DEV).manual_seed(v)
    tokens = torch.randint(0, v, (m, given), generator=g, device=DEV, dtype=torch.int32)
    lp, en, tl = (torch.empty(*s, device=DEV) for s in ((m, given), (m,), (m, top)))
    ids = empty(m * top, torch.int32)
    ws = empty(qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, m, v, top))
    qll.qll_token_logprobs(x, CODE[x.dtype], tokens, given, lp, en, top, ids, tl, m, v, ws=ws)
    ids = ids.view(m, top)
    for i in range(0, m, 64):
        rows = slice(i, i + 64)
        d = x[rows].double()
        d = d - d.amax(1, keepdim=True)
        want = d - torch.log(torch.exp(d).sum(1, keepdim=True))
        p = torch.exp(want)
        for what, got, w in (("given tokens", lp[rows], want.gather(1, tokens[rows].long())),
                             ("chosen tokens", tl[rows], want.gather(1, ids[rows].long())),
                             ("entropy", en[rows], -torch.where(p > 0, p * want, 0.0).sum(1))):
            masked = torch.isinf(w)
            assert torch.equal(got[masked].double(), w[masked])
            err = (got.double() - w).abs()[~masked] / (1 + w[~masked].abs())
            assert err.numel() == 0 or err.max() <= BOUND, f"{what}: {(err.max() / BOUND).item()} of the bound"


def rows(m, v, scale, seed=0):
    g = torch.Generator(device=DEV).manual_seed(m + v + seed)
    return torch.randn(m, v, generator=g, device=DEV) * scale


@pytest.mark.parametrize("dtype", CODE, ids=str)
@pytest.mark.parametrize("m,v", [(3, 5), (3, 100), (2, 8193), (257, 8193), (1, 128256), (256, 32001)])
@pytest.mark.parametrize("scale", [0.1, 1.0, 3.0, 8.0])
def test_random_rows(qll_gpu, m, v, scale, dtype):
    assert_published_bound(rows(m, v, scale).to(dtype))


@pytest.mark.parametrize("dtype", CODE, ids=str)
@pytest.mark.parametrize("m", [1, 256])
@pytest.mark.parametrize("peak", [0.0, 13.8])
def test_flat_rows(qll_gpu, m, peak, dtype):
    """With the peak, half of the weight is one token's and half is spread over 2^20."""
    x = rows(m, 1 << 20 if m == 1 else 1 << 17, 0.05)
    x[:, 5] += peak
    assert_published_bound(x.to(dtype))


@pytest.mark.parametrize("dtype", CODE, ids=str)
@pytest.mark.parametrize("m", [1, 256])
@pytest.mark.parametrize("below", [15.99, 12.3, 3.3])
@pytest.mark.parametrize("noise", [0.0, 0.3])
def test_first_logits_below_the_rest(qll_gpu, m, below, noise, dtype):
    x = rows(m, 1 << 17, noise) + torch.arange(m, device=DEV)[:, None] * 0.37
    x[:, :8192 if m >= 256 else 2048] -= below
    assert_published_bound(x.to(dtype))


@pytest.mark.parametrize("creep", [1e-6, 1e-3])
def test_reference_that_moves_in_every_step(qll_gpu, creep):
    m, v, step = 256, 1 << 18, 4096  # steps of 512 threads' two pieces of four
    at = torch.arange(v, device=DEV)
    lane, st = at // 4 % 64, (at // step).float()
    x = torch.full((m, v), -5000.0, device=DEV)
    x[:, lane == 0] = (st * creep)[lane == 0] * (1 + torch.arange(m, device=DEV)[:, None] / 64)
    x[:, lane == 1] = (16.2 * st - 1200.0)[lane == 1]
    assert_published_bound(x)


@pytest.mark.parametrize("dtype", CODE, ids=str)
@pytest.mark.parametrize("m", [2, 256])
def test_rising_and_masked_rows(qll_gpu, m, dtype):
    v = 20000
    x = torch.linspace(-30, 30, v, device=DEV).repeat(m, 1) + torch.arange(m, device=DEV)[:, None] / 64
    x[1] = x[1].flip(0)
    assert_published_bound(x.to(dtype))
    x = rows(m, v, 3.0, 1)
    x[:, ::3] = -float("inf")
    x[0, 7:] = torch.finfo(dtype).min
    assert_published_bound(x.to(dtype))
