"""qll_token_logprobs against its 64-bit form (logprob_refs): log probabilities
and entropies within derived bounds, the chosen tokens equal."""
import numpy as np
import pytest
import torch

import logprob_refs as R
import quantized_linear_layer_amd as qll
from gpu_util import empty

pytestmark = pytest.mark.gpu

CODE = {torch.float32: qll.QLL_DTYPE_F32, torch.bfloat16: qll.QLL_DTYPE_BF16, torch.float16: qll.QLL_DTYPE_F16}
DTYPES = list(CODE)
GUARD = 32


def call(x, tokens, top, entropy=True, stream=None):
    m, v = x.shape
    t = tokens.shape[1]
    xd = x.cuda()
    lp = torch.full((m * t + GUARD,), 9.0, device="cuda")
    en = torch.full((m + GUARD,), 9.0, device="cuda")
    ids = torch.full((m * top + GUARD,), -9, dtype=torch.int32, device="cuda")
    tl = torch.full((m * top + GUARD,), 9.0, device="cuda")
    ws = empty(qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, m, v, top))
    ws.fill_(0xff)  # nothing in it is relied on: NaN everywhere
    qll.qll_token_logprobs(xd, CODE[x.dtype], torch.from_numpy(tokens.astype(np.int32)).cuda() if t else None, t,
                           lp if t else None, en if entropy else None, top, ids if top else None,
                           tl if top else None, m, v, ws=ws, stream=stream)
    torch.cuda.synchronize()
    lp, en, ids, tl = (a.cpu().numpy() for a in (lp, en, ids, tl))
    assert (lp[m * t:] == 9).all() and (en[m if entropy else 0:] == 9).all()
    assert (ids[m * top:] == -9).all() and (tl[m * top:] == 9).all()
    return lp[:m * t].reshape(m, t), en[:m], ids[:m * top].reshape(m, top), tl[:m * top].reshape(m, top)


def check(x, tokens, top, **kw):
    got = call(x, tokens, top, **kw)
    want = R.reference(x.float().numpy(), tokens, top)
    assert np.array_equal(got[2], want[2]), "other tokens chosen"
    R.assert_close(got[0], want[0], want[4], "given tokens")
    R.assert_close(got[3], want[3], want[4], "chosen tokens")
    if kw.get("entropy", True):
        R.assert_close(got[1], want[1], want[5], "entropy")


def logits(seed, m, v, dtype, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, v, generator=g) * scale).to(dtype), torch.randint(0, v, (m, 3), generator=g).numpy()


# one logit to a whole vocabulary, around the chunk sizes (2048 and 8192), with
# few rows (short chunks) and many (long ones)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,v,top", [(1, 1, 1), (2, 2, 2), (5, 3, 1), (3, 63, 5), (1, 64, 64), (4, 65, 64),
                                     (2, 255, 20), (300, 1000, 20), (1, 2047, 64), (3, 2048, 5), (2, 2049, 20),
                                     (260, 2049, 7), (1, 8191, 20), (2, 8193, 33), (257, 8193, 20), (1, 32001, 20),
                                     (40, 50257, 5), (1, 128256, 64)])
def test_sizes(qll_gpu, m, v, top, dtype):
    x, tokens = logits(m + v, m, v, dtype)
    check(x, tokens, top)


def test_largest_vocabulary(qll_gpu):
    x, tokens = logits(1, 1, 1 << 20, torch.float32)
    check(x, tokens, 64)   # too many short lists to join: long chunks
    check(x, tokens, 8)


@pytest.mark.parametrize("top,t,entropy", [(0, 3, True), (5, 0, True), (0, 0, True), (4, 1, False), (0, 1, False)])
def test_parts_left_out(qll_gpu, top, t, entropy):
    x, tokens = logits(2, 3, 5000, torch.bfloat16)
    check(x, tokens[:, :t], top, entropy=entropy)


def test_many_given_tokens_and_padding(qll_gpu):
    x, _ = logits(3, 4, 777, torch.float32)
    tokens = np.random.default_rng(0).integers(0, 777, (4, 1000))
    tokens[1, 5], tokens[2, 6], tokens[3, 7], tokens[0, 0] = -1, 777, 2 ** 31 - 1, -2 ** 31
    tokens[0, 1:4] = 5  # the same index several times
    check(x, tokens, 3)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("v", [70, 9000])
@pytest.mark.parametrize("m", [6, 262])
def test_masked_rows(qll_gpu, m, v, dtype):
    x, tokens = logits(m + v, m, v, dtype)
    inf = float("inf")
    x[0] = -inf                    # nothing left
    x[1] = -inf
    x[1, v - 1] = 1.5              # one token left: log p = 0, entropy 0
    x[2, :v - 7] = -inf            # fewer left than are asked for
    x[3, ::2] = -inf
    x[4, 5:] = torch.finfo(dtype).min  # masked by the type's lowest value
    check(x, tokens, 20)


@pytest.mark.parametrize("v", [70, 9000])
def test_nan_and_inf_rows(qll_gpu, v):
    x, tokens = logits(v, 5, v, torch.float32)
    x[1, v // 2] = float("nan")
    x[2, 3] = float("inf")
    x[3] = float("nan")
    lp, en, ids, tl = call(x, tokens, 20)
    for r in (1, 2, 3):
        assert np.isnan(lp[r]).all() and np.isnan(en[r]) and np.isnan(tl[r]).all()
        assert ((ids[r] >= 0) & (ids[r] < v)).all()
    want = R.reference(x[[0, 4]].numpy(), tokens[[0, 4]], 20)
    assert np.array_equal(ids[[0, 4]], want[2])
    R.assert_close(lp[[0, 4]], want[0], want[4], "rows beside them")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,v", [(1, 9001), (264, 9001)])
def test_ties(qll_gpu, m, v, dtype):
    g = torch.Generator().manual_seed(4)
    x = torch.zeros(m, v)
    x[0] = 2.5                                                    # every logit equal
    if m > 1:
        x[1:100] = torch.randint(0, 3, (99, v), generator=g).float()  # three values
        x[100:200] = torch.randint(-1, 1, (100, v), generator=g).float() * 0.0  # zeros of both signs
        x[200:] = (torch.randn(64, v, generator=g) * 4).round()
    check(x.to(dtype), np.zeros((m, 1), int), 64)


@pytest.mark.parametrize("top", [20, 64])
@pytest.mark.parametrize("m", [1, 260])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=str)
def test_good_logits_crowded_on_few_lanes(qll_gpu, m, top, dtype):
    """More elements pass the bound than are ranked by counting."""
    v = 16384
    per = 4 if dtype == torch.float32 else 8  # logits of one lane that lie together
    x, tokens = logits(5, m, v, dtype, 1.0)
    lane = (torch.arange(v) // per) % 64
    x[:, lane < top - 1] += 50.0
    check(x, tokens, top)


def test_sorted_rows(qll_gpu):
    v = 20000
    up = torch.linspace(-20, 20, v).repeat(3, 1)
    up[1] = up[1].flip(0)
    up[2] = -1e30
    up[2, 77] = 1e30  # all the weight on one token
    check(up, np.array([[0], [5], [77]]), 20)


def test_another_stream_and_determinism(qll_gpu):
    x, tokens = logits(8, 3, 50257, torch.bfloat16)
    first = call(x, tokens, 20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = call(x, tokens, 20)
    third = call(x, tokens, 20, stream=s)
    for a, b, c in zip(first, second, third):
        assert np.array_equal(a, b) and np.array_equal(a, c)


def test_row_does_not_depend_on_its_batch_in_what_it_chooses(qll_gpu):
    x, tokens = logits(9, 300, 9000, torch.float16)
    many, one = call(x, tokens, 64), call(x[7:8].clone(), tokens[7:8], 64)
    assert np.array_equal(many[2][7], one[2][0])


@pytest.mark.parametrize("count", [65, 127, 128, 129])
@pytest.mark.parametrize("m", [200, 256])  # in segments of a row, and whole rows
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_full_list_then_only_better_logits(qll_gpu, dtype, m, count):
    """`count` entries in a wave's list (it holds 192), then a step whose every
    logit is better than all of them, worst first: a search for a bound that
    took the first 64 of the step again and again would not end."""
    v, piece = 16384, 16 // torch.empty(0, dtype=dtype).element_size()
    threads = 256 if m < 256 else 512
    pieces = 8 // piece if m < 256 else 2
    step = threads * pieces * piece
    g = torch.Generator().manual_seed(11)
    x = torch.randn(m, v, generator=g) * 0.1 - 8
    own = (torch.arange(v) // piece) % threads < 64  # the first wave's logits
    first = torch.nonzero(own[:step])[:, 0]
    x[:, first] = -40.0
    # (a lane's logits of a step lie piece by piece: all of the first lanes')
    lane = (first // piece) % threads
    few = first[torch.argsort(lane, stable=True)][:count]
    x[:, few] = -2.0 + 0.01 * torch.rand(m, count, generator=g)
    second = step + first
    place = (first // (piece * threads)) * piece + first % piece
    x[:, second] = 4.0 + (place * 64 + lane).float() / 256
    check(x.to(dtype), np.full((m, 1), 7), 64)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m", [2, 256])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_rising_rows(qll_gpu, dtype, m, top):
    v = 20000
    x = torch.linspace(-30, 30, v).repeat(m, 1) + torch.arange(m)[:, None] / 64
    x[1] = x[1].flip(0)
    check(x.to(dtype), np.full((m, 1), 3), top)


@pytest.mark.parametrize("v", [3, 8])  # a thread per row, and a workgroup per row
def test_more_rows_than_one_grid_holds(qll_gpu, v):
    """Workgroups of 512 threads for 2^23 + 3 rows: 2^32 threads and more."""
    m = (1 << 23) + 3
    x = torch.zeros(m, v, dtype=torch.bfloat16, device="cuda")
    x[1 << 22, 1], x[m - 1, 2] = 2.0, 1.0
    tokens = torch.zeros(m, dtype=torch.int32, device="cuda")
    tokens[m - 1] = 2
    lp, en = torch.full((m + 8,), 9.0, device="cuda"), torch.full((m + 8,), 9.0, device="cuda")
    ids = torch.full((m + 8,), -9, dtype=torch.int32, device="cuda")
    tl = torch.full((m + 8,), 9.0, device="cuda")
    ws = empty(qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, m, v, 1))
    qll.qll_token_logprobs(x, qll.QLL_DTYPE_BF16, tokens, 1, lp, en, 1, ids, tl, m, v, ws=ws)
    torch.cuda.synchronize()
    rows = [0, (1 << 22) - 1, 1 << 22, m - 2, m - 1]
    want = R.reference(x[rows].float().cpu().numpy(), tokens[rows].cpu().numpy()[:, None], 1)
    R.assert_close(lp[rows].cpu().numpy()[:, None], want[0], want[4], "given tokens")
    R.assert_close(en[rows].cpu().numpy(), want[1], want[5], "entropy")
    R.assert_close(tl[rows].cpu().numpy()[:, None], want[3], want[4], "chosen tokens")
    assert np.array_equal(ids[rows].cpu().numpy()[:, None], want[2])
    even = torch.ones(m, dtype=torch.bool, device="cuda")
    even[[1 << 22, m - 1]] = False
    assert (lp[:m][even] == lp[0]).all() and (en[:m][even] == en[0]).all() and (ids[:m][even] == 0).all()
    assert (lp[m:] == 9).all() and (en[m:] == 9).all() and (ids[m:] == -9).all() and (tl[m:] == 9).all()


def test_offsets_past_32_bits(qll_gpu):
    m, v = 4099, 1 << 20
    x = torch.zeros(m, v, dtype=torch.float16, device="cuda")
    tail, tokens = logits(15, 3, v, torch.float16)
    x[-3:] = tail.cuda()
    given = torch.zeros(m, 3, dtype=torch.int32, device="cuda")
    given[-3:] = torch.from_numpy(tokens.astype(np.int32)).cuda()
    lp, en = torch.empty(m * 3, device="cuda"), torch.empty(m, device="cuda")
    ids, tl = torch.empty(m * 5, dtype=torch.int32, device="cuda"), torch.empty(m * 5, device="cuda")
    ws = empty(qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, m, v, 5))
    qll.qll_token_logprobs(x, qll.QLL_DTYPE_F16, given, 3, lp, en, 5, ids, tl, m, v, ws=ws)
    torch.cuda.synchronize()
    want = R.reference(tail.float().numpy(), tokens, 5)
    R.assert_close(lp[-9:].cpu().numpy().reshape(3, 3), want[0], want[4], "given tokens")
    R.assert_close(en[-3:].cpu().numpy(), want[1], want[5], "entropy")
    assert np.array_equal(ids[-15:].cpu().numpy().reshape(3, 5), want[2])
    R.assert_close(tl[-15:].cpu().numpy().reshape(3, 5), want[3], want[4], "chosen tokens")


@pytest.mark.parametrize("m,v,top", [(1, 128256, 20), (1, 128256, 33), (3, 200000, 64), (1, 262144, 7), (40, 50257, 64),
                                     (200, 9000, 64), (1, 5000, 64), (1, 300000, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_joined_lists(qll_gpu, dtype, m, v, top):
    """Few to many segments and alternatives; the best in one segment, spread over
    all, and tied."""
    x, tokens = logits(m * v, m, v, dtype)
    x[0] = torch.linspace(-9, 9, v).to(dtype)
    check(x, tokens, top)
    x[:, :100] += 40.0
    x[0] = 1.0
    check(x, tokens, top)


@pytest.mark.parametrize("left", [1, 20, 64, 65, 300])
@pytest.mark.parametrize("m", [1, 256])
def test_few_logits_left_by_a_mask(qll_gpu, m, left):
    v = 30000
    x, tokens = logits(left, m, v, torch.float32)
    keep = torch.zeros(v, dtype=torch.bool)
    keep[torch.randperm(v, generator=torch.Generator().manual_seed(left))[:left]] = True
    x[:, ~keep] = -float("inf")
    check(x, tokens, 64)
