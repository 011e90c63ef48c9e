"""qll_rmsnorm_q8_0 and qll_rmsnorm_i8_rows against their definition in 64
bits: h bit for bit, every code and code sum equal, every scale equal.

Why equality.  A code is round-half-away(127 p / A) with p and A exact in f64
(products of two 24-bit significands), so the kernel and numpy evaluate the
same correctly rounded f64 quotient.  A scale is an f64 value (relative error
a few 1e-16 on either side) rounded to f32: the two differ only where that
value lies within 1e-15 of an f32 rounding border, about one block in 10^8."""
import numpy as np
import pytest
import torch

import quantized_linear_layer_amd as qll
from gpu_util import DEV

pytestmark = pytest.mark.gpu

CODE = {torch.float32: qll.QLL_DTYPE_F32, torch.bfloat16: qll.QLL_DTYPE_BF16, torch.float16: qll.QLL_DTYPE_F16}
DTYPES = list(CODE)


def definition(x, res, w, eps, q8):
    """(h, codes, scale, sum) in numpy from CPU tensors: scale is binary16 d
    per block, or act_scale per row."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hd = h.double().numpy()
    m, k = hd.shape
    p = hd * w.double().numpy()
    rms = np.sqrt((hd * hd).sum(1, keepdims=True) / k + np.float64(np.float32(eps)))
    g = p.reshape(m, -1, 32) if q8 else p.reshape(m, 1, k)
    a = np.abs(g).max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        t = np.where(a > 0, 127.0 * np.abs(g) / a, 0.0)
        codes = np.copysign(np.floor(t + 0.5), g).astype(np.int64)
        if q8:
            d = np.where(a[..., 0] > 0, a[..., 0] / (127.0 * rms), 0.0).astype(np.float32).astype(np.float16)
            return h, codes.reshape(m, k), d, None
        s = np.where(a[:, 0] > 0, 127.0 * rms / a[:, 0], 0.0).astype(np.float32)
    s = np.where(np.isfinite(s), s, np.float32(0))
    codes = np.where(s > 0, codes.reshape(m, k), 0)
    return h, codes, s[:, 0], codes.sum(1)


def call(form, x, res, w, eps, h, stream=None, guard=0):
    """The library's outputs for CPU tensors x, res, w; h: None, "new", "x" or
    "res" (in place).  Returns (h, codes, scale, sum) as numpy."""
    m, k = x.shape
    xd, wd = x.to(DEV), w.to(DEV)
    rd = None if res is None else res.to(DEV)
    hd = {None: None, "new": torch.empty_like(xd), "x": xd, "res": rd}[h]
    code = CODE[x.dtype]
    if form == "q8_0":
        xq = torch.full((m * (k // 32) * 34 + guard,), 0xA5, dtype=torch.uint8, device=DEV)
        qll.qll_rmsnorm_q8_0(xd, code, rd, wd, eps, hd, xq, m, k, stream=stream)
        torch.cuda.synchronize()
        raw = xq.cpu().numpy()
        assert (raw[m * (k // 32) * 34:] == 0xA5).all(), "bytes behind the last block changed"
        b = raw[:m * (k // 32) * 34].reshape(m, k // 32, 34)
        scale = b[..., :2].copy().view(np.float16)[..., 0]
        codes, total = b[..., 2:].copy().view(np.int8).reshape(m, k).astype(np.int64), None
    else:
        xq = torch.full((m * k + guard,), 0x5A, dtype=torch.int8, device=DEV)
        s = torch.full((m + guard,), -7.0, device=DEV)
        t = torch.full((m + guard,), -7, dtype=torch.int32, device=DEV)
        qll.qll_rmsnorm_i8_rows(xd, code, rd, wd, eps, hd, xq, s, t, m, k, stream=stream)
        torch.cuda.synchronize()
        raw, s, t = xq.cpu().numpy(), s.cpu().numpy(), t.cpu().numpy()
        assert (raw[m * k:] == 0x5A).all() and (s[m:] == -7).all() and (t[m:] == -7).all(), "wrote past the rows"
        scale, total, codes = s[:m], t[:m], raw[:m * k].reshape(m, k).astype(np.int64)
    if res is not None and h != "res":
        assert torch.equal(rd.cpu().view(torch.uint8), res.view(torch.uint8))
    if h != "x":
        assert torch.equal(xd.cpu().view(torch.uint8), x.view(torch.uint8))
    return None if hd is None else hd.cpu(), codes, scale, total


def check(form, x, res, w, eps=1e-5, h="new", **kw):
    want = definition(x, res, w, eps, form == "q8_0")
    got = call(form, x, res, w, eps, h, **kw)
    if h is not None:
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)), "the sum differs"
    bad = np.argwhere(got[1] != want[1])
    assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0].tolist()}"
    assert np.array_equal(got[2], want[2]), "scales differ"
    if want[3] is not None:
        assert np.array_equal(got[3], want[3]), "code sums differ"


def stream_rows(seed, m, k, dtype):
    g = torch.Generator().manual_seed(seed)
    spread = torch.ones(k)
    spread[torch.randint(0, k, (1 + k // 200,), generator=g)] = 30.0  # a few channels large in every row
    return ((torch.randn(m, k, generator=g) * spread).to(dtype), (torch.randn(m, k, generator=g) * spread).to(dtype),
            0.5 + torch.rand(k, generator=g))


# every launch shape: a wave per row (one or four pieces), 256 and 1024
# threads, held rows and two sweeps, with rows that fill none of them evenly
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,k", [(1, 32), (5, 64), (3, 256), (7, 288), (2, 1024), (1, 1056), (4, 4096), (257, 1056),
                                 (300, 4096), (2, 4128), (1, 8192), (3, 14336), (1, 16384), (2, 16416), (1, 65536)])
def test_q8_0(qll_gpu, m, k, dtype):
    x, r, w = stream_rows(m * 7 + k, m, k, dtype)
    check("q8_0", x, r, w, guard=64)
    check("q8_0", x, None, w, h=None)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,k", [(1, 1), (3, 2), (2, 5), (9, 64), (5, 63), (2, 257), (6, 260), (3, 1000), (1, 1025),
                                 (2, 2560), (260, 2560), (270, 1001), (2, 4097), (4, 6912), (1, 16383), (1, 16388),
                                 (2, 16387), (1, 40001)])
def test_i8_rows(qll_gpu, m, k, dtype):
    x, r, w = stream_rows(m * 11 + k, m, k, dtype)
    check("i8", x, r, w, guard=64)
    check("i8", x, None, w, h=None)


@pytest.mark.parametrize("form", ["q8_0", "i8"])
@pytest.mark.parametrize("k", [96, 4096, 16416])
@pytest.mark.parametrize("h", [None, "x", "res"])
def test_sum_in_place_or_not_kept(qll_gpu, form, k, h):
    x, r, w = stream_rows(5, 3, k, torch.float32)
    check(form, x, r, w, h=h)


@pytest.mark.parametrize("form", ["q8_0", "i8"])
def test_copy_of_the_stream(qll_gpu, form):
    x, _, w = stream_rows(6, 2, 160, torch.bfloat16)
    check(form, x, None, w, h="new")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("form", ["q8_0", "i8"])
def test_values_on_code_borders(qll_gpu, form, dtype):
    """127 p / A = j + 1/2 exactly: A a multiple of 127, p of A / 254; and one
    unit in the last place to either side."""
    k = 96
    t = 5 if dtype == torch.float16 else 3 if dtype == torch.float32 else 1
    top = 127.0 * t
    v = torch.zeros(6, k)
    for row in range(6):
        odd = 2 * torch.randint(0, 127 if t == 1 else 120, (k,), generator=torch.Generator().manual_seed(row)) + 1
        v[row] = odd * (t / 2) * (1 if row % 2 else -1)
        v[row, ::32] = top
    x = v.to(dtype)
    if dtype != torch.bfloat16:
        assert torch.equal(x.float(), v)  # the borders themselves are representable
    x[2:4] = torch.nextafter(x[2:4].float(), torch.zeros(2, k)).to(dtype) if dtype == torch.float32 else x[2:4]
    x[4:6] = torch.nextafter(x[4:6].float(), torch.full((2, k), 1e9)).to(dtype) if dtype == torch.float32 else x[4:6]
    x[:, ::32] = top
    check(form, x, None, torch.ones(k), h=None)
    check(form, x, None, torch.full((k,), 0.25), h=None)


@pytest.mark.parametrize("k", [64, 4096, 16416])
@pytest.mark.parametrize("form", ["q8_0", "i8"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_zero_rows_blocks_and_weights(qll_gpu, form, eps, k):
    x, r, w = stream_rows(3, 5, k, torch.float32)
    x[1] = 0.0
    r[1] = 0.0          # a padded row: no value at all
    x[2], r[2] = 1.5, -1.5  # a sum that cancels
    x[3, 32:64] = 0.0
    r[3, 32:64] = 0.0   # one empty block
    w[:32] = 0.0        # weights that empty a block of every row
    check(form, x, r, w, eps=eps)


def test_scales_at_the_ends_of_their_range(qll_gpu):
    k = 128
    w = torch.ones(k)
    x = torch.zeros(5, k)
    x[0, 7] = 1e-45      # a row whose act_scale overflows: all zero
    x[1, 7] = 1e-38      # a finite one, near the top
    x[2] = 3e37          # squares far past f32's range
    x[3, :] = 1e-30      # squares far below it
    x[4, 5] = -3e38
    check("i8", x, None, w)
    check("q8_0", x, None, w)
    check("i8", x, None, w, eps=0.0)


def test_another_stream_and_repeated_calls_agree(qll_gpu):
    x, r, w = stream_rows(9, 64, 2560, torch.float16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check("i8", x, r, w)
        check("q8_0", x, r, w)
    check("i8", x, r, w, stream=s)
    a, b = call("q8_0", x, r, w, 1e-5, "new"), call("q8_0", x, r, w, 1e-5, "new")
    assert np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2])


def test_codes_of_a_row_do_not_depend_on_its_batch(qll_gpu):
    # 256-thread and 1024-thread launches of the same row
    x, r, w = stream_rows(10, 300, 4096, torch.float32)
    many = call("q8_0", x, r, w, 1e-5, "new")
    one = call("q8_0", x[17:18].clone(), r[17:18].clone(), w, 1e-5, "new")
    assert np.array_equal(many[1][17], one[1][0]) and np.array_equal(many[2][17], one[2][0])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("form", ["q8_0", "i8"])
@pytest.mark.parametrize("m,k", [(7, 96), (7, 4096), (260, 4096), (7, 16416)])
def test_rows_with_nan_or_infinity(qll_gpu, form, m, k, dtype):
    x, r, w = stream_rows(12, m, k, dtype)
    bad = [1, 2, 4, 5]
    x[1, 40] = float("nan")
    r[2] = float("nan")
    x[4, 3] = float("inf")
    x[5, 7] = r[5, 7] = torch.finfo(dtype).max  # a sum that overflows
    got = call(form, x, r, w, 1e-5, "new")
    h, codes, scale, total = definition(x, r, w, 1e-5, form == "q8_0")
    good = [i for i in range(m) if i not in bad]
    assert np.array_equal(got[1][good], codes[good]) and np.array_equal(got[2][good], scale[good])
    same = (got[0] == h) | (torch.isnan(got[0]) & torch.isnan(h))
    assert same.all()
    if form == "q8_0":
        assert np.isnan(got[2][bad]).all()
    else:
        assert np.array_equal(got[3][good], total[good])
        assert (got[1][bad] == 0).all() and (got[2][bad] == 0).all() and (got[3][bad] == 0).all()


@pytest.mark.parametrize("form", ["q8_0", "i8"])
@pytest.mark.parametrize("h", ["new", "x"])
@pytest.mark.parametrize("k", [64, 4096, 16416])
def test_stream_added_to_itself(qll_gpu, form, h, k):
    x, _, w = stream_rows(13, 3, k, torch.bfloat16)
    xd, wd = x.to(DEV), w.to(DEV)
    hd = xd if h == "x" else torch.empty_like(xd)
    want = definition(x, x, w, 1e-5, form == "q8_0")
    if form == "q8_0":
        xq = torch.empty(3 * (k // 32) * 34, dtype=torch.uint8, device=DEV)
        qll.qll_rmsnorm_q8_0(xd, qll.QLL_DTYPE_BF16, xd, wd, 1e-5, hd, xq, 3, k)
        codes = xq.cpu().numpy().reshape(3, k // 32, 34)[..., 2:].copy().view(np.int8).reshape(3, k)
    else:
        xq = torch.empty(3 * k, dtype=torch.int8, device=DEV)
        s, t = torch.empty(3, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
        qll.qll_rmsnorm_i8_rows(xd, qll.QLL_DTYPE_BF16, xd, wd, 1e-5, hd, xq, s, t, 3, k)
        codes = xq.cpu().numpy().reshape(3, k)
        assert np.array_equal(s.cpu().numpy(), want[2]) and np.array_equal(t.cpu().numpy(), want[3])
    assert torch.equal(hd.cpu(), want[0]) and np.array_equal(codes, want[1])


def test_more_rows_than_one_grid_holds(qll_gpu):
    """2^26 + 3 rows of one wave each: 2^32 threads and more."""
    m, k = (1 << 26) + 3, 1
    x = torch.zeros(m, k, dtype=torch.float16, device=DEV)
    x[0], x[(1 << 21) - 1], x[1 << 21], x[m - 1] = 1.0, -2.0, 3.0, -4.0
    w = torch.full((k,), 0.5, device=DEV)
    xq = torch.full((m + 4,), 7, dtype=torch.int8, device=DEV)
    s, t = torch.full((m + 4,), -7.0, device=DEV), torch.full((m + 4,), -7, dtype=torch.int32, device=DEV)
    qll.qll_rmsnorm_i8_rows(x, qll.QLL_DTYPE_F16, None, w, 0.0, None, xq, s, t, m, k)
    torch.cuda.synchronize()
    at = torch.tensor([0, (1 << 21) - 1, 1 << 21, m - 1], device=DEV)
    want = torch.tensor([127, -127, 127, -127], device=DEV)
    assert torch.equal(xq[at].int(), want.int()) and torch.equal(t[at], want.int())
    assert torch.equal(s[at], torch.full((4,), 254.0, device=DEV))
    assert int((xq[:m] != 0).sum()) == 4 and int((t[:m] != 0).sum()) == 4 and int((s[:m] != 0).sum()) == 4
    assert (xq[m:] == 7).all() and (s[m:] == -7).all() and (t[m:] == -7).all()


@pytest.mark.parametrize("form", ["q8_0", "i8"])
def test_offsets_past_32_bits(qll_gpu, form):
    m, k = (1 << 20) + 5, 4096
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    tail, _, w = stream_rows(14, 5, k, torch.bfloat16)
    x[-5:] = tail.to(DEV)
    xt, wd = x[-5:].cpu(), w.to(DEV)
    want = definition(xt, None, w, 1e-5, form == "q8_0")
    if form == "q8_0":
        xq = torch.empty(m * (k // 32) * 34, dtype=torch.uint8, device=DEV)
        qll.qll_rmsnorm_q8_0(x, qll.QLL_DTYPE_BF16, None, wd, 1e-5, x, xq, m, k)
        codes = xq[-5 * (k // 32) * 34:].cpu().numpy().reshape(5, k // 32, 34)[..., 2:].copy().view(np.int8)
    else:
        xq = torch.empty(m * k, dtype=torch.int8, device=DEV)
        s, t = torch.empty(m, device=DEV), torch.empty(m, dtype=torch.int32, device=DEV)
        qll.qll_rmsnorm_i8_rows(x, qll.QLL_DTYPE_BF16, None, wd, 1e-5, x, xq, s, t, m, k)
        codes = xq[-5 * k:].cpu().numpy()
        assert np.array_equal(s[-5:].cpu().numpy(), want[2]) and np.array_equal(t[-5:].cpu().numpy(), want[3])
    assert np.array_equal(codes.reshape(5, k), want[1]) and torch.equal(x[-5:].cpu(), xt)
