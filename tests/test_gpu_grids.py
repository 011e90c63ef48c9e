"""Calls whose work takes 2^32 threads and more: a grid of that size would wrap
around, so they go out in parts, loop, or are refused.  Inputs are zeros but for a
few rows around the borders of the parts; every output is written."""
import pytest
import torch

import quantized_linear_layer_amd as qll
from gpu_util import DEV, empty

pytestmark = pytest.mark.gpu

ONE = (0x00, 0x3c)  # binary16 1.0, little-endian


@pytest.fixture(autouse=True)
def memory_given_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def room(gib):
    free = torch.cuda.mem_get_info()[0]
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory, {free >> 30} are free")


def marks(n, *borders):
    at = sorted({r for b in (0, n, *borders) for r in (b - 1, b) if 0 <= r < n})
    return torch.tensor(at, device=DEV)


def q4_0_rows(n, rows):
    """One block a row: zeros, but in `rows` scale 1 and codes of -8 and 1 + index % 7."""
    w = torch.zeros(n * 18, dtype=torch.uint8, device=DEV).view(n, 18)
    code = 8 + 1 + torch.arange(len(rows), device=DEV) % 7
    w[rows, 2:] = (code << 4).to(torch.uint8)[:, None]  # elements 0..15: code 0 (-8), 16..31: `code`
    w[rows] = w[rows].index_copy(1, torch.tensor([0, 1], device=DEV),
                                 torch.tensor(ONE, dtype=torch.uint8, device=DEV).repeat(len(rows), 1))
    return w.view(-1), 16.0 * (code - 8 - 8).float()  # its product with a row of ones


def q8_0_ones(m):
    xq = torch.ones(m, 34, dtype=torch.uint8, device=DEV)
    xq[:, 0], xq[:, 1] = ONE
    return xq.view(-1)


def assert_only(y, rows, want):
    """y is `want` in rows and 0 everywhere else."""
    assert torch.equal(y[rows], want)
    assert int((y != 0).sum()) == int((want != 0).sum()), "other rows written, or rows left out"


def test_gated_and_linear_of_one_row(qll_gpu):
    room(40)
    n = (1 << 29) + 40
    rows = marks(n, 1 << 28, 1 << 29)
    w, want = q4_0_rows(n, rows)
    xq, y = q8_0_ones(1), torch.full((n,), float("nan"), device=DEV)
    qll.qll_q4_0_q8_0_gated(w, w, xq, qll.QLL_ACT_NONE, y, 1, n, 32)
    assert_only(y, rows, want * want)
    y.fill_(float("nan"))
    qll.qll_q4_0_q8_0_linear(w, xq, None, qll.QLL_ACT_RELU, None, y, 1, n, 32)
    assert_only(y, rows, want.clamp_min(0))
    y.fill_(float("nan"))
    qll.qll_q4_0_q8_0_gemv(w, xq, y, n, 32)
    assert_only(y, rows, want)


def test_two_rows(qll_gpu):
    room(60)
    n = (1 << 30) + 72
    rows = marks(n, 1 << 29, 1 << 30)
    w, want = q4_0_rows(n, rows)
    xq, y = q8_0_ones(2), torch.full((2, n), float("nan"), device=DEV)
    bias = torch.zeros(n, device=DEV)
    bias[rows] = 3.0
    qll.qll_q4_0_q8_0_linear(w, xq, bias, qll.QLL_ACT_NONE, None, y, 2, n, 32)
    for i in (0, 1):
        assert_only(y[i], rows, want + 3.0)
    y.fill_(float("nan"))
    qll.qll_q4_0_q8_0_gemm(w, xq, y, 2, n, 32)
    for i in (0, 1):
        assert_only(y[i], rows, want)


def test_repacked_pair(qll_gpu):
    room(200)
    n, k = (1 << 25) + 64, 2048
    nb, tiles = k // 32, n // 64
    w = torch.zeros(n * nb * 18, dtype=torch.uint8, device=DEV)
    some = [0, (1 << 18) - 1, 1 << 18, tiles // 2 - 1, tiles // 2, tiles - 2, tiles - 1]
    g = torch.Generator(device=DEV).manual_seed(1)
    for t in some:
        w[t * 64 * nb * 18:(t + 1) * 64 * nb * 18] = torch.randint(0, 256, (64 * nb * 18,), generator=g, device=DEV,
                                                                   dtype=torch.uint8)
    need = qll.qll_q4_0_repacked_gated_bytes(n, k)
    wp = torch.empty(need, dtype=torch.uint8, device=DEV)
    wp[-256 * nb:] = 0xA5
    qll.qll_q4_0_repack_gated(w, w, wp, n, k)
    chunk = nb * 128 * 24  # a tile's codes: 128 rows of 32 six-bit ones a block
    codes, scales = wp[:tiles * chunk].view(tiles, -1), wp[tiles * chunk:].view(tiles, -1)
    one = torch.empty(qll.qll_q4_0_repacked_gated_bytes(64, k), dtype=torch.uint8, device=DEV)
    for t in some:
        part = w[t * 64 * nb * 18:(t + 1) * 64 * nb * 18].clone()
        qll.qll_q4_0_repack_gated(part, part, one, 64, k)
        assert torch.equal(codes[t], one[:chunk]) and torch.equal(scales[t], one[chunk:]), t
    assert int(scales[1].max()) == 0 and int(scales[tiles - 3].max()) == 0


def test_quantize_i8_rows(qll_gpu):
    m, k = (1 << 24) + 5, 4
    x = torch.zeros(m, k, device=DEV)
    rows = marks(m, 1 << 23, 1 << 24)
    x[rows, 1] = -2.0
    q = torch.full((m, k), 7, dtype=torch.int8, device=DEV)
    s, t = torch.full((m,), -7.0, device=DEV), torch.full((m,), -7, dtype=torch.int32, device=DEV)
    qll.qll_quantize_i8_rows(x, q, s, t, m, k)
    assert_only(t, rows, torch.full((len(rows),), -127, dtype=torch.int32, device=DEV))
    assert_only(s, rows, torch.full((len(rows),), 63.5, device=DEV))
    assert_only(q[:, 1], rows, torch.full((len(rows),), -127, dtype=torch.int8, device=DEV))
    assert int((q != 0).sum()) == len(rows)


def test_quantize_q8_0(qll_gpu):
    room(120)
    m = (1 << 29) + 3
    x = torch.zeros(m, 32, device=DEV)
    rows = marks(m, 1 << 28, 1 << 29)
    x[rows, 31] = 127.0
    xq = torch.full((m, 34), 7, dtype=torch.uint8, device=DEV)
    qll.qll_quantize_q8_0(x, xq, m, 32)
    del x
    assert torch.equal(xq[rows, 33], torch.full((len(rows),), 127, dtype=torch.uint8, device=DEV))
    for c in range(34):
        written = {1: ONE[1], 33: 127}.get(c, 0)
        assert int((xq[:, c] != 0).sum()) == (len(rows) if written else 0)
        assert torch.equal(xq[rows, c], torch.full((len(rows),), written, dtype=torch.uint8, device=DEV))


def test_ternary_gemv(qll_gpu):
    n, k = (1 << 29) + 40, 64
    w = torch.full((n, 4), 0x55555555, dtype=torch.int32, device=DEV)  # every code 0
    rows = marks(n, 1 << 28, 1 << 29)
    w[rows] = -0x55555556  # 0xaaaaaaaa: every code +1
    xq = torch.full((k,), 2, dtype=torch.int8, device=DEV)
    s, t = torch.ones(1, device=DEV), torch.full((1,), 2 * k, dtype=torch.int32, device=DEV)
    y = torch.full((n,), float("nan"), device=DEV)
    qll.qll_ternary_gemv(w, 0.5, xq, s, t, y, n, k)
    assert_only(y, rows, torch.full((len(rows),), float(k), device=DEV))


@pytest.mark.parametrize("n,k,border", [((1 << 26) + 40, 5, 1 << 25), ((1 << 29) + 40, 4, 1 << 28)])
def test_gemv_nt(qll_gpu, n, k, border):
    w = torch.zeros(n, k, device=DEV)
    rows = marks(n, border, 2 * border)
    w[rows] = 1.5
    y = torch.full((n,), float("nan"), device=DEV)
    qll.qll_gemm_nt(torch.ones(k, device=DEV), w, qll.QLL_DTYPE_F32, y, 1, n, k)
    assert_only(y, rows, torch.full((len(rows),), 1.5 * k, device=DEV))


def test_ternary_gemm_is_refused(qll_gpu):
    n, k, m = 1 << 29, 16, 2
    w = torch.full((n,), 0x55555555, dtype=torch.int32, device=DEV)
    xq, s = torch.ones(m, k, dtype=torch.int8, device=DEV), torch.ones(m, device=DEV)
    t, y = torch.full((m,), k, dtype=torch.int32, device=DEV), torch.zeros(m, n, device=DEV)
    with pytest.raises(qll.QllError):
        qll.qll_ternary_gemm(w, 0.5, xq, s, t, y, m, n, k)
