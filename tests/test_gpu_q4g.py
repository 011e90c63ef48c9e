"""4-bit weights with group scales: packing and qll_q4g_linear against 64 bits,
on every kernel it dispatches to, with derived bounds (q4g_refs).  Outputs are
written into a buffer with guard values behind them."""
import numpy as np
import pytest
import torch

import epilogue_refs as E
import q4g_refs as R
import quantized_linear_layer_amd as qll
import synth
from gpu_util import dev, empty, pack_q4_0

pytestmark = pytest.mark.gpu
GUARD = 64
FMTS = [0, qll.QLL_Q4G_BF16, qll.QLL_Q4G_ZEROS, qll.QLL_Q4G_BF16 | qll.QLL_Q4G_ZEROS]


def draw_x(rng, m, k, dtype):
    """Activations with a few large channels, on the device, and their values."""
    x = rng.standard_normal((m, k))
    x[:, rng.integers(0, k, 1 + k // 256)] *= 30.0
    t = torch.from_numpy(x).to(R.TYPES[dtype]).cuda()
    return t, R.f64(t)


def call(w, x, dtype, bias, act, residual, y_dtype, in_place=False, stream=None):
    m, n = x.shape[0], w.n
    y = torch.full((m * n + GUARD,), 3.25, dtype=R.TYPES[y_dtype], device="cuda")
    if in_place:
        y[:m * n] = residual.reshape(-1)
        residual = y
    ws = workspace(m, n, w.k)
    qll.qll_q4g_linear(w.wp, w.group, w.fmt, x, R.CODES[dtype], bias, E.ACTS[act], residual, y, R.CODES[y_dtype], m, n,
                       w.k, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert (y[m * n:] == 3.25).all(), "wrote past the outputs"
    return y[:m * n].view(m, n)


def workspace(m, n, k):
    need = qll.qll_workspace_bytes(qll.QLL_OP_Q4G_LINEAR, m, n, k)
    return torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None


# (m, n, k / group): one row to more than a group of 64, row tiles cut short, k from one
# group to many, ends inside a tile of 128 and a chunk of 512
SHAPES = [(1, 1, 1), (1, 16, 2), (1, 515, 9), (2, 33, 5), (4, 100, 16), (5, 47, 3), (8, 64, 17), (16, 130, 12),
          (17, 31, 4), (33, 200, 7), (64, 96, 13), (65, 40, 6), (130, 129, 11), (260, 72, 10)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,groups", SHAPES)
def test_products(qll_gpu, m, n, groups, dtype, group):
    rng = np.random.default_rng(m * 1000 + n + group)
    fmt = FMTS[(m + n + groups) % 4]
    w = R.Weights(rng, n, groups * group, group, fmt)
    x, xv = draw_x(rng, m, w.k, dtype)
    for y_dtype in {dtype, "f32"}:
        y = call(w, x, dtype, None, "none", None, y_dtype)
        E.assert_bound(R.f64(y), *R.linear(w, xv, None, "none", None, y_dtype), f"{dtype} -> {y_dtype} fmt {fmt}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_every_weight_alone(qll_gpu, dtype, group, fmt):
    """One activation of one at a time: the weights themselves, exactly (a
    difference of small integers times a 16-bit scale)."""
    rng = np.random.default_rng(group + fmt)
    n, k = 37, 5 * 128
    w = R.Weights(rng, n, k, group, fmt)
    s, z, c = w.values()
    want = (s * (c - z)).T
    x = torch.eye(k, dtype=R.TYPES[dtype], device="cuda")
    for at in range(0, k, 64):
        y = call(w, x[at:at + 64], dtype, None, "none", None, "f32")
        assert np.array_equal(R.f64(y), want[at:at + 64])
    for at in (0, 31, 32, 100, 127, 128, 511, 512, 639):  # one row, and a few: other kernels
        assert np.array_equal(R.f64(call(w, x[at:at + 1], dtype, None, "none", None, "f32")), want[at:at + 1])
    assert np.array_equal(R.f64(call(w, x[500:516], dtype, None, "none", None, "f32")), want[500:516])


@pytest.mark.parametrize("n,k", [(1, 32), (40, 96), (16, 512), (100, 1440)])
def test_q4_0_weights(qll_gpu, n, k):
    """The packed form of Q4_0 blocks is that of their codes and scales."""
    rng = np.random.default_rng(n + k)
    codes, d_bits = synth.q4_0_weights(rng, n, k)
    size = qll.qll_q4g_packed_bytes(n, k, 32, 0)
    a, b = (torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    qll.qll_q4g_from_q4_0(pack_q4_0(codes, d_bits), a, n, k)
    qll.qll_q4g_pack(dev(codes), dev(np.asarray(d_bits, np.uint16).view(np.int16)), None, 32, 0, b, n, k)
    assert torch.equal(a, b) and (a[size:] == 0xA5).all()
    x = torch.eye(k, device="cuda")[:32]
    y = torch.empty(32, n, device="cuda")
    qll.qll_q4g_linear(a, 32, 0, x, 0, None, 0, None, y, 0, 32, n, k, ws=workspace(32, n, k))
    d = np.asarray(d_bits, np.uint16).view(np.float16).astype(np.float64).reshape(n, -1)[:, :1]
    assert np.array_equal(R.f64(y), (d * (codes[:, :32].astype(np.float64) - 8.0)).T)


@pytest.mark.parametrize("act", list(E.ACTS))
@pytest.mark.parametrize("dtype,y_dtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                           ("f32", "f16")])
@pytest.mark.parametrize("m", [1, 6, 40])
def test_epilogues(qll_gpu, m, dtype, y_dtype, act):
    rng = np.random.default_rng(m)
    w = R.Weights(rng, 75, 320, 64, qll.QLL_Q4G_ZEROS, scale=0.02)
    x, xv = draw_x(rng, m, w.k, dtype)
    bias = synth.normal_f32(rng, (w.n,))
    res = torch.from_numpy(rng.standard_normal((m, w.n))).to(R.TYPES[y_dtype]).cuda()
    for with_bias, residual in ((True, None), (False, res), (True, res)):
        for in_place in (False, True) if residual is not None else (False,):
            y = call(w, x, dtype, dev(bias) if with_bias else None, act, residual, y_dtype, in_place)
            E.assert_bound(R.f64(y), *R.linear(w, xv, bias if with_bias else None, act,
                                               None if residual is None else R.f64(residual), y_dtype), act)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [1, 3, 16, 40, 70])
def test_a_row_with_nan_leaves_the_others(qll_gpu, m, dtype):
    rng = np.random.default_rng(m)
    w = R.Weights(rng, 48, 640, 128, qll.QLL_Q4G_ZEROS)
    x, _ = draw_x(rng, m, w.k, dtype)
    good = call(w, x, dtype, None, "none", None, "f32")
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[m // 2, 639] = bad
        got = call(w, y, dtype, None, "none", None, "f32")
        keep = torch.arange(m, device="cuda") != m // 2
        assert torch.equal(got[keep], good[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_small_and_large_activations(qll_gpu, dtype):
    """Subnormal and large values count in full."""
    rng = np.random.default_rng(1)
    w = R.Weights(rng, 64, 256, 64, qll.QLL_Q4G_ZEROS, scale=1.0)
    for size in (torch.finfo(R.TYPES[dtype]).smallest_normal / 4, 2000.0 if dtype == "f16" else 1e30):
        x = torch.from_numpy(rng.standard_normal((5, 256)) * size).to(R.TYPES[dtype]).cuda()
        y = call(w, x, dtype, None, "none", None, "f32")
        want, bound = w.product(R.f64(x))
        E.assert_bound(R.f64(y), want, bound + 2.0 ** -126, size)  # an f32 result below its normal range may be cut off


@pytest.mark.parametrize("dtype,m", [("bf16", 1), ("f32", 5), ("f16", 33), ("bf16", 200)])
def test_captured_and_on_another_stream(qll_gpu, dtype, m):
    rng = np.random.default_rng(m)
    w = R.Weights(rng, 300, 1024, 128, 0)
    x, _ = draw_x(rng, m, w.k, dtype)
    want = call(w, x, dtype, None, "silu", None, dtype)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    assert torch.equal(call(w, x, dtype, None, "silu", None, dtype, stream=other), want)
    y, ws = torch.zeros_like(want), workspace(m, w.n, w.k)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            qll.qll_q4g_linear(w.wp, 128, 0, x, R.CODES[dtype], None, qll.QLL_ACT_SILU, None, y, R.CODES[dtype], m,
                               w.n, w.k, ws=ws)
    for i in range(4):
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {i}"


# The kernels whose workgroups hold activation rows in LDS take products too large for the
# oracle's side on the CPU: (m, n, k, group), of 16-bit rows with 8, 16, 32 and 64 of them at once, k in
# parts over workgroups and not, ends of k inside a tile and a chunk; of f32 rows with 8 and 16.
LARGE = [("bf16", 8, 70001, 3872, 32), ("f16", 5, 66000, 4160, 64), ("bf16", 16, 1000, 33664, 64),
         ("f16", 9, 517, 66432, 32), ("f16", 20, 33001, 4128, 32), ("bf16", 32, 32800, 4224, 128),
         ("bf16", 70, 13000, 4256, 32), ("f16", 130, 8200, 4224, 128), ("bf16", 512, 520, 16576, 64),
         ("f16", 300, 3000, 8288, 32), ("f32", 7, 33000, 4128, 32), ("f32", 8, 32800, 4224, 128),
         ("f32", 12, 1000, 33664, 64), ("f32", 40, 11000, 4192, 32), ("f32", 130, 3700, 4224, 128),
         ("f32", 64, 600, 57472, 64)]
# The same with 17 rows and more near the sizes where they begin, in one to eight parts of k, with one to
# eight sets of waves a workgroup, one chunk of k and hundreds.
MIDDLE = [("bf16", 512, 1800, 1792, 64), ("f16", 500, 6000, 544, 32), ("bf16", 511, 33, 98304, 128),
          ("f16", 200, 16, 500000, 32), ("bf16", 128, 4099, 3104, 32), ("f16", 100, 20001, 768, 128),
          ("bf16", 64, 6500, 3904, 64), ("f16", 33, 70000, 512, 32), ("bf16", 17, 14000, 4160, 64),
          ("bf16", 32, 4000, 14400, 32), ("f32", 512, 1300, 1280, 128), ("f32", 64, 3300, 3840, 32),
          ("f32", 20, 26000, 1024, 64), ("f32", 100, 129, 57344, 128), ("f32", 257, 3000, 992, 32)]


@pytest.mark.parametrize("dtype,m,n,k,group", LARGE + MIDDLE)
def test_rows_in_lds(qll_gpu, dtype, m, n, k, group):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    fmt = FMTS[(m + n) % 4]
    groups, sdt = k // group, torch.bfloat16 if fmt & qll.QLL_Q4G_BF16 else torch.float16
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(n, groups, generator=g, device="cuda") - 0.5) / k ** 0.5).to(sdt)
    zeros = torch.randint(0, 16, (n, groups), generator=g, device="cuda", dtype=torch.uint8)
    wp = empty(qll.qll_q4g_packed_bytes(n, k, group, fmt))
    qll.qll_q4g_pack(codes, scales, zeros, group, fmt, wp, n, k)
    if not fmt & qll.QLL_Q4G_ZEROS:
        zeros.fill_(8)
    x = torch.randn(m, k, generator=g, device="cuda").to(R.TYPES[dtype])
    bias, res = torch.randn(n, generator=g, device="cuda"), torch.randn(m, n, generator=g, device="cuda").to(x.dtype)
    y = torch.full((m * n + GUARD,), 3.25, dtype=x.dtype, device="cuda")
    assert qll.qll_workspace_bytes(qll.QLL_OP_Q4G_LINEAR, m, n, k) > 0 or dtype != "f32"
    for _ in range(2):  # again in the same workspace
        qll.qll_q4g_linear(wp, group, fmt, x, R.CODES[dtype], bias, qll.QLL_ACT_SILU, res, y, R.CODES[dtype], m, n, k,
                           ws=workspace(m, n, k))
    torch.cuda.synchronize()
    assert (y[m * n:] == 3.25).all(), "wrote past the outputs"
    xd = x.double()
    for at in range(0, n, 8192):  # the bounds of q4g_refs, some rows at a time
        rows = slice(at, min(at + 8192, n))
        s = scales[rows].double().repeat_interleave(group, 1)
        z = zeros[rows].double().repeat_interleave(group, 1)
        c = codes[rows].double()
        want = xd @ (s * (c - z)).T
        mag = xd.abs() @ (s.abs() * (c - z).abs()).T
        off = 3 * group * R.U * (xd.abs() @ (s.abs() * (32.0 + c + z)).T)
        off += (groups + 12) * R.U * (mag + off) + 1e-36
        want, off = E.linear(want.cpu().numpy(), off.cpu().numpy(), bias[rows].cpu().numpy(), "silu", R.f64(res[:, rows]))
        E.assert_bound(R.f64(y[:m * n].view(m, n)[:, rows]), want, R.rounded(want, off, dtype), f"rows from {at}")


def test_offsets_past_32_bits(qll_gpu):
    """Codes of 4.3 GB: the first, the middle and the last rows, as packed on their own."""
    n, k, group, fmt = (1 << 21) + 40, 4096, 128, qll.QLL_Q4G_ZEROS
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(n, k // group, generator=g, device="cuda").half()
    zeros = torch.randint(0, 16, (n, k // group), generator=g, device="cuda", dtype=torch.uint8)
    wp = empty(qll.qll_q4g_packed_bytes(n, k, group, fmt))
    qll.qll_q4g_pack(codes, scales, zeros, group, fmt, wp, n, k)
    for m in (1, 20):
        x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        y = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
        qll.qll_q4g_linear(wp, group, fmt, x, 1, None, 0, None, y, 1, m, n, k, ws=workspace(m, n, k))
        for at in (0, (n // 2) // 16 * 16, n - 40):
            part = empty(qll.qll_q4g_packed_bytes(40, k, group, fmt))
            z = torch.empty(m, 40, device="cuda")
            rows = slice(at, at + 40)
            qll.qll_q4g_pack(codes[rows].contiguous(), scales[rows].contiguous(), zeros[rows].contiguous(), group, fmt,
                             part, 40, k)
            qll.qll_q4g_linear(part, group, fmt, x, 1, None, 0, None, z, 0, m, 40, k, ws=workspace(m, 40, k))
            # the two differ in how k is split: f32 sums of 32 groups, then one rounding to bf16
            assert torch.allclose(y[:, rows].float(), z, rtol=2.0 ** -8, atol=1e-3)
