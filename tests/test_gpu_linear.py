"""qll_q4_0_q8_0_linear, the gated projection and their repacked forms against
64-bit evaluation of the oracle's products, on every kernel they dispatch to,
with derived bounds (epilogue_refs).  Outputs are written into a buffer with
guard values behind them."""
import numpy as np
import pytest
import torch

import epilogue_refs as E
import oracle as O
import quantized_linear_layer_amd as qll
import synth
from gpu_util import dev, empty, pack_q4_0, q4_gemm, quantize_q8_0

pytestmark = pytest.mark.gpu
GUARD = 64


class Layer:
    """Raw draws, device operands and the oracle's products of one shape."""

    def __init__(self, seed, m, n, k, pair=False):
        rng = np.random.default_rng(seed)
        self.m, self.n, self.k = m, n, k
        self.raw = [synth.q4_0_weights(rng, n, k) for _ in range(2 if pair else 1)]
        x = synth.normal_f32(rng, (m, k)) * np.float32(3.0)
        self.w = [pack_q4_0(*r) for r in self.raw]
        self.xq = quantize_q8_0(x)
        xq_ref = O.quantize_q8_0(x)
        self.products = [E.product(c, d, xq_ref, m) for c, d in self.raw]
        self.bias = synth.normal_f32(rng, (n,))
        self.residual = synth.normal_f32(rng, (m, n))

    def out(self):
        return torch.full((self.m * self.n + GUARD,), 3.25, device="cuda")

    def host(self, y):
        torch.cuda.synchronize()
        a = y.cpu().numpy()
        assert (a[self.m * self.n:] == 3.25).all(), "wrote past the outputs"
        return a[:self.m * self.n].reshape(self.m, self.n)


def workspace(op, m, n, k):
    need = qll.qll_workspace_bytes(op, m, n, k)
    return empty(need) if need else None


def run_linear(layer, repacked, bias, act, residual, in_place=False, stream=None):
    m, n, k = layer.m, layer.n, layer.k
    b = dev(layer.bias) if bias else None
    y = layer.out()
    if in_place:
        y[:m * n] = dev(layer.residual).reshape(-1)
        r = y
    else:
        r = dev(layer.residual) if residual else None
    a = E.ACTS[act]
    if repacked:
        wp = empty(qll.qll_q4_0_repacked_bytes(n, k))
        qll.qll_q4_0_repack(layer.w[0], wp, n, k)
        ws = workspace(qll.QLL_OP_Q4_0_REPACKED_GEMM, m, n, k)
        qll.qll_q4_0_repacked_q8_0_linear(wp, layer.xq, b, a, r, y, m, n, k, ws=ws, stream=stream)
    else:
        ws = workspace(qll.QLL_OP_Q4_0_LINEAR, m, n, k)
        qll.qll_q4_0_q8_0_linear(layer.w[0], layer.xq, b, a, r, y, m, n, k, ws=ws, stream=stream)
    return layer.host(y)


EPILOGUES = [("none", False, False), ("relu", True, False), ("gelu", True, True), ("gelu_tanh", False, True),
             ("silu", True, False)]

# the GEMV (even and odd block counts, few and many blocks), the GEMV-style
# kernel (m = 2 and 4 on tall matrices, rows under eight blocks), the int8
# matrix-core kernel (each number of staged rows, one and two weight tiles,
# groups of 16 and 32 rows), its form for tall matrices, the 128-row GEMM with and
# without a split k
BLOCKS = [(1, 1, 32), (1, 67, 96), (1, 300, 4096), (1, 129, 14368), (1, 20000, 320), (1, 5, 49152),
          (2, 8200, 512), (4, 32770, 256), (5, 64, 96), (40, 70, 224),
          (9, 8200, 224), (13, 33000, 32), (64, 130, 64), (33, 8192, 96), (16, 50, 192),
          (3, 200, 1024), (8, 33, 256), (16, 300, 2048), (27, 77, 288), (20, 8200, 256), (33, 96, 512), (64, 40, 1056), (37, 4100, 4096), (64, 65600, 256), (50, 33, 288), (17, 2048, 2048),
          (48, 8200, 1056), (33, 300, 16416), (49, 14336, 2560), (64, 6144, 288),
          (7, 32800, 256), (12, 32770, 288),
          (65, 257, 1024), (130, 129, 96), (128, 128, 4096), (257, 132, 544), (512, 300, 256), (1000, 17, 288),
          (4096, 20, 256), (4097, 20, 256), (130, 2100, 96), (64, 4100, 224), (70, 32800, 256), (2000, 130, 64)]


@pytest.mark.parametrize("m,n,k", BLOCKS)
def test_linear(qll_gpu, m, n, k):
    layer = Layer(m + n + k, m, n, k)
    v, ev = layer.products[0]
    for act, bias, residual in EPILOGUES:
        got = run_linear(layer, False, bias, act, residual)
        want, bound = E.linear(v, ev, layer.bias if bias else None, act, layer.residual if residual else None)
        E.assert_bound(got, want, bound, f"{act} bias={bias} residual={residual}")
        if act == "none" and (m <= 16 or (m > 64 and qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, m, n, k))):  # the same kernels
            plain = q4_gemm(layer.w[0], layer.xq, m, n, k)
            torch.cuda.synchronize()
            assert np.array_equal(got.view(np.uint32), plain.cpu().numpy().reshape(m, n).view(np.uint32)), \
                "without an epilogue it is the plain product bit for bit"


@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 130, 4096), (17, 64, 256), (65, 257, 1024), (130, 129, 96),
                                   (128, 128, 64), (300, 130, 4096)])
def test_linear_repacked(qll_gpu, m, n, k):
    layer = Layer(m + n + k + 1, m, n, k)
    v, ev = layer.products[0]
    for act, bias, residual in EPILOGUES:
        got = run_linear(layer, True, bias, act, residual)
        want, bound = E.linear(v, ev, layer.bias if bias else None, act, layer.residual if residual else None)
        E.assert_bound(got, want, bound, f"{act} bias={bias} residual={residual}")


@pytest.mark.parametrize("repacked", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 512), (16, 300, 512), (40, 70, 96), (65, 257, 1024), (130, 1024, 128)])
def test_residual_in_place(qll_gpu, m, n, k, repacked):
    layer = Layer(m * n + k, m, n, k)
    v, ev = layer.products[0]
    got = run_linear(layer, repacked, True, "none", True, in_place=True)
    E.assert_bound(got, *E.linear(v, ev, layer.bias, "none", layer.residual), "in place")
    other = run_linear(layer, repacked, True, "none", True)
    assert np.array_equal(got.view(np.uint32), other.view(np.uint32))


@pytest.mark.parametrize("act", list(E.ACTS))
@pytest.mark.parametrize("m", [1, 9, 70])
def test_activations_far_from_zero(qll_gpu, act, m):
    """Arguments from -1e4 to 1e4 through the bias, zero among them."""
    layer = Layer(77 + m, m, 201, 256)
    layer.bias = np.concatenate([-np.logspace(-4, 4, 100), [0.0], np.logspace(-4, 4, 100)]).astype(np.float32)
    v, ev = layer.products[0]
    got = run_linear(layer, False, True, act, False)
    E.assert_bound(got, *E.linear(v, ev, layer.bias, act, None), act)


def run_gated(layer, repacked, act):
    m, n, k = layer.m, layer.n, layer.k
    y = layer.out()
    if repacked:
        wp = torch.full((qll.qll_q4_0_repacked_gated_bytes(n, k) + GUARD,), 0x77, dtype=torch.uint8, device="cuda")
        qll.qll_q4_0_repack_gated(layer.w[0], layer.w[1], wp, n, k)
        assert (wp[-GUARD:] == 0x77).all()
        ws = workspace(qll.QLL_OP_Q4_0_REPACKED_GATED, m, n, k)
        qll.qll_q4_0_repacked_q8_0_gated(wp, layer.xq, E.ACTS[act], y, m, n, k, ws=ws)
    else:
        ws = workspace(qll.QLL_OP_Q4_0_GATED, m, n, k)
        qll.qll_q4_0_q8_0_gated(layer.w[0], layer.w[1], layer.xq, E.ACTS[act], y, m, n, k, ws=ws)
    return layer.host(y)


# the GEMV, the matrix-core kernel (each number of staged rows and waves, one
# row past the GEMV's k, groups of 32), the 128-row GEMM (short rows, split)
GATED = [(1, 1, 32), (1, 67, 96), (1, 300, 4096), (1, 33, 14368), (1, 20000, 320), (1, 9, 49152), (1, 17, 49184),
         (2, 200, 1024), (4, 33, 256), (6, 16, 4096), (8, 300, 2048), (12, 4100, 256), (16, 15, 8192), (27, 77, 288),
         (32, 5000, 512), (33, 96, 512), (64, 40, 1056), (9, 16500, 256), (37, 2100, 4096), (64, 33000, 256), (20, 1024, 1024),
         (64, 500, 2080), (48, 4100, 2080), (61, 300, 512), (17, 4096, 1024),
         (2, 64, 96), (40, 70, 224), (65, 257, 1024), (130, 129, 96), (257, 132, 544), (128, 64, 4096),
         (500, 33, 1056), (4096, 20, 256), (4097, 20, 256), (70, 33000, 256), (4100, 40, 4096)]


@pytest.mark.parametrize("m,n,k", GATED)
def test_gated(qll_gpu, m, n, k):
    layer = Layer(3 * m + n + k, m, n, k, pair=True)
    (g, eg), (u, eu) = layer.products
    for act in E.ACTS:
        E.assert_bound(run_gated(layer, False, act), *E.gated(g, eg, u, eu, act), act)


@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 130, 4096), (17, 64, 256), (65, 257, 1024), (130, 129, 96),
                                   (128, 63, 64), (300, 130, 4096), (129, 1000, 544)])
def test_gated_repacked(qll_gpu, m, n, k):
    layer = Layer(5 * m + n + k, m, n, k, pair=True)
    (g, eg), (u, eu) = layer.products
    for act in E.ACTS:
        E.assert_bound(run_gated(layer, True, act), *E.gated(g, eg, u, eu, act), act)


def test_repacked_pair_is_two_repacks_interleaved(qll_gpu):
    """Byte for byte: 64-row halves of each 128-row tile."""
    n, k = 200, 96
    layer = Layer(11, 1, n, k, pair=True)
    nb = k // 32
    wp = empty(qll.qll_q4_0_repacked_gated_bytes(n, k))
    qll.qll_q4_0_repack_gated(layer.w[0], layer.w[1], wp, n, k)
    rows = -(-n // 64) * 128
    both = torch.zeros(rows, nb, 18, dtype=torch.uint8, device="cuda")
    both[..., 2:] = 0x88  # code 8: weight zero, as a padded row has it
    for h, w in enumerate(layer.w):
        w = w.view(n, nb, 18)
        for r0 in range(0, n, 64):
            c = min(64, n - r0)
            both[2 * r0 + 64 * h:2 * r0 + 64 * h + c] = w[r0:r0 + c]
    want = empty(qll.qll_q4_0_repacked_bytes(rows, k))
    qll.qll_q4_0_repack(both.reshape(-1), want, rows, k)
    torch.cuda.synchronize()
    assert torch.equal(wp, want)


@pytest.mark.parametrize("m", [1, 16, 512])
def test_8b_layer_every_output(qll_gpu, m):
    """The gate and up projections (4096 -> 14336) and the down projection with
    its residual (14336 -> 4096) at full size."""
    layer = Layer(123, m, 14336, 4096, pair=True)
    (g, eg), (u, eu) = layer.products
    E.assert_bound(run_gated(layer, False, "silu"), *E.gated(g, eg, u, eu, "silu"), "gated")
    if m == 512:
        E.assert_bound(run_gated(layer, True, "silu"), *E.gated(g, eg, u, eu, "silu"), "gated repacked")
    del layer
    down = Layer(124, m, 4096, 14336)
    v, ev = down.products[0]
    want, bound = E.linear(v, ev, None, "none", down.residual)
    E.assert_bound(run_linear(down, False, False, "none", True), want, bound, "down")
    if m == 512:
        E.assert_bound(run_linear(down, True, False, "none", True), want, bound, "down repacked")


def test_another_stream_and_determinism(qll_gpu):
    layer = Layer(9, 65, 300, 1024)
    s = torch.cuda.Stream()
    first = run_linear(layer, False, True, "gelu", True)
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        second = run_linear(layer, False, True, "gelu", True)
    third = run_linear(layer, False, True, "gelu", True, stream=torch.cuda.current_stream())
    assert np.array_equal(first.view(np.uint32), second.view(np.uint32))
    assert np.array_equal(first.view(np.uint32), third.view(np.uint32))


@pytest.mark.parametrize("repacked", [False, True])
@pytest.mark.parametrize("m", [1, 2, 40, 70])
@pytest.mark.parametrize("act", list(E.ACTS))
def test_nan_and_infinity_reach_the_output(qll_gpu, act, m, repacked):
    layer = Layer(31, m, 70, 256)
    clean = run_linear(layer, repacked, True, act, True)
    layer.bias[3], layer.bias[40] = np.nan, np.inf
    layer.residual[m - 1, 5], layer.residual[0, 6] = np.nan, -np.inf
    got = run_linear(layer, repacked, True, act, True)
    assert np.isnan(got[:, 3]).all() and (got[:, 40] == np.inf).all()
    assert np.isnan(got[m - 1, 5]) and got[0, 6] == -np.inf
    got[:, [3, 40]] = clean[:, [3, 40]]
    got[m - 1, 5], got[0, 6] = clean[m - 1, 5], clean[0, 6]
    assert np.array_equal(got.view(np.uint32), clean.view(np.uint32)), "other outputs changed"


@pytest.mark.parametrize("m", [1, 7, 40, 70])
def test_gate_and_up_the_same_matrix(qll_gpu, m):
    layer = Layer(32, m, 70, 256)
    layer.raw, layer.w, layer.products = layer.raw * 2, layer.w * 2, layer.products * 2
    (g, eg), (u, eu) = layer.products
    for repacked in (False, True):
        E.assert_bound(run_gated(layer, repacked, "relu"), *E.gated(g, eg, u, eu, "relu"), "relu")


def test_outputs_past_32_bits(qll_gpu):
    """65600 x 33000 outputs, the residual in place: the last rows are those of
    a small call."""
    m, n, k, last = 65600, 33000, 32, 70
    rng = np.random.default_rng(33)
    w = [pack_q4_0(*synth.q4_0_weights(rng, n, k)) for _ in range(2)]
    xq = quantize_q8_0(synth.normal_f32(rng, (m, k)))
    tail = xq.reshape(m, -1)[-last:].clone().reshape(-1)  # (the slice itself is not 16-byte aligned)
    y, ys = torch.ones(m * n, device="cuda"), torch.ones(last * n, device="cuda")
    b = dev(synth.normal_f32(rng, (n,)))
    for rows, q, out in ((m, xq, y), (last, tail, ys)):
        ws = workspace(qll.QLL_OP_Q4_0_LINEAR, rows, n, k)
        qll.qll_q4_0_q8_0_linear(w[0], q, b, qll.QLL_ACT_GELU, out, out, rows, n, k, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(y[-last * n:], ys)
    for rows, q, out in ((m, xq, y), (last, tail, ys)):
        ws = workspace(qll.QLL_OP_Q4_0_GATED, rows, n, k)
        qll.qll_q4_0_q8_0_gated(*w, q, qll.QLL_ACT_SILU, out, rows, n, k, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(y[-last * n:], ys)
