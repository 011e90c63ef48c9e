"""The router and the mixture-of-experts layer on 4-bit weights against 64 bits,
with derived bounds (q4g_refs)."""
import numpy as np
import pytest
import torch

import epilogue_refs as E
import q4g_refs as R
import quantized_linear_layer_amd as qll
import synth
from gpu_util import dev, empty

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = qll.QLL_SCORE_SOFTMAX, qll.QLL_SCORE_SIGMOID
FMTS = [0, qll.QLL_Q4G_BF16, qll.QLL_Q4G_ZEROS, qll.QLL_Q4G_BF16 | qll.QLL_Q4G_ZEROS]


def of(rng, shape, dtype, size=1.0):
    t = torch.from_numpy(rng.standard_normal(shape) * size).to(R.TYPES[dtype]).cuda()
    return t, R.f64(t)


def route_call(x, dtype, wr, wr_dtype, bias, score, renorm, scale, top, stream=None):
    m, k = x.shape
    e = wr.shape[0]
    ids = torch.full((m * top + 16,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((m * top + 16,), 3.25, device="cuda")
    ws = torch.full((qll.qll_workspace_bytes(qll.QLL_OP_MOE_ROUTE, m, e, top),), 0xFF, dtype=torch.uint8, device="cuda")
    qll.qll_moe_route(x, R.CODES[dtype], wr, R.CODES[wr_dtype], bias, score, renorm, scale, ids, w, top, m, e, k,
                      ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert (ids[m * top:] == -7).all() and (w[m * top:] == 3.25).all(), "wrote past the outputs"
    return ids[:m * top].view(m, top), w[:m * top].view(m, top)


# (m, experts, top, k): one token to more than two hundred, one expert to the most, odd k
ROUTES = [(1, 1, 1, 1), (1, 2, 1, 7), (3, 5, 5, 33), (1, 128, 8, 2048), (64, 64, 6, 256), (7, 1024, 32, 100),
          (65, 300, 4, 65), (2, 63, 3, 1000), (130, 17, 2, 512), (5, 257, 8, 4095), (200, 8, 2, 128)]


@pytest.mark.parametrize("m,e,top,k", ROUTES)
@pytest.mark.parametrize("dtype,wr_dtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                            ("f32", "f16")])
def test_route(qll_gpu, m, e, top, k, dtype, wr_dtype):
    rng = np.random.default_rng(m + e + top + k)
    x, xv = of(rng, (m, k), dtype)
    wr, wv = of(rng, (e, k), wr_dtype, 1.5 / np.sqrt(k))
    bias = (0.1 * synth.normal_f32(rng, (e,))).astype(np.float32)
    for score in (SOFTMAX, SIGMOID):
        for b in (None, bias):
            for renorm in (0, 1):
                ids, w = route_call(x, dtype, wr, wr_dtype, None if b is None else dev(b), score, renorm, 2.5, top)
                want, ww = R.route(xv, wv, b, score, renorm, 2.5, top)
                assert np.array_equal(ids.cpu().numpy(), want), (score, renorm)
                # f64 scores, rounded to f32 once (or cut off below its normal range)
                assert np.all(np.abs(R.f64(w) - ww) <= 2.0 ** -23 * np.abs(ww) + 2.0 ** -126)


def test_route_ties_and_extremes(qll_gpu):
    """Equal logits go to the lower index, also across lanes and as -0 and +0; a
    bias moves the choice and not the weight; far logits."""
    e, k = 200, 4
    wr = torch.zeros(e, k, device="cuda")
    x = torch.ones(3, k, device="cuda")
    x[1] = -1.0  # every logit -0
    ids, w = route_call(x, "f32", wr, "f32", None, SOFTMAX, 0, 1.0, 10)
    assert torch.equal(ids.cpu(), torch.arange(10, dtype=torch.int32).repeat(3, 1))
    assert torch.allclose(w, torch.full_like(w, 1 / e), rtol=1e-6, atol=0)
    wr[70] = wr[6] = wr[199] = 1.0
    wr[130] = 300.0
    ids, w = route_call(x[:1], "f32", wr, "f32", None, SOFTMAX, 0, 1.0, 6)
    assert ids[0].tolist() == [130, 6, 70, 199, 0, 1] and w[0].tolist() == [1.0, 0.0, 0.0, 0.0, 0.0, 0.0]
    bias = torch.zeros(e, device="cuda")
    bias[150] = 4.0
    ids, w = route_call(x[:1], "f32", wr, "f32", bias, SIGMOID, 1, 1.0, 2)
    assert ids[0].tolist() == [150, 130]
    assert torch.allclose(w[0].cpu(), torch.tensor([1 / 3, 2 / 3]), rtol=1e-6, atol=0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_of_a_bad_row(qll_gpu, bad, score):
    rng = np.random.default_rng(5)
    x, _ = of(rng, (6, 64), "f32")
    wr, _ = of(rng, (40, 64), "f32", 0.2)
    good, gw = route_call(x, "f32", wr, "f32", None, score, 1, 1.0, 8)
    y = x.clone()
    y[4, 10] = bad
    ids, w = route_call(y, "f32", wr, "f32", None, score, 1, 1.0, 8)
    keep = torch.arange(6, device="cuda") != 4
    assert torch.equal(ids[keep], good[keep]) and torch.equal(w[keep], gw[keep])
    row = ids[4].tolist()
    assert len(set(row)) == 8 and min(row) >= 0 and max(row) < 40


class Experts:
    def __init__(self, rng, e, n, k, group, fmt):
        self.e, self.n, self.k, self.group, self.fmt = e, n, k, group, fmt
        self.wg, self.wu = (R.Weights(rng, n, k, group, fmt, e) for _ in range(2))
        self.wd = R.Weights(rng, k, n, group, fmt, e)


def moe_call(ex, x, dtype, ids, weights, act, residual, in_place=False, stream=None):
    m, top = ids.shape
    y = torch.full((m * ex.k + 64,), 3.25, dtype=x.dtype, device="cuda")
    if in_place:
        y[:m * ex.k] = residual.reshape(-1)
        residual = y
    ws = torch.full((qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, ex.n, top),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    qll.qll_q4g_moe(x, R.CODES[dtype], ids, weights, top, ex.wg.wp, ex.wu.wp, ex.wd.wp, ex.group, ex.fmt, E.ACTS[act],
                    residual, y, m, ex.n, ex.k, ex.e, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert (y[m * ex.k:] == 3.25).all(), "wrote past the outputs"
    return y[:m * ex.k].view(m, ex.k)


def choices(rng, m, e, top):
    ids = np.stack([rng.permutation(e)[:top] for _ in range(m)]).astype(np.int32)
    return ids, rng.uniform(0.05, 1.0, (m, top)).astype(np.float32)


def check(ex, xv, ids, weights, act, residual, dtype, y, what):
    E.assert_bound(R.f64(y), *R.moe(xv, ids, weights, ex.wg, ex.wu, ex.wd, act,
                                    None if residual is None else R.f64(residual), dtype), what)


# (m, experts, top, n / group, k / group)
LAYERS = [(1, 1, 1, 1, 1), (1, 4, 2, 3, 5), (1, 9, 8, 9, 4), (2, 7, 3, 5, 2), (5, 3, 2, 4, 7), (16, 20, 4, 2, 3),
          (23, 2, 1, 6, 5), (40, 2, 2, 3, 4), (64, 5, 3, 5, 3), (67, 6, 2, 2, 5), (130, 3, 1, 1, 2)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,e,top,n,k", LAYERS)
def test_experts(qll_gpu, m, e, top, n, k, dtype, group):
    rng = np.random.default_rng(m + e + n + k)
    ex = Experts(rng, e, n * group, k * group, group, FMTS[(m + n) % 4])
    x, xv = of(rng, (m, ex.k), dtype)
    ids, weights = choices(rng, m, e, top)
    act = list(E.ACTS)[(m + e) % 5]
    residual = of(rng, (m, ex.k), dtype)[0] if n % 2 else None
    y = moe_call(ex, x, dtype, dev(ids), dev(weights), act, residual)
    check(ex, xv, ids, weights, act, residual, dtype, y, act)
    if residual is not None:
        assert torch.equal(moe_call(ex, x, dtype, dev(ids), dev(weights), act, residual, in_place=True), y)


@pytest.mark.parametrize("m", [1, 9, 64, 70])
def test_padding_and_repeated_choices(qll_gpu, m):
    """Ids outside [0, e) add nothing, with weights that are not numbers; rows of them
    keep their residual; an expert named twice counts with both weights."""
    rng = np.random.default_rng(m)
    ex = Experts(rng, 6, 96, 64, 32, qll.QLL_Q4G_ZEROS)
    x, xv = of(rng, (m, 64), "f32")
    ids = rng.integers(0, 6, (m, 5)).astype(np.int32)  # repeats
    weights = rng.uniform(0.05, 1.0, (m, 5)).astype(np.float32)
    out = rng.random((m, 5)) < 0.3
    ids[out] = rng.choice([-1, 6, 2 ** 31 - 1, -2 ** 31], out.sum())
    weights[out] = np.nan
    ids[m // 2] = -1
    residual, rv = of(rng, (m, 64), "f32")
    for res in (None, residual):
        y = moe_call(ex, x, "f32", dev(ids), dev(weights), "silu", res)
        check(ex, xv, ids, weights, "silu", res, "f32", y, "padded")
        assert torch.equal(y[m // 2], torch.zeros(64, device="cuda") if res is None else residual[m // 2])
    nothing = np.full((m, 5), -1, np.int32)
    y = moe_call(ex, x, "f32", dev(nothing), dev(weights), "silu", residual)
    assert torch.equal(y, residual)


def test_many_experts_and_the_widest_choice(qll_gpu):
    rng = np.random.default_rng(3)
    ex = Experts(rng, 1024, 32, 32, 32, 0)
    for m in (1, 64):
        x, xv = of(rng, (m, 32), "bf16")
        ids, weights = choices(rng, m, 1024, 32)
        y = moe_call(ex, x, "bf16", dev(ids), dev(weights), "gelu", None)
        check(ex, xv, ids, weights, "gelu", None, "bf16", y, f"m = {m}")


def test_all_tokens_on_one_expert(qll_gpu):
    rng = np.random.default_rng(4)
    ex = Experts(rng, 3, 320, 192, 64, qll.QLL_Q4G_ZEROS)
    for m in (4, 5, 16, 17, 33, 64):
        x, xv = of(rng, (m, 192), "f16")
        ids = np.full((m, 1), 2, np.int32)
        weights = rng.uniform(-1.0, 1.0, (m, 1)).astype(np.float32)
        y = moe_call(ex, x, "f16", dev(ids), dev(weights), "relu", None)
        check(ex, xv, ids, weights, "relu", None, "f16", y, f"m = {m}")


def test_a_token_with_nan_leaves_the_others(qll_gpu):
    rng = np.random.default_rng(6)
    ex = Experts(rng, 4, 128, 256, 128, qll.QLL_Q4G_ZEROS)
    for dtype in R.TYPES:
        x, _ = of(rng, (20, 256), dtype)
        ids, weights = choices(rng, 20, 4, 2)
        good = moe_call(ex, x, dtype, dev(ids), dev(weights), "silu", None)
        x[11, 200] = float("nan")
        y = moe_call(ex, x, dtype, dev(ids), dev(weights), "silu", None)
        keep = torch.arange(20, device="cuda") != 11
        assert torch.equal(y[keep], good[keep]), dtype


@pytest.mark.parametrize("m,dtype", [(1, "bf16"), (1, "f32"), (13, "f16"), (64, "bf16"), (100, "f32")])
def test_layer_is_its_parts_eager_and_captured(qll_gpu, m, dtype):
    """qll_q4g_moe_layer gives what the router and the experts give one after
    the other; captured, replays give it again, on inputs that change."""
    rng = np.random.default_rng(m)
    e, top = 12, 3
    ex = Experts(rng, e, 256, 384, 64, qll.QLL_Q4G_ZEROS)
    wr, _ = of(rng, (e, 384), "f32", 0.1)
    bias = dev(0.05 * synth.normal_f32(rng, (e,)))
    x, _ = of(rng, (m, 384), dtype)
    residual, _ = of(rng, (m, 384), dtype)
    sizes = (qll.qll_workspace_bytes(qll.QLL_OP_MOE_ROUTE, m, e, top), qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, 256, top))
    ws = empty(sum(sizes))
    ids, w, y = empty(m * top, torch.int32), empty(m * top, torch.float32), torch.zeros_like(x)

    def layer():
        qll.qll_q4g_moe_layer(x, R.CODES[dtype], wr, 0, bias, SIGMOID, 1, 2.5, ids, w, top, ex.wg.wp, ex.wu.wp,
                              ex.wd.wp, 64, ex.fmt, qll.QLL_ACT_SILU, residual, y, m, 256, 384, e, ws=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            layer()
    for i in range(4):
        x.copy_(of(rng, (m, 384), dtype)[0])
        pi, pw = route_call(x, dtype, wr, "f32", bias, SIGMOID, 1, 2.5, top)
        want = moe_call(ex, x, dtype, pi.contiguous(), pw.contiguous(), "silu", residual)
        for run in (layer, g.replay):
            for t in (ids, w, y):
                t.zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert torch.equal(ids.view(m, top), pi) and torch.equal(w.view(m, top), pw) and torch.equal(y, want), i
