"""The operators on 4-bit group-scaled weights in the order a decoder uses them:
a projection added to the stream, the mixture-of-experts layer added to it, the
vocabulary projection, log probabilities.  Every step against the 64-bit form
of what it was given; the run captured into two graphs that share a workspace
and replayed in turn; two runs on two streams at once; and the experts at
sizes where tokens go in groups and rows pass through LDS in chunks."""
import numpy as np
import pytest
import torch

import epilogue_refs as E
import logprob_refs as L
import q4g_refs as R
import quantized_linear_layer_amd as qll
from gpu_util import dev, empty

pytestmark = pytest.mark.gpu

HIDDEN, FFN, VOCAB, EXPERTS, CHOSEN, TOP = 320, 192, 1003, 12, 3, 5
FMT, GROUP = qll.QLL_Q4G_ZEROS | qll.QLL_Q4G_BF16, 64
F32 = qll.QLL_DTYPE_F32


class Run:
    """Weights, inputs and outputs for m rows of a stream of type dtype."""

    def __init__(self, m, dtype, seed, vocab=VOCAB, hidden=HIDDEN):
        rng = np.random.default_rng(seed)
        t, self.code = R.TYPES[dtype], R.CODES[dtype]
        self.m, self.dtype, self.vocab, self.hidden = m, dtype, vocab, hidden
        self.wo = R.Weights(rng, hidden, hidden, 32, 0)
        self.wg, self.wu = (R.Weights(rng, FFN, hidden, GROUP, FMT, EXPERTS) for _ in range(2))
        self.wd = R.Weights(rng, hidden, FFN, GROUP, FMT, EXPERTS)
        self.head = R.Weights(rng, vocab, hidden, 32, qll.QLL_Q4G_ZEROS)
        self.wr = torch.from_numpy(rng.standard_normal((EXPERTS, hidden)) * 0.1).float().cuda()
        self.bias = dev(rng.uniform(-0.05, 0.05, EXPERTS).astype(np.float32))
        self.a, self.x = (torch.zeros(m, hidden, dtype=t, device="cuda") for _ in range(2))
        self.h, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.ids, self.w = empty(m * CHOSEN, torch.int32), empty(m * CHOSEN, torch.float32)
        self.tokens, self.logits = empty(m, torch.int32), empty(m * vocab, torch.float32)
        self.lp, self.en = empty(m, torch.float32), empty(m, torch.float32)
        self.top_ids, self.top_lp = empty(m * TOP, torch.int32), empty(m * TOP, torch.float32)
        need = qll.qll_workspace_bytes
        self.need = max(16, need(qll.QLL_OP_Q4G_LINEAR, m, hidden, hidden), need(qll.QLL_OP_Q4G_LINEAR, m, vocab, hidden),
                        need(qll.QLL_OP_MOE_ROUTE, m, EXPERTS, CHOSEN) + need(qll.QLL_OP_Q4G_MOE, m, FFN, CHOSEN),
                        need(qll.QLL_OP_TOKEN_LOGPROBS, m, vocab, TOP))
        self.ws = empty(self.need)

    def feed(self, seed):
        rng = np.random.default_rng(seed)
        for t in (self.a, self.x):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape)))
        self.tokens.copy_(dev(rng.integers(0, self.vocab, self.m).astype(np.int32)))
        torch.cuda.synchronize()

    def run(self, stream=None):
        m, k, t, ws = self.m, self.hidden, self.code, self.ws
        qll.qll_q4g_linear(self.wo.wp, 32, 0, self.a, t, None, qll.QLL_ACT_NONE, self.x, self.h, t, m, k, k, ws=ws,
                           stream=stream)
        qll.qll_q4g_moe_layer(self.h, t, self.wr, F32, self.bias, qll.QLL_SCORE_SIGMOID, 1, 2.5, self.ids, self.w,
                              CHOSEN, self.wg.wp, self.wu.wp, self.wd.wp, GROUP, FMT, qll.QLL_ACT_SILU, self.h, self.y,
                              m, FFN, k, EXPERTS, ws=ws, stream=stream)
        qll.qll_q4g_linear(self.head.wp, 32, qll.QLL_Q4G_ZEROS, self.y, t, None, qll.QLL_ACT_NONE, None, self.logits,
                           F32, m, self.vocab, k, ws=ws, stream=stream)
        qll.qll_token_logprobs(self.logits, F32, self.tokens, 1, self.lp, self.en, TOP, self.top_ids, self.top_lp, m,
                               self.vocab, ws=ws, stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.h, self.ids, self.w, self.y, self.logits, self.lp, self.en, self.top_ids,
                                    self.top_lp)]


def moe_by_expert(x, ids, weights, wg, wu, wd, act, residual, dtype):
    """q4g_refs.moe, an expert's rows at a time."""
    m, top = ids.shape
    y, b, mag = (np.zeros((m, wd.n)) for _ in range(3))
    for e in range(wg.count):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        h, eh = E.gated(*wg.product(x[t], i=e), *wu.product(x[t], i=e), act)
        if dtype != "f32":
            eh = eh + (np.abs(h) + eh) * 2.0 ** -16
        d, ed = wd.product(h, eh, i=e)
        w = weights[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, w * d)
        np.add.at(b, t, np.abs(w) * ed)
        np.add.at(mag, t, np.abs(w) * (np.abs(d) + ed))
    b += (top + 12) * R.U * mag
    if residual is not None:
        y = y + residual
        b = b + R.U * (np.abs(y) + b)
    return y, R.rounded(y, b, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [1, 6, 80])
def test_run(qll_gpu, m, dtype):
    r = Run(m, dtype, m)
    r.feed(m)
    r.run()
    h, ids, w, y, logits, lp, en, top_ids, top_lp = r.outputs()
    E.assert_bound(R.f64(h), *R.linear(r.wo, R.f64(r.a), None, "none", R.f64(r.x), dtype), "projection")
    want, ww = R.route(R.f64(h), R.f64(r.wr), r.bias.cpu().numpy(), qll.QLL_SCORE_SIGMOID, 1, 2.5, CHOSEN)
    ids, w = ids.cpu().numpy().reshape(m, CHOSEN), w.cpu().numpy().reshape(m, CHOSEN)
    assert np.array_equal(ids, want)
    assert np.all(np.abs(w - ww) <= 2.0 ** -23 * np.abs(ww))
    E.assert_bound(R.f64(y), *moe_by_expert(R.f64(h), ids, w, r.wg, r.wu, r.wd, "silu", R.f64(h), dtype), "experts")
    v, b = r.head.product(R.f64(y))
    E.assert_bound(R.f64(logits).reshape(m, VOCAB), v, R.rounded(v, b, "f32"), "logits")
    want = L.reference(logits.cpu().numpy().reshape(m, VOCAB), r.tokens.cpu().numpy().reshape(m, 1), TOP)
    assert np.array_equal(top_ids.cpu().numpy().reshape(m, TOP), want[2])
    L.assert_close(lp.cpu().numpy().reshape(m, 1), want[0], want[4], "given")
    L.assert_close(top_lp.cpu().numpy().reshape(m, TOP), want[3], want[4], "chosen")
    L.assert_close(en.cpu().numpy(), want[1], want[5], "entropy")


# (m, type, columns of the vocabulary, hidden): the last two's vocabulary projection splits f32 rows
# into parts in the workspace, or takes them from LDS
RUNS = [(1, "bf16", VOCAB, HIDDEN), (80, "f32", VOCAB, HIDDEN), (7, "f32", 70016, 2048), (80, "bf16", 30016, 2048)]


@pytest.mark.parametrize("m,dtype,vocab,hidden", RUNS)
def test_two_graphs_share_a_workspace(qll_gpu, m, dtype, vocab, hidden):
    runs = [Run(m, dtype, seed, vocab, hidden) for seed in (1, 2)]
    runs[1].ws = runs[0].ws
    graphs = []
    for i, r in enumerate(runs):
        r.feed(i)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            r.run()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.run()
        graphs.append(g)
    for seed in range(10, 14):
        for i, r in enumerate(runs):
            r.feed(2 * seed + i)
        for g in graphs:
            g.replay()
        got = [r.outputs() for r in runs]
        runs[0].ws.fill_(255)
        for r, outs in zip(runs, got):
            r.run()
            for a, b in zip(outs, r.outputs()):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), seed


def test_two_streams_at_once(qll_gpu):
    runs = [Run(m, dtype, m) for m, dtype in ((1, "bf16"), (9, "f32"), (80, "f16"))]
    want = []
    for r in runs:
        r.feed(r.m)
        r.run()
        want.append(r.outputs())
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for r in runs:
            r.y.zero_(), r.logits.zero_()
        torch.cuda.synchronize()
        for r, s in zip(runs, streams):
            r.run(stream=s)
        for r, outs in zip(runs, want):
            for a, b in zip(r.outputs(), outs):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# (m, experts, top, n, k, group, type).  Up to 64 tokens go at once, fewer where their choices' down products
# would take more than 32 MiB: the first ones go in groups of 4 and 1, 9 and 3, 51 and 9, 1.  The others' rows
# pass through LDS in several chunks, of 4, 8 and 16 of them, gate, up and down.
SIZES = [(5, 3, 2, 32, 40064, 32, "bf16"), (12, 3, 2, 64, 40064, 64, "f32"), (60, 2, 1, 64, 40960, 32, "f32"),
         (3, 5, 4, 32, 300032, 32, "f16"),
         (24, 2, 1, 1120, 2080, 32, "bf16"), (40, 3, 2, 1152, 2176, 128, "f32"), (64, 3, 1, 1088, 1088, 64, "f16"),
         (14, 2, 1, 2304, 4160, 64, "bf16"), (14, 2, 1, 640, 1664, 128, "f32")]


@pytest.mark.parametrize("m,e,top,n,k,group,dtype", SIZES)
def test_groups_of_tokens_and_chunks_of_rows(qll_gpu, m, e, top, n, k, group, dtype):
    rng = np.random.default_rng(m + n)
    fmt = (m + n // 32) % 4
    wg, wu = (R.Weights(rng, n, k, group, fmt, e) for _ in range(2))
    wd = R.Weights(rng, k, n, group, fmt, e)
    x = torch.from_numpy(rng.standard_normal((m, k))).to(R.TYPES[dtype]).cuda()
    ids = np.stack([rng.permutation(e)[:top] for _ in range(m)]).astype(np.int32)
    weights = rng.uniform(0.05, 1.0, (m, top)).astype(np.float32)
    ws = empty(qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, n, top) + 64)
    ws.fill_(0xFF)
    y = torch.full((m * k + 64,), 3.25, dtype=x.dtype, device="cuda")
    qll.qll_q4g_moe(x, R.CODES[dtype], dev(ids), dev(weights), top, wg.wp, wu.wp, wd.wp, group, fmt, qll.QLL_ACT_SILU,
                    x, y, m, n, k, e, ws=ws[:-64])
    torch.cuda.synchronize()
    assert (y[m * k:] == 3.25).all() and (ws[-64:] == 0xFF).all(), "wrote past the outputs"
    E.assert_bound(R.f64(y[:m * k].view(m, k)), *moe_by_expert(R.f64(x), ids, weights, wg, wu, wd, "silu", R.f64(x), dtype),
                   "experts")


def test_workspaces_too_small(qll_gpu):
    r = Run(7, "f32", 0, vocab=70016, hidden=2048)
    need = qll.qll_workspace_bytes(qll.QLL_OP_Q4G_LINEAR, 7, 70016, 2048)
    assert need >= 7 * 2048 * 6
    layer = (qll.qll_workspace_bytes(qll.QLL_OP_MOE_ROUTE, 7, EXPERTS, CHOSEN) +
             qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, 7, FFN, CHOSEN))
    for ws in (None, r.ws[:need - 1]):
        with pytest.raises(qll.QllError, match="workspace"):
            qll.qll_q4g_linear(r.head.wp, 32, qll.QLL_Q4G_ZEROS, r.y, F32, None, 0, None, r.logits, F32, 7, 70016, 2048,
                               ws=ws)
    with pytest.raises(qll.QllError, match="workspace"):
        qll.qll_q4g_moe_layer(r.h, F32, r.wr, F32, r.bias, 0, 1, 1.0, r.ids, r.w, CHOSEN, r.wg.wp, r.wu.wp, r.wd.wp,
                              GROUP, FMT, 0, None, r.y, 7, FFN, 2048, EXPERTS, ws=r.ws[:layer - 1])
