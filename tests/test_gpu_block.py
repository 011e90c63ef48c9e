"""The operators in the order a transformer uses them: residual sum and norm
into Q8_0, gated projection, quantization, down projection added to the
stream, norm again, vocabulary projection, log probabilities; and the BitNet
entry (norm into int8 rows, ternary linear).  Each step is checked against the
64-bit form of what it was given, and the whole run is captured into a HIP
graph and replayed on changed inputs, with eager work and synchronisations
between the replays."""
import numpy as np
import pytest
import torch

import epilogue_refs as E
import logprob_refs as R
import oracle as O
import quantized_linear_layer_amd as qll
import synth
from gpu_util import dev, empty, pack_q4_0, pack_ternary
from test_gpu_norm import definition

pytestmark = pytest.mark.gpu

HIDDEN, FFN, VOCAB, TOP = 256, 544, 1003, 5


class Model:
    """Weights, buffers and workspaces of the run for m rows."""

    def __init__(self, m, repacked, seed=0):
        rng = np.random.default_rng(seed)
        self.m, self.repacked = m, repacked
        self.raw = {k: synth.q4_0_weights(rng, n, kk) for k, (n, kk) in
                    {"gate": (FFN, HIDDEN), "up": (FFN, HIDDEN), "down": (HIDDEN, FFN), "head": (VOCAB, HIDDEN)}.items()}
        self.w = {k: pack_q4_0(*r) for k, r in self.raw.items()}
        self.norm = [dev(synth.uniform_f32(rng, (HIDDEN,), 0.5, 1.5)) for _ in range(2)]
        self.bias = dev(synth.normal_f32(rng, (VOCAB,)))
        if repacked:
            self.pair = empty(qll.qll_q4_0_repacked_gated_bytes(FFN, HIDDEN))
            qll.qll_q4_0_repack_gated(self.w["gate"], self.w["up"], self.pair, FFN, HIDDEN)
            self.down = empty(qll.qll_q4_0_repacked_bytes(HIDDEN, FFN))
            qll.qll_q4_0_repack(self.w["down"], self.down, HIDDEN, FFN)
        f = torch.float32
        self.x, self.delta = empty(m * HIDDEN, f), empty(m * HIDDEN, f)
        self.tokens = empty(m, torch.int32)
        self.h, self.h2 = empty(m * HIDDEN, f), empty(m * HIDDEN, f)
        self.a1, self.a3 = empty(m * HIDDEN // 32 * 34), empty(m * HIDDEN // 32 * 34)
        self.a2, self.f = empty(m * FFN // 32 * 34), empty(m * FFN, f)
        self.logits = empty(m * VOCAB, f)
        self.lp, self.en = empty(m, f), empty(m, f)
        self.ids, self.tl = empty(m * TOP, torch.int32), empty(m * TOP, f)
        gated = qll.QLL_OP_Q4_0_REPACKED_GATED if repacked else qll.QLL_OP_Q4_0_GATED
        lin = qll.QLL_OP_Q4_0_REPACKED_GEMM if repacked else qll.QLL_OP_Q4_0_LINEAR
        self.ws = empty(max(16, qll.qll_workspace_bytes(gated, m, FFN, HIDDEN),
                            qll.qll_workspace_bytes(lin, m, HIDDEN, FFN),
                            qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, m, VOCAB, HIDDEN),
                            qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, m, VOCAB, TOP)))

    def feed(self, seed):
        rng = np.random.default_rng(seed)
        self.x.copy_(dev(synth.normal_f32(rng, (self.m * HIDDEN,))))
        self.delta.copy_(dev(synth.normal_f32(rng, (self.m * HIDDEN,))))
        self.tokens.copy_(dev(rng.integers(0, VOCAB, self.m).astype(np.int32)))

    def run(self):
        m, ws = self.m, self.ws
        qll.qll_rmsnorm_q8_0(self.x, qll.QLL_DTYPE_F32, self.delta, self.norm[0], 1e-5, self.h, self.a1, m, HIDDEN)
        if self.repacked:
            qll.qll_q4_0_repacked_q8_0_gated(self.pair, self.a1, qll.QLL_ACT_SILU, self.f, m, FFN, HIDDEN, ws=ws)
        else:
            qll.qll_q4_0_q8_0_gated(self.w["gate"], self.w["up"], self.a1, qll.QLL_ACT_SILU, self.f, m, FFN, HIDDEN,
                                    ws=ws)
        qll.qll_quantize_q8_0(self.f, self.a2, m, FFN)
        lin = qll.qll_q4_0_repacked_q8_0_linear if self.repacked else qll.qll_q4_0_q8_0_linear
        lin(self.down if self.repacked else self.w["down"], self.a2, None, qll.QLL_ACT_NONE, self.h, self.h2, m,
            HIDDEN, FFN, ws=ws)
        qll.qll_rmsnorm_q8_0(self.h2, qll.QLL_DTYPE_F32, None, self.norm[1], 1e-5, None, self.a3, m, HIDDEN)
        qll.qll_q4_0_q8_0_linear(self.w["head"], self.a3, self.bias, qll.QLL_ACT_NONE, None, self.logits, m, VOCAB,
                                 HIDDEN, ws=ws)
        qll.qll_token_logprobs(self.logits, qll.QLL_DTYPE_F32, self.tokens, 1, self.lp, self.en, TOP, self.ids,
                               self.tl, m, VOCAB, ws=ws)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.cpu().numpy().copy() for t in (self.h, self.a1, self.f, self.a2, self.h2, self.a3, self.logits,
                                                 self.lp, self.en, self.ids, self.tl)]


def check_norm(x, res, w, h, xq, m):
    want = definition(x.view(m, HIDDEN).cpu(), None if res is None else res.view(m, HIDDEN).cpu(), w.cpu(), 1e-5, True)
    b = xq.reshape(m, HIDDEN // 32, 34)
    if h is not None:
        assert np.array_equal(h.reshape(m, HIDDEN), want[0].numpy())
    assert np.array_equal(b[..., 2:].copy().view(np.int8).reshape(m, HIDDEN), want[1])
    assert np.array_equal(b[..., :2].copy().view(np.float16)[..., 0], want[2])


@pytest.mark.parametrize("repacked", [False, True])
@pytest.mark.parametrize("m", [1, 5, 80])
def test_run(qll_gpu, m, repacked):
    M = Model(m, repacked)
    M.feed(1)
    M.run()
    h, a1, f, a2, h2, a3, logits, lp, en, ids, tl = M.outputs()
    check_norm(M.x, M.delta, M.norm[0], h, a1, m)
    (g, eg), (u, eu) = (E.product(*M.raw[k], a1.reshape(m, -1), m) for k in ("gate", "up"))
    E.assert_bound(f, *E.gated(g, eg, u, eu, "silu"), "gated")
    assert np.array_equal(a2, O.quantize_q8_0(f.reshape(m, FFN)).reshape(-1))
    v, ev = E.product(*M.raw["down"], a2.reshape(m, -1), m)
    E.assert_bound(h2, *E.linear(v, ev, None, "none", h.reshape(m, HIDDEN)), "down")
    check_norm(M.h2, None, M.norm[1], None, a3, m)
    v, ev = E.product(*M.raw["head"], a3.reshape(m, -1), m)
    E.assert_bound(logits, *E.linear(v, ev, M.bias.cpu().numpy(), "none", None), "logits")
    want = R.reference(logits.reshape(m, VOCAB), M.tokens.cpu().numpy().reshape(m, 1), TOP)
    assert np.array_equal(ids.reshape(m, TOP), want[2])
    R.assert_close(lp.reshape(m, 1), want[0], want[4], "given")
    R.assert_close(tl.reshape(m, TOP), want[3], want[4], "chosen")
    R.assert_close(en, want[1], want[5], "entropy")


@pytest.mark.parametrize("repacked", [False, True])
@pytest.mark.parametrize("m", [1, 80])
def test_captured_and_replayed(qll_gpu, m, repacked):
    """Two graphs with workspaces of their own, replayed in turn."""
    models = [Model(m, repacked, seed) for seed in (1, 2)]
    graphs = []
    for i, M in enumerate(models):
        M.feed(i)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            M.run()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.run()
        graphs.append(g)
    for seed in range(10, 14):
        for M in models:
            M.feed(seed)
        for g in graphs:
            g.replay()
        got = [M.outputs() for M in models]
        for M, outs in zip(models, got):
            M.run()
            for a, b in zip(outs, M.outputs()):
                assert np.array_equal(a.view(np.uint8), b.view(np.uint8))


def test_bitnet_entry(qll_gpu):
    m, n, k = 5, 96, 320
    rng = np.random.default_rng(3)
    codes = synth.ternary_codes(rng, n, k)
    x = dev(synth.normal_f32(rng, (m, k))).bfloat16()
    r = dev(synth.normal_f32(rng, (m, k))).bfloat16()
    w = dev(synth.uniform_f32(rng, (k,), 0.5, 1.5))
    h, q = torch.empty_like(x), empty(m * k, torch.int8)
    s, t = empty(m, torch.float32), empty(m, torch.int32)
    qll.qll_rmsnorm_i8_rows(x, qll.QLL_DTYPE_BF16, r, w, 1e-5, h, q, s, t, m, k)
    y = empty(m * n, torch.float32)
    qll.qll_ternary_gemm(pack_ternary(codes), 0.05, q, s, t, y, m, n, k)
    torch.cuda.synchronize()
    want = definition(x.cpu(), r.cpu(), w.cpu(), 1e-5, False)
    assert np.array_equal(q.cpu().numpy().reshape(m, k), want[1]) and np.array_equal(s.cpu().numpy(), want[2])
    assert np.array_equal(t.cpu().numpy(), want[3])
    y_ref, mag = O.ternary(O.pack_ternary(codes), np.float32(0.05), want[1].astype(np.int8), want[2],
                           want[3].astype(np.int32), n, k)
    # one product and one division: two roundings of the exact integer dot
    assert (np.abs(y.cpu().numpy().reshape(m, n) - y_ref) <= 4 * E.U * np.abs(y_ref)).all()
