"""Weights of chosen experts whose scores are too small for f64: the ratios of
exp(logit), which both scores are there, and not 0 / 0."""
import numpy as np
import pytest
import torch

import quantized_linear_layer_amd as qll
from gpu_util import empty

pytestmark = pytest.mark.gpu


def route(logits, bias, score, renorm, top):
    """One activation of 1 a token: the router's column is the logits."""
    e = len(logits)
    wr = torch.tensor(logits, dtype=torch.float32, device="cuda").view(e, 1)
    b = None if bias is None else torch.tensor(bias, dtype=torch.float32, device="cuda")
    m = 3
    ids, w = empty(m * top, torch.int32), empty(m * top, torch.float32)
    qll.qll_moe_route(torch.ones(m, 1, device="cuda"), 0, wr, 0, b, score, renorm, 2.0, ids, w, top, m, e, 1,
                      ws=empty(qll.qll_workspace_bytes(qll.QLL_OP_MOE_ROUTE, m, e, top)))
    torch.cuda.synchronize()
    ids, w = ids.view(m, top), w.view(m, top)
    assert torch.equal(ids, ids[:1].expand(m, top)) and torch.equal(w, w[:1].expand(m, top))
    return ids[0].tolist(), w[0].double().cpu().numpy()


def check(w, logits):
    l = np.asarray(logits, np.float64)
    want = np.exp(l - l.max())
    want *= 2.0 / want.sum()
    assert np.all(np.abs(w - want) <= 2.0 ** -23 * want)


@pytest.mark.parametrize("base", [-600.0, -640.0, -720.0, -750.0, -800.0, -1e30])
def test_sigmoid(qll_gpu, base):
    logits = [base - 1.0, base, base - 4.0, base - 0.5, base - 9.0] if base > -1e4 else [2 * base, base, 3 * base, base, 4 * base]
    ids, w = route(logits, None, qll.QLL_SCORE_SIGMOID, 1, 3)
    assert ids == [1, 3, 0]
    check(w, [np.float32(logits[i]) for i in ids])
    ids, w = route(logits, None, qll.QLL_SCORE_SIGMOID, 0, 3)
    assert np.all(w == 0.0)


@pytest.mark.parametrize("base", [-600.0, -700.0, -740.0, -1000.0])
def test_softmax_and_a_bias_that_moves_the_choice(qll_gpu, base):
    logits = [0.0, base, base - 2.0, 1.0, base - 0.25]
    ids, w = route(logits, [0.0, 3.0, 4.0, 0.0, 2.0], qll.QLL_SCORE_SOFTMAX, 1, 3)
    assert ids == [2, 1, 4]
    check(w, [np.float32(logits[i]) for i in ids])
