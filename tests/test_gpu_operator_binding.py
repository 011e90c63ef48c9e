"""Refusals of the operators' Python entries on device tensors (host checks:
nothing is launched): short, strided and host tensors beside good ones, a
workspace missing or too small, and a shape the library does not take."""
import pytest
import torch

import quantized_linear_layer_amd as qll
from gpu_util import empty

pytestmark = pytest.mark.gpu


def test_short_strided_and_host_tensors(qll_gpu):
    f = torch.float32
    x, w, xq, h = empty(4 * 64, f), empty(64, f), empty(4 * 2 * 34), empty(4 * 64, f)
    good = [x, 0, None, w, 1e-5, h, xq, 4, 64]
    for at, bad, what in ((0, empty(4 * 64 - 1, f), "x holds"), (3, empty(63, f), "weight holds"),
                          (5, empty(4 * 64 - 1, f), "h holds"), (6, empty(4 * 2 * 34 - 1), "xq holds"),
                          (2, torch.zeros(4 * 64), "CUDA"), (3, empty(128, f)[::2], "contiguous")):
        a = list(good)
        a[at] = bad
        with pytest.raises(ValueError, match=what):
            qll.qll_rmsnorm_q8_0(*a)
    ids = empty(5, torch.int32)
    with pytest.raises(ValueError, match="top_logprob holds"):
        qll.qll_token_logprobs(x, 0, None, 0, None, None, 5, ids, empty(4, f), 1, 256, ws=empty(4096))


def test_workspaces_and_shapes(qll_gpu):
    f = torch.float32
    m, n, k = 65, 4100, 32
    w, xq, y = empty(n * 18), empty(m * 34), empty(m * n, f)
    need = qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, m, n, k)
    for ws in (None, empty(need - 1)):
        with pytest.raises(qll.QllError, match="workspace") as e:
            qll.qll_q4_0_q8_0_linear(w, xq, None, 0, None, y, m, n, k, ws=ws)
        assert e.value.status == -4
        with pytest.raises(qll.QllError, match="workspace"):
            qll.qll_q4_0_q8_0_gated(w, w, xq, 0, y, m, n, k, ws=ws)
    with pytest.raises(qll.QllError, match="shape"):
        qll.qll_q4_0_q8_0_linear(w, xq, None, 0, None, y, m, n, 48)
    with pytest.raises(qll.QllError, match="value"):
        qll.qll_q4_0_q8_0_linear(w, xq, None, 7, None, y, 1, n, k)
    with pytest.raises(qll.QllError, match="16-byte"):
        qll.qll_rmsnorm_q8_0(empty(68, f)[1:65], 0, None, empty(64, f), 1e-5, None, empty(2 * 34), 1, 64)
