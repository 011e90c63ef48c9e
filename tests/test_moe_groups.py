"""The workspace of qll_q4g_moe holds what the header says goes at once: for T of up
to 64 tokens, each with max(top, 2) f32 values a column, k = 32768 columns or, where
that is less, 2^23 / (T * max(top, 2)) of them."""
import pytest

import quantized_linear_layer_amd as qll

N = 32


def room(m, top):
    """The workspace but for the plan (its size is that of one token, which needs nothing else but h) and the
    gated products, three parts of 16 bits a choice and inner column."""
    def h(tokens):
        return (tokens * top * N * 6 + 255) // 256 * 256
    one = qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, 1, N, top) - h(1)
    return qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, N, top) - one - h(min(m, 64))


@pytest.mark.parametrize("m", [2, 3, 7, 31, 63, 64, 65, 1000])
@pytest.mark.parametrize("top", [1, 2, 3, 4, 5, 8, 31, 32])
def test_tokens_that_go_at_once(m, top):
    tokens, each = min(m, 64), 4 * max(top, 2)
    k = min(32768, 2 ** 23 // (tokens * max(top, 2)))
    assert room(m, top) // (each * k) >= tokens, "fewer tokens at once than documented"
    assert room(m, top) // (each * (k + 1)) < tokens, "more than documented"
    assert room(m, top) <= 32 << 20
