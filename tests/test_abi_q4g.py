"""Refusals of the 4-bit group-scaled products, the router and the experts, on
the CPU: every call below has an argument that is checked on the host before any
device call; and other element types in the binding."""
import pytest
import torch

import quantized_linear_layer_amd as qll
from test_abi_operators import ALIGN, GOOD, MIS, NUL, NULL, SHAPE, SIZE_MAX, VALUE, WORKSPACE, refusals
from test_operator_types import OnDevice, taken  # noqa: F401 (a fixture)

BIG = 2 ** 40


@pytest.fixture(scope="module")
def L():
    return qll.load()


def test_sizes(L):
    P, W = qll.qll_q4g_packed_bytes, qll.qll_workspace_bytes
    # tiles of 16 x 128: codes, scales of a chunk of 512, zero points
    assert P(1, 32, 32, 0) == 1024 + 16 * 32
    for n, k, group, fmt, size in ((16, 128, 128, 0, 1024 + 16 * 8), (17, 128, 128, 0, 2 * (1024 + 16 * 8)),
                                   (16, 640, 64, 2, 5 * 1024 + 2 * 16 * (16 + 4)), (16, 512, 32, 3, 4096 + 16 * 40)):
        assert P(n, k, group, fmt) == (size + 255) // 256 * 256
    for n, k, group, fmt in ((0, 32, 32, 0), (1, 0, 32, 0), (1, 48, 32, 0), (1, 64, 128, 0), (1, 64, 16, 0),
                             (1, 64, 64, 4), (1, 64, 64, -1), (2 ** 31, 64, 64, 0), (2 ** 30, 2 ** 12, 64, 0)):
        assert P(n, k, group, fmt) == SIZE_MAX
    assert W(qll.QLL_OP_Q4G_LINEAR, 3, 5, 96) < SIZE_MAX
    for m, n, k in ((0, 5, 96), (3, 0, 96), (3, 5, 0), (3, 5, 40), (3, 5, 2 ** 24)):
        assert W(qll.QLL_OP_Q4G_LINEAR, m, n, k) == SIZE_MAX
    assert 0 < W(qll.QLL_OP_MOE_ROUTE, 1, 1, 1) < SIZE_MAX and W(qll.QLL_OP_MOE_ROUTE, 4, 1024, 32) < SIZE_MAX
    for m, e, top in ((0, 8, 2), (1, 0, 1), (1, 1025, 2), (1, 8, 0), (1, 8, 9), (1, 64, 33)):
        assert W(qll.QLL_OP_MOE_ROUTE, m, e, top) == SIZE_MAX
    assert 0 < W(qll.QLL_OP_Q4G_MOE, 1, 32, 1) < SIZE_MAX
    # groups of 64 tokens share it
    assert W(qll.QLL_OP_Q4G_MOE, 1000, 96, 4) == W(qll.QLL_OP_Q4G_MOE, 64, 96, 4)
    for m, n, top in ((0, 32, 1), (1, 0, 1), (1, 40, 1), (1, 2 ** 24, 1), (1, 32, 0), (1, 32, 33)):
        assert W(qll.QLL_OP_Q4G_MOE, m, n, top) == SIZE_MAX
    for op in (qll.QLL_OP_MOE_ROUTE, qll.QLL_OP_Q4G_MOE):
        assert W(op, 5, 32, 3) % 16 == 0  # one stands behind the other in the layer's


def test_pack(L):
    ok = [GOOD, GOOD, GOOD, 64, 2, GOOD, 8, 128, None]
    f = L.qll_q4g_pack
    for i in (0, 1, 2, 5):
        refusals(f, ok, {i: NUL}, NULL)
        refusals(f, ok, {i: MIS}, ALIGN)
    for group in (0, -32, 16, 33, 256):
        refusals(f, ok, {3: group}, VALUE)
    for fmt in (-1, 4):
        refusals(f, ok, {4: fmt}, VALUE)
    for n, k in ((0, 128), (8, 0), (8, 96), (2 ** 31, 64), (-1, 64)):
        refusals(f, ok, {6: n, 7: k}, SHAPE)
    ok = [GOOD, GOOD, 8, 96, None]
    f = L.qll_q4g_from_q4_0
    for i in (0, 1):
        refusals(f, ok, {i: NUL}, NULL)
        refusals(f, ok, {i: MIS}, ALIGN)
    for n, k in ((0, 96), (8, 0), (8, 40)):
        refusals(f, ok, {2: n, 3: k}, SHAPE)


def test_linear(L):
    ok = [GOOD, 64, 2, GOOD, 1, GOOD, 2, GOOD, GOOD, 1, 5, 70, 128, GOOD, BIG, None]
    f = L.qll_q4g_linear
    for i in (0, 3, 8):
        refusals(f, ok, {i: NUL}, NULL)
    for i in (0, 3, 5, 7, 8, 13):
        refusals(f, ok, {i: MIS}, ALIGN)
    for at, values in ((1, (0, 16, 48, 256)), (2, (-1, 4)), (4, (-1, 3)), (6, (-1, 5)), (9, (-1, 3))):
        for v in values:
            refusals(f, ok, {at: v}, VALUE)
    W = qll.qll_workspace_bytes
    for m, n, k in ((1, 2 ** 20, 4096), (4, 14336, 4096), (8, 14336, 4096), (64, 1024, 1024), (512, 64, 96)):
        assert W(qll.QLL_OP_Q4G_LINEAR, m, n, k) == 0
    for m, n, k in ((16, 4096, 14336), (512, 14336, 4096)):  # parts of k, or f32 rows as parts
        need = W(qll.QLL_OP_Q4G_LINEAR, m, n, k)
        assert need > 0
        for v in (0, 1, 2):
            refusals(f, ok, {4: v, 10: m, 11: n, 12: k, 14: need - 1}, WORKSPACE)
            refusals(f, ok, {4: v, 10: m, 11: n, 12: k, 13: NUL, 14: 0}, WORKSPACE)
    for m, n, k in ((0, 70, 128), (5, 0, 128), (5, 70, 0), (5, 70, 96), (5, 70, 2 ** 24), (2 ** 31, 70, 128),
                    (2 ** 25, 2 ** 25, 128)):
        refusals(f, ok, {10: m, 11: n, 12: k}, SHAPE)


ROUTE = [GOOD, 1, GOOD, 0, GOOD, 1, 1, 2.5, GOOD, GOOD, 4]


def route_refusals(f, ok, m, e, k, ws):
    for i in (0, 2, 8, 9, ws):
        refusals(f, ok, {i: NUL}, NULL)
    for i in (0, 2, 4, 8, 9, ws):
        refusals(f, ok, {i: MIS}, ALIGN)
    for at, values in ((1, (-1, 3)), (3, (-1, 3)), (5, (-1, 2)), (7, (float("nan"), float("inf")))):
        for v in values:
            refusals(f, ok, {at: v}, VALUE)
    for at, values in ((10, (0, -1, 17, 33)), (m, (0, -1, 2 ** 31)), (e, (0, 3, 1025)), (k, (0, 2 ** 24))):
        for v in values:
            refusals(f, ok, {at: v}, SHAPE)
    refusals(f, ok, {10: 33, e: 64}, SHAPE)


def test_route(L):
    ok = ROUTE + [3, 16, 77, GOOD, BIG, None]
    route_refusals(L.qll_moe_route, ok, 11, 12, 13, 14)
    need = qll.qll_workspace_bytes(qll.QLL_OP_MOE_ROUTE, 3, 16, 4)
    refusals(L.qll_moe_route, ok, {15: need - 1}, WORKSPACE)


def expert_refusals(f, ok, at, ws):
    """at: where wg stands."""
    for i in (0, at, at + 1, at + 2, at + 7, ws):
        refusals(f, ok, {i: NUL}, NULL)
    for i in (0, at, at + 1, at + 2, at + 6, at + 7, ws):
        refusals(f, ok, {i: MIS}, ALIGN)
    for i, values in ((1, (-1, 3)), (at + 3, (0, 16, 256)), (at + 4, (-1, 4)), (at + 5, (-1, 5))):
        for v in values:
            refusals(f, ok, {i: v}, VALUE)
    for i, values in ((at + 8, (0, 2 ** 31)), (at + 9, (0, 96, 2 ** 24)), (at + 10, (0, 96, 2 ** 24)),
                      (at + 11, (0, 3, 1025))):
        for v in values:
            refusals(f, ok, {i: v}, SHAPE)


def test_experts(L):
    ok = [GOOD, 1, GOOD, GOOD, 4, GOOD, GOOD, GOOD, 64, 2, 4, GOOD, GOOD, 3, 128, 192, 16, GOOD, BIG, None]
    f = L.qll_q4g_moe
    expert_refusals(f, ok, 5, 17)
    for i in (2, 3):
        refusals(f, ok, {i: NUL}, NULL)
        refusals(f, ok, {i: MIS}, ALIGN)
    for top in (0, 17, 33):
        refusals(f, ok, {4: top}, SHAPE)
    refusals(f, ok, {18: qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, 3, 128, 4) - 1}, WORKSPACE)


def test_layer(L):
    ok = ROUTE + [GOOD, GOOD, GOOD, 64, 2, 4, GOOD, GOOD, 3, 128, 192, 16, GOOD, BIG, None]
    f = L.qll_q4g_moe_layer
    route_refusals(f, ok, 19, 22, 21, 23)
    expert_refusals(f, ok, 11, 23)
    need = sum(qll.qll_workspace_bytes(*a) for a in ((qll.QLL_OP_MOE_ROUTE, 3, 16, 4), (qll.QLL_OP_Q4G_MOE, 3, 128, 4)))
    refusals(f, ok, {24: need - 1}, WORKSPACE)


def test_binding_refuses_host_tensors():
    t = torch.zeros(4096)
    route, experts = (t, 0, t, 0, None, 0, 0, 1.0, t, t, 1), (t, t, t, 32, 0, 0, None, t, 1, 32, 32, 2)
    for call in (lambda: qll.qll_q4g_pack(t, t, None, 32, 0, t, 1, 32), lambda: qll.qll_q4g_from_q4_0(t, t, 1, 32),
                 lambda: qll.qll_q4g_linear(t, 32, 0, t, 0, None, 0, None, t, 0, 1, 1, 32),
                 lambda: qll.qll_moe_route(*route, 1, 2, 32), lambda: qll.qll_q4g_moe(t, 0, t, t, 1, *experts),
                 lambda: qll.qll_q4g_moe_layer(*route, *experts)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


F, D, H, B, I, LONG, U = (torch.float32, torch.float64, torch.float16, torch.bfloat16, torch.int32, torch.int64,
                          torch.uint8)


def t(dtype):
    return OnDevice(dtype, 1 << 16)


TYPED = {  # entry: arguments, and by position of a typed one the types that it refuses
    "qll_q4g_pack": ([t(U), t(B), t(U), 32, 3, t(U), 8, 64], {1: (H, F)}),
    "qll_q4g_linear": ([t(U), 32, 0, t(B), 1, t(F), 0, t(H), t(H), 2, 2, 8, 64], {3: (H, F), 5: (D, B), 7: (B, F), 8: (B,)}),
    "qll_moe_route": ([t(H), 2, t(F), 0, t(F), 0, 1, 1.0, t(I), t(F), 2, 3, 4, 50],
                      {0: (B, F), 2: (D, I), 4: (D,), 8: (LONG, F), 9: (D,)}),
    "qll_q4g_moe": ([t(B), 1, t(I), t(F), 2, t(U), t(U), t(U), 32, 0, 0, t(B), t(B), 3, 32, 64, 4],
                    {0: (H, F), 2: (LONG,), 3: (D,), 11: (H,), 12: (F,)}),
    "qll_q4g_moe_layer": ([t(B), 1, t(F), 0, t(F), 0, 1, 1.0, t(I), t(F), 2, t(U), t(U), t(U), 32, 0, 0, t(B), t(B), 3,
                           32, 64, 4], {0: (H,), 2: (D,), 4: (D,), 8: (LONG,), 9: (D,), 17: (H,), 18: (F,)}),
}


@pytest.mark.parametrize("name", TYPED)
def test_other_types_are_refused(taken, name):  # noqa: F811
    args, bad = TYPED[name]
    getattr(qll, name)(*args)
    assert taken == [name]
    for at, types in bad.items():
        for dtype in types:
            a = list(args)
            a[at] = t(dtype)
            with pytest.raises(ValueError, match="is of type"):
                getattr(qll, name)(*a)
    assert taken == [name]


SHORT = {  # entry: position, bytes that are one too few, and the name of a tensor
    "qll_q4g_pack": ((0, 8 * 64 - 1, "codes"), (1, 8 * 2 * 2 - 2, "scales"), (2, 8 * 2 - 1, "zeros"), (5, 1024, "wp")),
    "qll_q4g_linear": ((0, 1024, "wp"), (3, 254, "x"), (5, 28, "bias"), (7, 30, "residual"), (8, 30, "y")),
    "qll_moe_route": ((0, 298, "x"), (2, 796, "wr"), (4, 12, "bias"), (8, 20, "ids"), (9, 20, "weights")),
    "qll_q4g_moe": ((0, 382, "x"), (2, 20, "ids"), (3, 20, "weights"), (5, 4096, "wg"), (6, 4096, "wu"), (7, 4096, "wd"),
                    (11, 382, "residual"), (12, 382, "y")),
}


@pytest.mark.parametrize("name", SHORT)
def test_short_tensors_are_refused(taken, name):  # noqa: F811
    args = TYPED[name][0]
    for at, nbytes, what in SHORT[name]:
        a = list(args)
        a[at] = t(args[at].dtype)
        a[at].nbytes = nbytes
        with pytest.raises(ValueError, match=f"{what} holds"):
            getattr(qll, name)(*a)
    assert taken == []
