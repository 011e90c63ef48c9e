"""Refusals of the operators around the linear layers, on the CPU: every call
below has an argument that is checked on the host before any device call."""
import ctypes

import pytest

import quantized_linear_layer_amd as qll

NULL, SHAPE, ALIGN, WORKSPACE, VALUE = -1, -2, -3, -4, -8
SIZE_MAX = 2 ** 64 - 1
GOOD, MIS, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None


@pytest.fixture(scope="module")
def L():
    return qll.load()


def test_status_of_values(L):
    assert "value" in qll.qll_status_string(VALUE)


def test_norm_q8_0(L):
    f = L.qll_rmsnorm_q8_0
    ok = [GOOD, 0, GOOD, GOOD, 1e-5, GOOD, GOOD, 4, 64, None]

    def rc(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 3, 6):
        assert rc(**{f"a{i}": NUL}) == NULL
    for i in (0, 2, 3, 5, 6):
        assert rc(**{f"a{i}": MIS}) == ALIGN
    for dtype in (-1, 3):
        assert rc(a1=dtype) == VALUE
    for eps in (-1e-5, float("nan"), float("inf")):
        assert rc(a4=eps) == VALUE
    for m, k in ((0, 64), (-1, 64), (4, 0), (4, 48), (4, 1), (4, 2 ** 24), (2 ** 31, 64)):
        assert rc(a7=m, a8=k) == SHAPE


def test_norm_i8_rows(L):
    f = L.qll_rmsnorm_i8_rows
    ok = [GOOD, 0, GOOD, GOOD, 1e-5, GOOD, GOOD, GOOD, GOOD, 4, 63, None]

    def rc(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 3, 6, 7, 8):
        assert rc(**{f"a{i}": NUL}) == NULL
    for i in (0, 2, 3, 5, 6, 7, 8):
        assert rc(**{f"a{i}": MIS}) == ALIGN
    assert rc(a1=7) == VALUE and rc(a4=-0.5) == VALUE
    for m, k in ((0, 64), (4, 0), (4, 2 ** 24), (2 ** 31, 63)):
        assert rc(a9=m, a10=k) == SHAPE


def test_binding_refuses_host_and_short_tensors():
    import torch
    x = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        qll.qll_rmsnorm_q8_0(x, 0, None, x, 1e-5, None, x, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        qll.qll_rmsnorm_i8_rows(x, 0, None, x, 1e-5, None, x, x, x, 1, 64)


def refusals(f, ok, at, expect):
    """f with the arguments `at` (index: value) of `ok` replaced returns expect."""
    a = list(ok)
    for i, v in at.items():
        a[i] = v
    assert f(*a) == expect, at


def test_linear(L):
    big = 2 ** 40
    ok = [GOOD, GOOD, GOOD, 2, GOOD, GOOD, 512, 8192, 1024, GOOD, big, None]  # large enough for the 128-row GEMM
    for f, ws_null in ((L.qll_q4_0_q8_0_linear, WORKSPACE), (L.qll_q4_0_repacked_q8_0_linear, NULL)):
        for i in (0, 1, 5):
            refusals(f, ok, {i: NUL}, NULL)
        for i in (0, 1, 2, 4, 5, 9):
            refusals(f, ok, {i: MIS}, ALIGN)
        for act in (-1, 5):
            refusals(f, ok, {3: act}, VALUE)
        for m, n, k in ((0, 8, 256), (100, 0, 256), (100, 8, 0), (100, 8, 48), (100, 8, 2 ** 24), (2 ** 31, 8, 256)):
            refusals(f, ok, {6: m, 7: n, 8: k}, SHAPE)
        refusals(f, ok, {9: NUL, 10: 0}, ws_null)
        refusals(f, ok, {10: 16}, WORKSPACE)
    # one row: the GEMV's limit on k
    refusals(L.qll_q4_0_q8_0_linear, ok, {6: 1, 8: 49152 + 32}, SHAPE)
    for m, n, k in ((1, 4096, 4096), (64, 4096, 4096), (512, 8192, 1024), (512, 4096, 14336)):
        assert qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, m, n, k) == \
            qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_Q8_0_GEMM, m, n, k)
    assert qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, 2, 8, 40) == SIZE_MAX
    for m, n, k in ((65, 257, 1024), (4096, 20, 256), (16, 2 ** 20, 96), (512, 512, 64), (191, 4096, 4096)):
        assert qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, m, n, k) == 0
    for m, n, k in ((4097, 20, 256), (192, 4096, 4096), (65, 32768, 256), (65, 32767, 256), (513, 512, 64), (2 ** 31 - 1, 2, 2 ** 23)):
        assert 0 < qll.qll_workspace_bytes(qll.QLL_OP_Q4_0_LINEAR, m, n, k)


def test_gated(L):
    big = 2 ** 40
    ok = [GOOD, GOOD, GOOD, 4, GOOD, 512, 8192, 1024, GOOD, big, None]
    f = L.qll_q4_0_q8_0_gated
    for i in (0, 1, 2, 4):
        refusals(f, ok, {i: NUL}, NULL)
    for i in (0, 1, 2, 4, 8):
        refusals(f, ok, {i: MIS}, ALIGN)
    for act in (-1, 5):
        refusals(f, ok, {3: act}, VALUE)
    for m, n, k in ((0, 8, 256), (100, -1, 256), (100, 8, 33), (100, 8, 2 ** 24), (1, 8, 2 ** 24)):
        refusals(f, ok, {5: m, 6: n, 7: k}, SHAPE)
    refusals(f, ok, {8: NUL, 9: 0}, WORKSPACE)
    refusals(f, ok, {5: 2, 7: 224, 8: NUL, 9: 0}, WORKSPACE)  # rows under eight blocks take the GEMM
    refusals(f, ok, {9: 16}, WORKSPACE)
    ok = [GOOD, GOOD, 4, GOOD, 100, 8, 256, GOOD, big, None]
    f = L.qll_q4_0_repacked_q8_0_gated
    for i in (0, 1, 3, 7):
        refusals(f, ok, {i: NUL}, NULL)
    for i in (0, 1, 3, 7):
        refusals(f, ok, {i: MIS}, ALIGN)
    refusals(f, ok, {2: 9}, VALUE)
    refusals(f, ok, {6: 2 ** 24}, SHAPE)
    refusals(f, ok, {8: 255}, WORKSPACE)
    ok = [GOOD, GOOD, GOOD, 8, 64, None]
    f = L.qll_q4_0_repack_gated
    for i in range(3):
        refusals(f, ok, {i: NUL}, NULL)
        refusals(f, ok, {i: MIS}, ALIGN)
    for n, k in ((0, 64), (8, 40)):
        refusals(f, ok, {3: n, 4: k}, SHAPE)
    W = qll.qll_workspace_bytes
    for m, n, k in ((1, 14336, 4096), (1, 64, 32), (1, 64, 65536), (64, 14336, 4096), (2, 7, 256)):
        assert W(qll.QLL_OP_Q4_0_GATED, m, n, k) == 0
    for m, n, k in ((2, 7, 224), (65, 14336, 4096)):
        assert 0 < W(qll.QLL_OP_Q4_0_GATED, m, n, k) < SIZE_MAX
    assert W(qll.QLL_OP_Q4_0_REPACKED_GATED, 1, 1, 32) > 0
    for op in (qll.QLL_OP_Q4_0_GATED, qll.QLL_OP_Q4_0_REPACKED_GATED):
        assert W(op, 2, 7, 40) == SIZE_MAX and W(op, 2, 7, 2 ** 24) == SIZE_MAX
    assert qll.qll_q4_0_repacked_gated_bytes(1, 32) == 3328
    assert qll.qll_q4_0_repacked_gated_bytes(65, 64) == 2 * 2 * 3328
    assert qll.qll_q4_0_repacked_gated_bytes(8, 48) == SIZE_MAX


def test_logprobs(L):
    big = 2 ** 40
    ok = [GOOD, 0, GOOD, 2, GOOD, GOOD, 5, GOOD, GOOD, 3, 1000, GOOD, big, None]
    f = L.qll_token_logprobs
    for i in (0, 2, 4, 7, 8, 11):
        refusals(f, ok, {i: NUL}, NULL)
    for i in (0, 2, 4, 5, 7, 8, 11):
        refusals(f, ok, {i: MIS}, ALIGN)
    for dtype in (-1, 3):
        refusals(f, ok, {1: dtype}, VALUE)
    for t, top, m, v in ((-1, 5, 3, 1000), (2, -1, 3, 1000), (2, 65, 3, 1000), (2, 5, 0, 1000), (2, 5, 3, 0),
                         (2, 5, 3, 4), (2, 5, 3, 2 ** 20 + 1), (2 ** 31, 5, 3, 1000), (2, 5, 2 ** 31, 1000)):
        refusals(f, ok, {3: t, 6: top, 9: m, 10: v}, SHAPE)
    refusals(f, ok, {12: qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, 3, 1000, 5) - 1}, WORKSPACE)
    refusals(f, ok, {3: 0, 2: NUL, 4: NUL, 6: 0, 7: NUL, 8: NUL, 12: 0}, WORKSPACE)  # the parts left out are not asked for
    W = qll.qll_workspace_bytes
    assert W(qll.QLL_OP_TOKEN_LOGPROBS, 1, 1, 0) > 0
    assert W(qll.QLL_OP_TOKEN_LOGPROBS, 1, 2 ** 20, 64) < SIZE_MAX
    for m, v, top in ((0, 10, 1), (1, 0, 0), (1, 10, 11), (1, 100, 65), (1, 2 ** 20 + 1, 1), (1, 10, -1)):
        assert W(qll.QLL_OP_TOKEN_LOGPROBS, m, v, top) == SIZE_MAX


def test_binding_refuses_host_tensors_of_every_operator():
    import torch
    t = torch.zeros(4096)
    for call in (lambda: qll.qll_q4_0_q8_0_linear(t, t, None, 0, None, t, 1, 8, 32),
                 lambda: qll.qll_q4_0_repacked_q8_0_linear(t, t, None, 0, None, t, 1, 8, 32),
                 lambda: qll.qll_q4_0_q8_0_gated(t, t, t, 0, t, 1, 8, 32),
                 lambda: qll.qll_q4_0_repack_gated(t, t, t, 8, 32),
                 lambda: qll.qll_q4_0_repacked_q8_0_gated(t, t, 0, t, 1, 8, 32),
                 lambda: qll.qll_token_logprobs(t, 0, None, 0, None, t, 0, None, None, 1, 8)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
