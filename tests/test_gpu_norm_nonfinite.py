"""NaN and infinities that stand alone among zero products in rows of the norms
into activations, against what the header promises of such rows."""
import numpy as np
import pytest
import torch

from test_gpu_norm import DTYPES, call, definition, stream_rows

pytestmark = pytest.mark.gpu

# a wave per row (one or four pieces), 1024 and 256 threads, eight pieces a thread, two sweeps
SHAPES = [(7, 32), (9, 64), (7, 1024), (7, 4096), (260, 4096), (260, 8192), (258, 16384), (7, 16416)]


def lone_values(m, k, dtype):
    """(x, res, w, rows that hold a NaN or an infinity): the value's block, or the
    whole row, has no other product but zeros."""
    x, r, w = stream_rows(m + k, m, k, dtype)
    x[0], r[0] = 0.0, 0.0
    x[0, k - 3] = float("nan")      # a row of zeros with one NaN
    x[1], r[1] = 0.0, 0.0
    r[1, 5] = float("nan")          # the same in the residual
    x[2, :32], r[2, :32] = 0.0, 0.0
    x[2, 9] = float("nan")          # a block of zeros with one NaN
    w[:32] = 0.0
    x[3, 4] = float("inf")          # an infinity times a weight of zero
    x[4], r[4] = 0.0, 0.0
    r[4, 31] = -float("inf")        # nothing but that
    x[5], r[5] = 0.0, 0.0           # a padded row: zeros
    return x, r, w, [0, 1, 2, 3, 4]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_q8_0_scales_show_a_lone_nan_or_infinity(qll_gpu, m, k, dtype, eps):
    x, r, w, bad = lone_values(m, k, dtype)
    good = [i for i in range(m) if i not in bad]
    for h in ("new", None):
        _, codes, scale, _ = call("q8_0", x, r, w, eps, h)
        with np.errstate(invalid="ignore"):
            _, want, d, _ = definition(x, r, w, eps, True)
        assert np.isnan(scale[bad]).all(), f"finite scales in rows {np.argwhere(~np.isnan(scale[bad]))[:4].tolist()}"
        assert np.array_equal(codes[good], want[good]) and np.array_equal(scale[good], d[good])
        assert (codes[5] == 0).all() and (scale[5] == 0).all()


@pytest.mark.parametrize("m,k", [(3, 60), (3, 63), (3, 1000), (3, 1001), (3, 4096), (260, 4096), (3, 16381),
                                 (258, 16384), (3, 16387), (3, 20000)])
@pytest.mark.parametrize("where", ["x", "x alone", "residual"])
def test_i8_rows_with_nan_of_any_bits_are_zero(qll_gpu, m, k, where):
    x, r, w = stream_rows(m + k, m, k, torch.float32)
    bits = torch.tensor([0x7fffffff, -1, 0x7fc00007], dtype=torch.int32)  # 0xff bytes among them
    at = [3, k // 2, k - 1]
    (r if where == "residual" else x)[0, at] = bits.view(torch.float32)
    (r if where == "residual" else x)[1] = bits[1:2].view(torch.float32)  # a row filled with 0xff
    res = None if where == "x alone" else r
    for h in ("new", None):
        _, codes, scale, total = call("i8", x, res, w, 1e-5, h)
        _, want, s, t = definition(x[2:], None if res is None else res[2:], w, 1e-5, False)
        assert (codes[:2] == 0).all() and (scale[:2] == 0).all()
        assert (total[:2] == 0).all(), f"code sums {total[:2]}"
        assert np.array_equal(codes[2:], want) and np.array_equal(scale[2:], s) and np.array_equal(total[2:], t)
