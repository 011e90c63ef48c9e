"""qll_q4g_pack takes codes and zero points one a byte: wider elements have bytes
enough, and would be read as other codes.  On the CPU, the library's call replaced."""
import pytest
import torch

import quantized_linear_layer_amd as qll
from test_operator_types import OnDevice, taken  # noqa: F401 (a fixture)

WIDER = (torch.int16, torch.int32, torch.int64, torch.float32, torch.float16, torch.bool)


def pack(codes, zeros, fmt):
    t = OnDevice(torch.uint8, 1 << 16)
    qll.qll_q4g_pack(OnDevice(codes, 1 << 16), OnDevice(torch.float16, 1 << 16), OnDevice(zeros, 1 << 16), 64, fmt, t, 8, 128)


@pytest.mark.parametrize("own", [torch.uint8, torch.int8])
def test_wider_codes_and_zero_points_are_refused(taken, own):  # noqa: F811
    pack(own, own, qll.QLL_Q4G_ZEROS)
    pack(own, torch.int32, 0)  # without zero points that argument is unused
    assert taken == ["qll_q4g_pack"] * 2
    for other in WIDER:
        with pytest.raises(ValueError, match="codes is of type"):
            pack(other, own, qll.QLL_Q4G_ZEROS)
        with pytest.raises(ValueError, match="zeros is of type"):
            pack(own, other, qll.QLL_Q4G_ZEROS)
    assert taken == ["qll_q4g_pack"] * 2
