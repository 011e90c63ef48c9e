"""Packing writes every byte of the packed form, those behind its regions too: two
packings of the same weights into different bytes are alike, and nothing behind
them changes."""
import numpy as np
import pytest
import torch

import quantized_linear_layer_amd as qll
import synth
from gpu_util import pack_q4_0

pytestmark = pytest.mark.gpu


def twice(size, pack):
    a, b = (torch.full((size + 256,), v, dtype=torch.uint8, device="cuda") for v in (0xA5, 0x5A))
    for t in (a, b):
        pack(t[:size])
    torch.cuda.synchronize()
    assert torch.equal(a[:size], b[:size])
    assert (a[size:] == 0xA5).all() and (b[size:] == 0x5A).all()
    return a[:size]


# (n, k / group): one tile, row tiles and pieces of 512 in odd numbers, where groups of 128 leave bytes behind the
# regions (128 of 256 without zero points; 96 to 224 with)
@pytest.mark.parametrize("fmt", [0, qll.QLL_Q4G_BF16, qll.QLL_Q4G_ZEROS, qll.QLL_Q4G_BF16 | qll.QLL_Q4G_ZEROS])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,groups", [(1, 1), (16, 1), (17, 5), (40, 3), (33, 13), (300, 9)])
def test_every_byte_is_written(qll_gpu, n, groups, group, fmt):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + group)
    k = groups * group
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    zeros = torch.randint(0, 16, (n, groups), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(n, groups, generator=g, device="cuda").to(torch.bfloat16 if fmt & qll.QLL_Q4G_BF16 else torch.float16)
    size = qll.qll_q4g_packed_bytes(n, k, group, fmt)
    packed = twice(size, lambda t: qll.qll_q4g_pack(codes, scales, zeros, group, fmt, t, n, k))
    tiles, pieces = (n + 15) // 16 * ((k + 127) // 128), (n + 15) // 16 * ((k + 511) // 512)
    end = 1024 * tiles + pieces * 16 * (1024 // group + (256 // group if fmt & qll.QLL_Q4G_ZEROS else 0))
    assert end <= size < end + 256 and (packed[end:] == 0).all()


@pytest.mark.parametrize("n,k", [(1, 32), (40, 96), (33, 1440)])
def test_every_byte_is_written_from_q4_0(qll_gpu, n, k):
    codes, d_bits = synth.q4_0_weights(np.random.default_rng(n), n, k)
    w = pack_q4_0(codes, d_bits)
    twice(qll.qll_q4g_packed_bytes(n, k, 32, 0), lambda t: qll.qll_q4g_from_q4_0(w, t, n, k))
