"""4-bit weights with group scales: every bit of an activation counts, a weight
of zero takes nothing from the others, and the largest activations the header
allows stay in range, on every kernel the linear layer and the experts dispatch
to.

Where a row has one value whose weight is not zero, that weight and its scale
are powers of two: every partial sum is the value's upper bits or all of them,
times a power of two, so the result is exact and is compared for equality.

Random rows: an output adds at most R = 3 k + k / g + 12 products, group sums and
partial sums (f32 activations count as three parts), each rounding off at most u
= 2^-24 of a partial sum, whose root mean square over random signs is at
most q = sqrt(sum t^2) of the terms t.  Independent roundings then add up to at
most u sqrt(R) q in the root mean square over outputs."""
import numpy as np
import pytest
import torch

import q4g_refs as R
import quantized_linear_layer_amd as qll
from gpu_util import empty

pytestmark = pytest.mark.gpu
BF16, ZEROS = qll.QLL_Q4G_BF16, qll.QLL_Q4G_ZEROS
LIMIT = 2.0 ** 117  # |x| below it

# (type, m, n, k): each wave with its own rows, one to many of them; then rows in LDS, 8, 16, 32 and 64 at once
# (8 and 16 of f32)
PATHS = [(t, m, 40, 1024) for t in ("f32", "bf16", "f16") for m in (1, 3, 6, 12, 40)] + [
    ("bf16", 8, 32800, 8192), ("f16", 12, 4128, 8192), ("bf16", 12, 4128, 8192), ("bf16", 32, 6200, 8192),
    ("f16", 512, 520, 8192), ("bf16", 512, 520, 8192), ("f32", 8, 16400, 8192), ("f32", 12, 4128, 8192),
    ("f32", 512, 520, 8192)]


class Drawn:
    """Codes, zero points and scales on the device, for a test to change before they are packed."""

    def __init__(self, n, k, group, fmt, seed, count=1):
        self.n, self.k, self.group, self.fmt, self.count = n, k, group, fmt, count
        g = self.g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        shape = (count, n, k // group)
        self.codes = torch.randint(0, 16, (count, n, k), generator=g, device="cuda", dtype=torch.uint8)
        self.zeros = (torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8) if fmt & ZEROS
                      else torch.full(shape, 8, device="cuda", dtype=torch.uint8))
        power = torch.randint(-7, 0, shape, generator=g, device="cuda")
        self.scales = torch.ldexp(torch.ones(shape, device="cuda"), power).to(torch.bfloat16 if fmt & BF16 else torch.float16)

    def set_difference(self, at, d):
        """c - z = d[.., n] in column at, or -d where that is no code."""
        z = self.zeros[:, :, at // self.group].int()
        c = z + d
        self.codes[:, :, at] = torch.where((c < 0) | (c > 15), z - d, c).to(torch.uint8)

    def column(self, at):
        """s * (c - z) of column at, [count, n], in 64 bits."""
        g = at // self.group
        return self.scales[:, :, g].double() * (self.codes[:, :, at].double() - self.zeros[:, :, g].double())

    def packed(self):
        size = qll.qll_q4g_packed_bytes(self.n, self.k, self.group, self.fmt)
        wp = empty(self.count * size)
        for i in range(self.count):
            qll.qll_q4g_pack(self.codes[i], self.scales[i], self.zeros[i], self.group, self.fmt,
                             wp[i * size:(i + 1) * size], self.n, self.k)
        return wp


def linear(w, x, dtype, wp=None):
    m = x.shape[0]
    y = torch.empty(m, w.n, device="cuda")
    need = qll.qll_workspace_bytes(qll.QLL_OP_Q4G_LINEAR, m, w.n, w.k)
    qll.qll_q4g_linear(w.packed() if wp is None else wp, w.group, w.fmt, x, R.CODES[dtype], None, 0, None, y, 0, m, w.n,
                       w.k, ws=empty(need) if need else None)
    torch.cuda.synchronize()
    return y


def full(dtype, shape, g):
    """Values in (-2, -1] and [1, 2) with all bits of the type's significand, the lowest one set."""
    bits = {"f32": 23, "bf16": 7, "f16": 10}[dtype]
    low = torch.randint(0, 1 << bits, shape, generator=g, device="cuda") | 1
    sign = torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1
    return (sign.double() * (1.0 + low.double() / (1 << bits))).to(R.TYPES[dtype])


def pairs(k, group):
    """(signal, outlier) columns of one group: neighbours, in other steps of 32, at the ends of k."""
    out = [(1, 0), (group - 1, 2), (k - 1, k - group), (k - 30, k - 5)]
    for base in (128, 512, k // 2):
        out += [(base + 3, base + group - 1), (base + group // 2 + 9, base)]
    return out


def place(w, g):
    """Weights of a power of two in the signal columns, of zero in the outliers'."""
    for signal, outlier in pairs(w.k, w.group):
        shape = (w.count, w.n)
        d = 1 << torch.randint(0, 3, shape, generator=g, device="cuda")
        w.set_difference(signal, d * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1))
        w.set_difference(outlier, torch.zeros(shape, device="cuda", dtype=torch.int64))


@pytest.mark.parametrize("group,fmt", [(32, ZEROS), (64, BF16 | ZEROS), (128, ZEROS), (128, 0)])
@pytest.mark.parametrize("dtype,m,n,k", PATHS)
def test_every_bit_beside_an_outlier(qll_gpu, dtype, m, n, k, group, fmt):
    w = Drawn(n, k, group, fmt, m + n + group)
    place(w, w.g)
    columns = pairs(k, group)
    value, large = full(dtype, (m,), w.g), full(dtype, (m,), w.g)
    large = large * (16384.0 if dtype == "f16" else 2.0 ** 30)
    wp = w.packed()
    for first in range(0, len(columns), m):  # every pair is some row's
        x = torch.zeros(m, k, dtype=R.TYPES[dtype], device="cuda")
        want = torch.empty(m, n, device="cuda", dtype=torch.float64)
        for i in range(m):
            signal, outlier = columns[(first + i) % len(columns)]
            x[i, signal], x[i, outlier] = value[i], large[i]
            want[i] = w.column(signal)[0] * value[i].double()
        assert torch.equal(linear(w, x, dtype, wp).double(), want)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,m,n,k", [p for p in PATHS if p[0] != "f16"])
def test_the_largest_activations(qll_gpu, dtype, m, n, k, group):
    """Rows of one sign just under the limit: on weights of zero the result is 0, on
    the largest differences within the f32 sums' bound, 3 g + k / g + 12 roundings."""
    w = Drawn(n, k, group, ZEROS, m + group)
    w.scales.fill_(2.0 ** -14)
    top = LIMIT * (1 - 2.0 ** -8)
    x = torch.full((m, k), top, dtype=R.TYPES[dtype], device="cuda")
    x[m // 2:] = -top  # the only row where there is one
    for code, zero in ((8, 8), (15, 15), (15, 0), (0, 15)):
        w.codes.fill_(code)
        w.zeros.fill_(zero)
        y, want = linear(w, x, dtype), (code - zero) * 2.0 ** -14 * k * x[:, :1].double()
        assert torch.all((y.double() - want).abs() <= (3 * group + k // group + 12) * R.U * want.abs()), (code, zero)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype,m,n,k", [p for p in PATHS if p[2] <= 4128])
def test_outliers_on_weights_of_zero(qll_gpu, dtype, m, n, k, group):
    w = Drawn(n, k, group, ZEROS, m + n)
    w.scales = (0.1 + torch.rand(w.scales.shape, generator=w.g, device="cuda")).half()
    x = torch.randn(m, k, generator=w.g, device="cuda")
    for at in (5, 300, k - 1):
        x[:, at] *= 1e4
        w.set_difference(at, torch.zeros(1, n, device="cuda", dtype=torch.int64))
    x = x.to(R.TYPES[dtype])
    y = linear(w, x, dtype).double()
    values = (w.scales[0].double().repeat_interleave(group, 1) *
              (w.codes[0].double() - w.zeros[0].double().repeat_interleave(group, 1)))
    error = (y - x.double() @ values.t()).square().mean().sqrt()
    q = (x.double().square() @ values.square().t()).mean().sqrt()
    assert error <= R.U * np.sqrt(3 * k + k // group + 12) * q, (error / (R.U * q)).item()


# (m, experts): one token, a few, and entries of up to four, eight and sixteen of them
@pytest.mark.parametrize("group,fmt", [(32, ZEROS), (64, BF16 | ZEROS), (128, 0)])
@pytest.mark.parametrize("m,e", [(1, 3), (3, 2), (6, 9), (6, 1), (20, 1), (64, 5)])
def test_every_bit_through_the_experts(qll_gpu, m, e, group, fmt):
    """f32 rows as above, each output one gated product times powers of two.  The
    product is cut to three parts of eight bits, of its f32 rounding or of the product itself (what the first part
    leaves may come of one fma): less than 2^-23 of it is left out; the parts' sum rounds at most once more, 2^-24."""
    n, k, top = 1152, 1280, min(2, e)
    gate, up, down = (Drawn(*s, group, fmt, m + i, e) for i, s in enumerate(((n, k), (n, k), (k, n))))
    g = gate.g
    place(gate, g), place(up, g)
    down.codes.copy_(down.zeros.repeat_interleave(group, 2))  # every weight zero but for one a row
    pick = torch.randint(0, n, (e, k), generator=g, device="cuda")
    power = 1 << torch.randint(0, 3, (e, k), generator=g, device="cuda")
    z = down.zeros.gather(2, (pick // group).unsqueeze(2)).squeeze(2).int()
    c = torch.where(z + power > 15, z - power, z + power)
    down.codes.scatter_(2, pick.unsqueeze(2), c.to(torch.uint8).unsqueeze(2))
    scale = down.scales.gather(2, (pick // group).unsqueeze(2)).squeeze(2).double()
    columns = pairs(k, group)
    value, large = full("f32", (m,), g), full("f32", (m,), g) * 2.0 ** 30
    x = torch.zeros(m, k, device="cuda")
    ids = torch.full((m, top), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((m, top), 0.5, device="cuda")
    want = torch.empty(m, k, device="cuda", dtype=torch.float64)
    for i in range(m):
        signal, outlier = columns[i % len(columns)]
        x[i, signal], x[i, outlier] = value[i], large[i]
        own = i % e
        ids[i, i % top] = own
        h = gate.column(signal)[own] * up.column(signal)[own] * value[i].double() ** 2
        want[i] = 0.5 * scale[own] * (c - z)[own].double() * h[pick[own]]
    y = torch.empty(m, k, device="cuda")
    qll.qll_q4g_moe(x, 0, ids, weights, top, gate.packed(), up.packed(), down.packed(), group, fmt, qll.QLL_ACT_NONE, None,
                    y, m, n, k, e, ws=empty(qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, n, top)))
    torch.cuda.synchronize()
    assert torch.all((y.double() - want).abs() <= 1.5 * 2.0 ** -23 * want.abs())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,e", [(1, 2), (3, 2), (4, 1), (6, 1), (20, 1)])
def test_gated_products_of_a_16_bit_stream(qll_gpu, m, e, dtype):
    """All but 2^-17 of their leading power of two is kept, of up to four tokens all but 2^-23: each output is the
    small difference of one in [1, 2) and of 1.5, which shows it; sums of few f32 terms below 2 add 4 u."""
    n, k, group = 640, 320, 64
    gate, up, down = (Drawn(*s, group, 0, m + i, e) for i, s in enumerate(((n, k), (n, k), (k, n))))
    g = gate.g
    for w in (gate, up, down):
        w.codes.fill_(8)
    gate.codes[:, :, 70] = up.codes[:, :, 70] = 9
    first = 1.0 + torch.rand(e, n, generator=g, device="cuda") * 0.5
    first[:, 0] = 1.0
    gate.scales[:, :, 1] = first.half()
    up.scales[:, :, 1] = (1.5 / gate.scales[:, :, 1].float()).half()
    h = gate.scales[:, :, 1].double() * up.scales[:, :, 1].double()
    assert (h[:, 0] == 1.5).all() and (h - 1.5).abs().max() < 2.0 ** -10
    down.scales.fill_(0.125)
    pick = torch.randint(1, n, (e, k), generator=g, device="cuda")
    down.codes.scatter_(2, pick.unsqueeze(2), 9)
    down.codes[:, :, 0] = 7
    x = torch.zeros(m, k, device="cuda", dtype=R.TYPES[dtype])
    x[:, 70] = 1.0
    ids = (torch.arange(m, device="cuda") % e).int().view(m, 1)
    y = torch.empty_like(x)
    qll.qll_q4g_moe(x, R.CODES[dtype], ids, torch.ones(m, 1, device="cuda"), 1, gate.packed(), up.packed(), down.packed(),
                    group, 0, qll.QLL_ACT_NONE, None, y, m, n, k, e, ws=empty(qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, n, 1)))
    torch.cuda.synchronize()
    want = 0.125 * (h.gather(1, pick) - 1.5)[ids[:, 0].long()].cpu().numpy()
    bound = R.rounded(want, np.full_like(want, 0.125 * ((2.0 ** -17 if m > 4 else 2.0 ** -23) + 4 * R.U)), dtype)
    assert np.all(np.abs(R.f64(y) - want) <= bound)
