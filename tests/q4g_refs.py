"""Plain 64-bit forms of the products with 4-bit group-scaled weights and of the
mixture-of-experts layer, with the error the kernels may make, as bounds per
output.

u = 2^-24 (half a step of f32).  A group's sum D of g products x (16 + c) and its
sum S of activations are f32 sums of at most 3 g terms in any order (f32
activations count as three parts): off by at most 3 g u sum |x| (16 + c) and
3 g u sum |x|; S is taken 16 + z times.  The difference, the scale's product and
the sum over the groups and the waves that share k add (k / g + 12) u of the
parts' magnitudes, which are sum |s x (c - z)| and what is off already."""
import numpy as np
import torch

import epilogue_refs as E
import quantized_linear_layer_amd as qll

U = E.U
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": qll.QLL_DTYPE_F32, "bf16": qll.QLL_DTYPE_BF16, "f16": qll.QLL_DTYPE_F16}


def f64(t):
    return t.double().cpu().numpy()


class Weights:
    """Draws of `count` matrices [n][k] and their packed form, one after another."""

    def __init__(self, rng, n, k, group, fmt, count=1, device="cuda", scale=None):
        self.n, self.k, self.group, self.fmt, self.count = n, k, group, fmt, count
        sdt = torch.bfloat16 if fmt & qll.QLL_Q4G_BF16 else torch.float16
        self.codes = rng.integers(0, 16, (count, n, k), dtype=np.uint8)
        s = rng.uniform(0.1, 1.0, (count, n, k // group)) * (scale or 0.3 / np.sqrt(k))
        s *= rng.choice([-1.0, 1.0], s.shape)
        self.scales = torch.from_numpy(s).to(sdt)
        zeros = bool(fmt & qll.QLL_Q4G_ZEROS)
        self.zeros = rng.integers(0, 16, (count, n, k // group), dtype=np.uint8) if zeros else None
        if device:
            self.pack(device)

    def pack(self, device):
        size = qll.qll_q4g_packed_bytes(self.n, self.k, self.group, self.fmt)
        # every byte is the packing's to write, and none behind them
        self.wp = torch.full((self.count * size + 64,), 0xA5, dtype=torch.uint8, device=device)
        for i in range(self.count):
            qll.qll_q4g_pack(torch.from_numpy(self.codes[i]).to(device), self.scales[i].contiguous().to(device),
                             None if self.zeros is None else torch.from_numpy(self.zeros[i]).to(device), self.group,
                             self.fmt, self.wp[i * size:(i + 1) * size], self.n, self.k)
        assert (self.wp[self.count * size:] == 0xA5).all(), "packing wrote past its bytes"

    def values(self, i=0):
        """(scale, zero point, code) of every weight in 64 bits, [n][k] each."""
        s = np.repeat(f64(self.scales[i]), self.group, 1)
        z = np.full(s.shape, 8.0) if self.zeros is None else np.repeat(self.zeros[i].astype(np.float64), self.group, 1)
        return s, z, self.codes[i].astype(np.float64)

    def product(self, x, ex=None, i=0):
        """x.W^T of matrix i in 64 bits and the bound on the kernel's; ex: how far x itself may be off."""
        s, z, c = self.values(i)
        a = np.abs(x) if ex is None else np.abs(x) + ex
        y = x @ (s * (c - z)).T
        parts = np.abs(s) * (32.0 + c + z)
        mag = a @ (np.abs(s) * np.abs(c - z)).T
        off = 3 * self.group * U * (a @ parts.T)
        off += (self.k // self.group + 12) * U * (mag + off)
        if ex is not None:
            off += ex @ (np.abs(s) * np.abs(c - z)).T
        return y, off + 1e-36


def rounded(y, bound, dtype):
    """The bound after one rounding to dtype: half a step of the value, or of the
    smallest normal one."""
    info = torch.finfo(TYPES[dtype])
    return bound + (np.abs(y) + bound) * (info.eps / 2) + info.smallest_normal * info.eps / 2


def linear(w, x, bias, act, residual, y_dtype):
    y, b = E.linear(*w.product(x), bias, act, residual)
    return y, rounded(y, b, y_dtype)


def route(x, wr, bias, score, renorm, scale, top):
    """ids, weights in 64 bits; ties go to the lower index."""
    l = x @ wr.T
    if score == qll.QLL_SCORE_SOFTMAX:
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-l))
    by = l if bias is None else p + bias.astype(np.float64)
    ids = np.argsort(-by, 1, kind="stable")[:, :top]
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        w = w / w.sum(1, keepdims=True)
    return ids.astype(np.int32), w * scale


def moe(x, ids, weights, wg, wu, wd, act, residual, dtype):
    """The layer in 64 bits on given ids and f32 weights, and its bound."""
    m, top = ids.shape
    y, b, mag = (np.zeros((m, wd.n)) for _ in range(3))
    for t in range(m):
        for j in range(top):
            e = ids[t, j]
            if not 0 <= e < wg.count:
                continue
            row = x[t:t + 1]
            h, eh = E.gated(*wg.product(row, i=e), *wu.product(row, i=e), act)
            if dtype != "f32":  # kept as two bf16 parts: the first cut off, the second rounded
                eh = eh + (np.abs(h) + eh) * 2.0 ** -16
            d, ed = wd.product(h, eh, i=e)
            w = float(weights[t, j])
            y[t] += w * d[0]
            b[t] += abs(w) * ed[0]
            mag[t] += abs(w) * (np.abs(d[0]) + ed[0])
    # weights and products into a wave's sum, the waves' sums, the residual
    b += (top + 12) * U * mag
    if residual is not None:
        y = y + residual
        b = b + U * (np.abs(y) + b)
    return y, rounded(y, b, dtype)
