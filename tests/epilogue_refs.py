"""Plain 64-bit forms of the linear and gated entries on the oracle's products,
with the error each kernel may make, as bounds per output.

u = 2^-24 (half a step of f32).  A product's f32 sum over nb blocks, in any
order, is off by at most (nb + 8) u sum_b |term_b| (nb - 1 additions and, per
term, the conversion, the scale product and the fma).  An activation has slope
at most 1.13; its own evaluation, x / (1 + exp(-t)), has a relative error of
a few steps plus exp's argument rounding |t| 2^-22 (t a cubic of x with four
roundings); the erf form's argument rounding moves erfc(z) by 2 z^2 2^-23
relative, and a fit of erfc and its evaluation are good to 16 steps with room."""
import numpy as np
from scipy import special

import oracle as O
import quantized_linear_layer_amd as qll

U = 2.0 ** -24
ACTS = {"none": qll.QLL_ACT_NONE, "relu": qll.QLL_ACT_RELU, "gelu": qll.QLL_ACT_GELU,
        "gelu_tanh": qll.QLL_ACT_GELU_TANH, "silu": qll.QLL_ACT_SILU}


def product(codes, d_bits, xq_ref, m):
    """(f64 product, bound on the kernel's f32 sum) for raw Q4_0 draws."""
    n, k = codes.shape
    y, mag = O.q4_0_q8_0(O.pack_q4_0(codes, d_bits), xq_ref, m, n, k)
    return y, (k // 32 + 8) * U * mag


def activated(v, ev, act):
    """act(v) in 64 bits and its bound, for v known up to ev."""
    if act == "none":
        return v, ev
    if act == "relu":
        return np.maximum(v, 0.0), ev
    if act == "gelu":
        y, steps = v * special.ndtr(v), 16 + v * v
    elif act == "gelu_tanh":
        t = 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        y, steps = v * special.expit(t), 16 + 4 * np.abs(t)
    else:
        y, steps = v * special.expit(v), 16 + 2 * np.abs(v)
    return y, 1.13 * ev + steps * 2 * U * np.abs(y) + 1e-36


def linear(v, ev, bias, act, residual):
    if bias is not None:
        v = v + bias.astype(np.float64)
        ev = ev + U * (np.abs(v) + ev)
    y, ey = activated(v, ev, act)
    if residual is not None:
        y = y + residual.astype(np.float64)
        ey = ey + U * (np.abs(y) + ey)
    return y, ey


def gated(g, eg, u, eu, act):
    a, ea = activated(g, eg, act)
    y = a * u
    return y, np.abs(a) * eu + np.abs(u) * ea + ea * eu + U * np.abs(y) + 1e-36


def assert_bound(y, want, bound, what):
    y = np.asarray(y, np.float64).reshape(want.shape)
    bad = ~(np.abs(y - want) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside their bound; first at "
                           f"{np.argwhere(bad)[0].tolist()}: got {y[bad][0]!r} want {want[bad][0]!r} +- {bound[bad][0]!r}")
