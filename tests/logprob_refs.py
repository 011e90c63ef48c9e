"""Token log probabilities in 64 bits, with the error the kernel may make.

u = 2^-24.  With d = M - x over the logits that count (exp(-80) is far below
an f32 sum's rounding), log S is off by at most (40 + 8 max d) u: at most 16
f32 additions (f64 beyond) and the weights that bring lanes, waves and
segments to one reference, and per term the roundings of the difference, of
its product with log2(e) and of that constant, each d u or less, and of
exp2.  The entropy's sum of p d has that relative error too."""
import numpy as np

U = 2.0 ** -24


def reference(x, tokens, top):
    """x: float32 values [m][v], tokens [m][t].  Returns (logprob, entropy,
    ids, top_logprob, bound on log p, bound on the entropy)."""
    x = x.astype(np.float64)
    m, v = x.shape
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        big = np.where(np.isnan(x), -np.inf, x).max(1, keepdims=True)
        d = x - big
        e = np.exp(d)
        s = e.sum(1, keepdims=True)
        lp = d - np.log(s)
        pd = np.where(e > 0, -d * e, np.where(np.isnan(e), np.nan, 0.0)).sum(1, keepdims=True) / s
        entropy = np.log(s) + pd
        spread = np.where(np.isfinite(d), np.minimum(-d, 80.0), 0.0).max(1, keepdims=True)
    eb = (40 + 8 * spread) * U
    ids = np.stack([np.lexsort((np.arange(v), -x[i]))[:top] for i in range(m)]) if top else np.zeros((m, 0), int)
    ok = (tokens >= 0) & (tokens < v)
    picked = np.where(ok, np.take_along_axis(lp, np.where(ok, tokens, 0), 1), np.nan)
    return (picked, entropy[:, 0], ids, np.take_along_axis(lp, ids, 1), eb,
            (eb * (1 + np.nan_to_num(pd)))[:, 0] + 2 * U * np.abs(np.nan_to_num(entropy[:, 0])))


def assert_close(got, want, bound, what):
    got = np.asarray(got, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    same = fine | np.isnan(want)
    assert np.array_equal(got[~same], want[~same]), f"{what}: infinities differ"
    err = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    lim = np.broadcast_to(bound, want.shape) + 2 * U * np.abs(np.where(fine, want, 0))
    assert (err <= lim).all(), f"{what}: off by {err.max()}, {(err > lim).sum()} outside"
