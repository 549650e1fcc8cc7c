"""Dense path in numpy, 64 bits (test infrastructure): 8-bit rows with scales, the RMS
norm in front of them, the 8-bit linear, log probabilities.

Written from the definitions in include/lb.h; shares no code with the CUDA path.
"""
import numpy as np


def quantize(v, size=None):
    """(codes, scales) of the rows of v; size multiplies the scale (1 without a norm).

    Rows of zeros: codes 0, scale 0.  Rows with a NaN or an infinity: codes 0, scale NaN.
    The quotients are formed in 64-bit significands: 127 v is exact there (60 bits at most),
    so a tie stays one, and what is no tie is at least 2^-62 away, relatively, which the one
    rounding (2^-64) does not bridge.
    """
    assert np.finfo(np.longdouble).nmant >= 63, "needs a long double of 64 bits or more"
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(all="ignore"):
        peak = np.max(np.abs(v), axis=1)
        fine = np.isfinite(peak) & (peak > 0)
        safe = np.where(fine, peak, 1.0)
        q = np.rint(np.where(fine[:, None], v, 0.0).astype(np.longdouble) * 127
                    / safe[:, None].astype(np.longdouble))
        scale = np.where(np.isfinite(peak), peak, np.nan) / 127.0
        if size is not None:
            scale = scale * size
    return q.astype(np.int8), np.where(peak == 0, 0.0, scale)


def rmsnorm_quantize(s, weight=None, eps=1e-5):
    """(codes, scales) of the RMS norm of the stored sums s, times weight."""
    s = np.asarray(s, dtype=np.float64)
    with np.errstate(all="ignore"):
        size = 1.0 / np.sqrt(np.mean(s * s, axis=1) + np.float64(np.float32(eps)))
    return quantize(s if weight is None else s * np.asarray(weight, dtype=np.float64)[None, :], size)


def linear_int8(xq, xs, wq, ws):
    """y = xs ws (xq wq^T), the integer sums exact (below 2^53 in 64-bit floats)."""
    acc = np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T
    return acc * np.asarray(xs, dtype=np.float64)[:, None] * np.asarray(ws, dtype=np.float64)[None, :]


def order(x, top):
    """Ids of the `top` largest of each row: NaN first, then falling, equal ones by rising id."""
    x = np.asarray(x, dtype=np.float64)
    ids = np.broadcast_to(np.arange(x.shape[1]), x.shape)
    nan = np.isnan(x)
    return np.lexsort((ids, -np.where(nan, 0.0, x), ~nan), axis=1)[:, :top]


def token_logprobs(x, tokens=None, top=0):
    """(logprob or None, entropy, ids, log probabilities of the ids)."""
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    lp = np.empty_like(x)
    entropy = np.empty(rows)
    for i in range(rows):
        if np.isnan(x[i]).any() or (x[i] == np.inf).any():
            lp[i], entropy[i] = np.nan, np.nan
        elif (x[i] == -np.inf).all():
            lp[i], entropy[i] = -np.inf, 0.0
        else:
            d = x[i] - x[i].max()
            lp[i] = d - np.log(np.sum(np.exp(d)))
            p = np.exp(lp[i])
            entropy[i] = -np.sum(p[p > 0] * lp[i][p > 0])
    given = None
    if tokens is not None:
        t = np.asarray(tokens)
        given = lp[np.arange(rows), np.clip(t, 0, vocab - 1)]
        given = np.where(t < 0, 0.0, np.where(t >= vocab, np.nan, given))
    ids = order(x, top)
    return given, entropy, ids, np.take_along_axis(lp, ids, axis=1)
