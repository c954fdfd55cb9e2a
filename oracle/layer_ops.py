"""float64 oracle of the layer operators (numpy; test infrastructure only).

The gated linear recurrence is stepped one row after another, each sequence by
itself; the norm and the 8-bit formats are written from their definitions.
Nothing here shares code with the CUDA library.
"""
import numpy as np

TOP, LEAST = 448.0, 2.0 ** -126


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def glr_coefficients(u, rate):
    """(a, m, s(r), s(i), x, l) of every row; u [T,3,D]."""
    r, i, x = u[:, 0], u[:, 1], u[:, 2]
    sr, si = sigmoid(r), sigmoid(i)
    left = rate * sr
    return np.exp(-left), np.sqrt(-np.expm1(-2 * left)), sr, si, x, left


def glr_scan(u, rate, h0, starts, h=None):
    """h [T,D] (rows in no sequence as in `h`, else NaN) and h_last [n,D]."""
    T, _, D = u.shape
    a, m, _, si, x, _ = glr_coefficients(u, rate)
    h = np.full((T, D), np.nan) if h is None else h.copy()
    last = h0.copy()
    for s in range(len(starts) - 1):
        y = h0[s]
        for t in range(starts[s], starts[s + 1]):
            y = a[t] * y + m[t] * si[t] * x[t]
            h[t] = y
        last[s] = y
    return h, last


def glr_adjoint(u, rate, h0, starts, h, dh, dh_last):
    """(du, drate, dh0, lam): gradients at the given states; du and lam are 0
    in rows of no sequence."""
    T, _, D = u.shape
    a, m, sr, si, x, left = glr_coefficients(u, rate)
    du, lam, dh0 = np.zeros((T, 3, D)), np.zeros((T, D)), dh_last.copy()
    drate = np.zeros(D)
    for s in range(len(starts) - 1):
        lo, hi = starts[s], starts[s + 1]
        back = dh_last[s].copy()  # gradient that reaches the row's state from behind
        for t in range(hi - 1, lo - 1, -1):
            g = dh[t] + back
            lam[t] = g
            before = h0[s] if t == lo else h[t - 1]
            with np.errstate(divide="ignore", invalid="ignore"):
                slope = np.where(left[t] > 0, a[t] ** 2 / m[t], 0.0)  # dm / dl
            dl = g * (si[t] * x[t] * slope - a[t] * before)
            du[t, 0] = dl * left[t] * (1 - sr[t])
            du[t, 1] = g * m[t] * x[t] * si[t] * (1 - si[t])
            du[t, 2] = g * m[t] * si[t]
            drate += dl * sr[t]
            back = a[t] * g
        if hi > lo:
            dh0[s] = back
    return du, drate, dh0, lam


def rms_norm(x, res, w, eps):
    v = x if res is None else x + res
    rstd = 1.0 / np.sqrt((v * v).mean(-1) + eps)
    return v * rstd[:, None] * w, v, rstd


def rms_norm_adjoint(dy, v, w, rstd, dv):
    """Gradients with rstd = 1/sqrt(mean v^2 + eps) as given."""
    n = v * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(-1, keepdims=True))
    return dx + (0 if dv is None else dv), (dy * n).sum(0)


def e4m3(z):
    """The e4m3 value nearest to z (ties to the even one), |z| up to 448."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6))) - 3)
    return np.clip(np.rint(z / step) * step, -TOP, TOP)


def block_scales(x, rows):
    """max(largest magnitude / 448, 2^-126) of each rows x 128 block."""
    M, K = x.shape
    out = np.empty((-(-M // rows), -(-K // 128)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = max(np.abs(x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]).max() / TOP, LEAST)
    return out


def spread(scale, rows, M, K):
    """A scale per entry."""
    return np.repeat(np.repeat(scale, rows, 0)[:M], 128, 1)[:, :K]


def fp8_project(x, xs, w, ws, bias):
    """(u, sum of the magnitudes that add up to it)."""
    wide, deep = x * spread(xs, 1, *x.shape), w * spread(ws, 128, *w.shape)
    u = wide @ deep.T
    return u + (0 if bias is None else bias), np.abs(wide) @ np.abs(deep).T
