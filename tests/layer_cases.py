"""Inputs and error bounds shared by the layer operators' tests.

EPS is half a unit in the last place of fp32 relative to the value.  The
elementary functions' errors come from their definitions in the PTX ISA:
ex2.approx 2 ulp (4 EPS), rcp.approx 1 ulp (2 EPS), sqrt / rsqrt.approx 1 to 2
ulp (4 EPS).
"""
import numpy as np
import torch

EPS = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def f64(t):
    return t.detach().cpu().double().numpy()


def glr_inputs(T, n_seq, D, dtype, seed, starts=None, fast=True):
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(T, 3, D, generator=g).to(dtype)
    rate = -torch.log(0.9 + 0.099 * torch.rand(D, generator=g))
    if fast:
        rate[::5] *= 40.0  # fast ones too, on both sides of the series' end
    h0 = 0.5 * torch.randn(n_seq, D, generator=g)
    if starts is None:
        starts = [T // n_seq * k for k in range(n_seq + 1)]
    return u, rate, h0, starts


# The largest relative error of s(x) with |x| <= 8: the rounded exponent's
# argument 8 EPS, ex2 4, both times 1 - s(x) <= 1, the sum 1, rcp 2.
SIG = 15 * EPS


def glr_bounds(u, rate, h0, starts):
    """Bound of |h - oracle|: a has an absolute error of EPS (it is 1 - p,
    rounded) and of p's, whose relative error is SIG + the product's EPS + the
    series' 4 EPS, or where l >= 1/4 (p >= 0.22) the far branch's 4 EPS e^-l +
    the argument's, below 25 EPS in all: 40 EPS p covers both.  m has half of
    q's relative error (p's + 3) and 4, m s(i) x 3 more and s(i)'s: 45 EPS.
    Folding rows in another order rounds every product of a's and every sum
    once more: 3 EPS of the state's envelope H, which bounds each partial
    sum."""
    from oracle import layer_ops as O
    a, m, _, si, x, _ = O.glr_coefficients(u, rate)
    T, _, D = u.shape
    bound, H = np.zeros((T, D)), np.zeros((T, D))
    last = np.zeros_like(h0)
    for s in range(len(starts) - 1):
        e, env = np.zeros(D), np.abs(h0[s])
        for t in range(starts[s], starts[s + 1]):
            b = np.abs(m[t] * si[t] * x[t])
            e = a[t] * e + EPS * ((4 * a[t] + 40 * (1 - a[t])) * env + 45 * b + a[t] * env + b)
            env = a[t] * env + b
            bound[t], H[t] = e, env
        last[s] = e
    return bound + 1e-30, last + 1e-30


def glr_adjoint_bounds(u, rate, h0, starts, h, dh, dh_last):
    """Bounds of (du, drate, dh0): lam's as the state's, run backward; the
    outputs' own factors then add less than 80 EPS of the magnitudes that go
    into each (1 - s taken as 1, since it is a difference)."""
    from oracle import layer_ops as O
    a, m, sr, si, x, left = O.glr_coefficients(u, rate)
    T, _, D = u.shape
    du, drate, dh0 = np.zeros((T, 3, D)), np.zeros(D), np.zeros_like(dh_last)
    size = np.zeros(D)
    rows = 0
    for s in range(len(starts) - 1):
        lo, hi = starts[s], starts[s + 1]
        e, env = np.zeros(D), np.abs(dh_last[s])
        for t in range(hi - 1, lo - 1, -1):
            env = env + np.abs(dh[t])
            e = e + EPS * env
            before = np.abs(h0[s] if t == lo else h[t - 1])
            with np.errstate(divide="ignore", invalid="ignore"):
                slope = np.where(left[t] > 0, a[t] ** 2 / m[t], 0.0)
            into = si[t] * np.abs(x[t]) * slope + a[t] * before
            every = e + 80 * EPS * env
            du[t, 0] = into * left[t] * every
            du[t, 1] = m[t] * np.abs(x[t]) * si[t] * every
            du[t, 2] = m[t] * si[t] * every
            drate += into * sr[t] * every
            size += into * sr[t] * env
            rows += 1
            e = a[t] * e + EPS * (6 * a[t] + 40 * (1 - a[t])) * env
            env = a[t] * env
        dh0[s] = e
    # the sum over rows: at most `rows` additions in a row in any order
    return du + 1e-30, drate + rows * EPS * size + 1e-30, dh0 + 1e-30
