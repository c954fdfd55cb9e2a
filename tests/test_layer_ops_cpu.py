"""The layer operators without a GPU: the oracle's own pins, the refusals of
the C entry points and of the binding, workspace sizes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import layer_ops as O
from tests import layer_cases as C

STARTS = [2, 2, 9, 10, 23, 23]  # empty, 7 rows, one row, 13 rows, empty; 2 rows before, 2 behind
T = 25


@pytest.fixture(scope="module")
def capi():
    from nonlinear_rnn_newton_b200 import build
    build.build()
    from nonlinear_rnn_newton_b200 import capi
    return capi


def arrays(seed=0):
    u, rate, h0, starts = C.glr_inputs(T, 5, 8, torch.float32, seed, STARTS)
    g = np.random.default_rng(seed)
    return C.f64(u), C.f64(rate), C.f64(h0), starts, g.standard_normal((T, 8)), g.standard_normal((5, 8))


# -------------------------------------------------------------- oracle pins

def test_recurrence_against_the_weighted_sum():
    """h_t = sum over k of (product of later a's) b_k, written out."""
    u, rate, h0, starts, _, _ = arrays()
    h, last = O.glr_scan(u, rate, h0, starts)
    a, m, _, si, x, _ = O.glr_coefficients(u, rate)
    for s, (lo, hi) in enumerate(zip(starts, starts[1:])):
        for t in range(lo, hi):
            want = np.prod(a[lo:t + 1], 0) * h0[s]
            for k in range(lo, t + 1):
                want = want + np.prod(a[k + 1:t + 1], 0) * m[k] * si[k] * x[k]
            assert np.allclose(h[t], want, rtol=1e-12, atol=1e-14)
        assert np.array_equal(last[s], h[hi - 1] if hi > lo else h0[s])
    assert np.isnan(h[:2]).all() and np.isnan(h[23:]).all()


def test_adjoint_against_differences():
    u, rate, h0, starts, dh, dh_last = arrays(3)
    h, _ = O.glr_scan(u, rate, h0, starts)
    du, drate, dh0, _ = O.glr_adjoint(u, rate, h0, starts, h, dh, dh_last)

    def loss(u, rate, h0):
        h, last = O.glr_scan(u, rate, h0, starts)
        return (np.where(np.isnan(h), 0, h) * dh).sum() + (last * dh_last).sum()

    g = np.random.default_rng(5)
    for k, (x, dx) in enumerate(((u, du), (rate, drate), (h0, dh0))):
        for _ in range(3):
            v = g.standard_normal(x.shape) * (x if k == 1 else 1)
            args = [[u, rate, h0], [u, rate, h0]]
            args[0][k], args[1][k] = x + 1e-6 * v, x - 1e-6 * v
            assert np.isclose((loss(*args[0]) - loss(*args[1])) / 2e-6, (dx * v).sum(), rtol=1e-6, atol=1e-7)


def test_shut_gates_hold_the_state():
    u, rate, h0, starts, dh, dh_last = arrays(1)
    u[:, 0] = -np.inf
    h, last = O.glr_scan(u, rate, h0, starts)
    assert np.array_equal(last, h0)
    du, drate, dh0, _ = O.glr_adjoint(u, rate, h0, starts, h, dh, dh_last)
    assert np.isfinite(du).all() and np.isfinite(drate).all()
    assert np.allclose(dh0[1], dh_last[1] + dh[2:9].sum(0))


def test_norm_adjoint_against_differences():
    g = np.random.default_rng(0)
    x, w, dy = g.standard_normal((3, 40)), g.standard_normal(40), g.standard_normal((3, 40))
    y, v, rstd = O.rms_norm(x, None, w, 1e-3)
    dx, dw = O.rms_norm_adjoint(dy, v, w, rstd, None)
    p, q = g.standard_normal(x.shape), g.standard_normal(w.shape)
    f = lambda k: (O.rms_norm(x + k * p, None, w + k * q, 1e-3)[0] * dy).sum()
    assert np.isclose((f(1e-6) - f(-1e-6)) / 2e-6, (dx * p).sum() + (dw * q).sum(), rtol=1e-6)


def test_e4m3_against_torch():
    z = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    z = torch.cat([z, torch.linspace(-0.05, 0.05, 4001, dtype=torch.float64)]).float()
    assert np.array_equal(O.e4m3(z.double().numpy()), z.to(torch.float8_e4m3fn).double().numpy())


def test_project_against_loops():
    g = np.random.default_rng(0)
    x, w = g.standard_normal((2, 144)), g.standard_normal((130, 144))
    xs, ws, bias = g.random((2, 2)), g.random((2, 2)), g.random(130)
    u, _ = O.fp8_project(x, xs, w, ws, bias)
    for m, n in ((0, 0), (1, 129), (0, 127), (1, 128)):
        want = bias[n] + sum(x[m, k] * xs[m, k // 128] * w[n, k] * ws[n // 128, k // 128] for k in range(144))
        assert np.isclose(u[m, n], want, rtol=1e-12)


# --------------------------------------------------------- C entry refusals
# (fake pointers: every refusal comes before any device call)

A = [1 << 20 << k for k in range(14)]  # far apart


def test_scan_refusals(capi):
    def call(u=A[0], dt=1, rate=A[1], h0=A[2], starts=None, h=A[9], last=A[3], T=8, n=2, D=16, ws=256, wsb=1 << 20):
        return capi.lib.pararnn_glr_scan(u, dt, rate, h0, starts, h, last, T, n, D, ws, wsb, None)

    for bad in (dict(u=None), dict(rate=None), dict(h=None), dict(u=A[0] + 8), dict(h0=A[2] + 4), dict(starts=A[4] + 2),
                dict(dt=2), dict(dt=7), dict(T=0), dict(n=0), dict(T=-1), dict(D=0), dict(T=9),  # 9 rows, 2 sequences
                dict(h=A[0]), dict(h=A[0] + 16), dict(last=A[2]), dict(last=A[9] + 64),
                dict(T=1 << 32, n=1), dict(T=1 << 30, D=1 << 20, n=1)):
        assert call(**bad) == capi.ERR_INVALID_ARG, bad
        assert capi.last_error()
    assert call(D=12) == capi.ERR_UNSUPPORTED
    assert call(ws=None) == capi.ERR_WORKSPACE
    assert call(ws=16) == capi.ERR_WORKSPACE
    assert call(wsb=8) == capi.ERR_WORKSPACE


def test_adjoint_refusals(capi):
    def call(u=A[0], dt=0, rate=A[1], h0=None, starts=A[2], h=A[3], dh=A[4], dl=None, du=A[5], dr=A[6], d0=A[7], T=8, n=3,
             D=16, ws=256, wsb=1 << 20):
        return capi.lib.pararnn_glr_adjoint(u, dt, rate, h0, starts, h, dh, dl, du, dr, d0, T, n, D, ws, wsb, None)

    for bad in (dict(u=None), dict(rate=None), dict(h=None), dict(dh=None), dict(du=None), dict(dr=None), dict(dt=2),
                dict(d0=A[7] + 8), dict(dl=A[8] + 2), dict(du=A[0]), dict(du=A[4] - 16), dict(d0=A[6]), dict(dl=A[7]),
                dict(starts=None)):  # 8 rows, 3 sequences
        assert call(**bad) == capi.ERR_INVALID_ARG, bad
    assert call(D=20) == capi.ERR_UNSUPPORTED
    assert call(ws=None) == capi.ERR_WORKSPACE
    assert call(wsb=16) == capi.ERR_WORKSPACE


def test_step_refusals(capi):
    def call(u=A[0], dt=1, rate=A[1], hp=None, hn=A[2], B=2, D=16):
        return capi.lib.pararnn_glr_step(u, dt, rate, hp, hn, B, D, None)

    for bad in (dict(u=None), dict(rate=None), dict(hn=None), dict(hn=A[2] + 8), dict(dt=2), dict(B=0),
                dict(hp=A[2] + 16), dict(hn=A[0])):
        assert call(**bad) == capi.ERR_INVALID_ARG, bad
    assert call(D=4) == capi.ERR_UNSUPPORTED


def test_norm_refusals(capi):
    def call(x=A[0], xd=1, r=A[1], rd=1, w=A[2], eps=1e-6, s=A[3], y=A[4], yd=2, sc=A[5], rs=A[6], T=4, D=32):
        return capi.lib.pararnn_rms_norm(x, xd, r, rd, w, eps, s, y, yd, sc, rs, T, D, None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(sc=None), dict(xd=2), dict(rd=2), dict(yd=3), dict(yd=-1),
                dict(x=A[0] + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(T=0), dict(D=0),
                dict(y=A[0]), dict(s=A[0]), dict(s=A[1] + 16), dict(y=A[1], s=A[1]), dict(y=A[3]), dict(rs=A[4]),
                dict(T=1 << 31)):
        assert call(**bad) == capi.ERR_INVALID_ARG, bad
    assert call(D=24) == capi.ERR_UNSUPPORTED  # 8 bits need a multiple of 16
    assert call(D=12, yd=1) == capi.ERR_UNSUPPORTED
    assert call(D=16384 + 16) == capi.ERR_UNSUPPORTED

    def adj(dy=A[0], yd=1, s=A[1], sd=1, w=A[2], rs=A[3], ds=None, dx=A[4], dw=A[5], T=4, D=32, ws=256, wsb=1 << 20):
        return capi.lib.pararnn_rms_norm_adjoint(dy, yd, s, sd, w, rs, ds, dx, dw, T, D, ws, wsb, None)

    for bad in (dict(dy=None), dict(s=None), dict(w=None), dict(rs=None), dict(dx=None), dict(dw=None), dict(yd=2),
                dict(sd=2), dict(dx=A[1]), dict(ds=A[4] + 16), dict(dw=A[4]), dict(T=0)):
        assert adj(**bad) == capi.ERR_INVALID_ARG, bad
    assert adj(D=12) == capi.ERR_UNSUPPORTED
    assert adj(ws=None) == capi.ERR_WORKSPACE
    assert adj(wsb=16) == capi.ERR_WORKSPACE


def test_fp8_refusals(capi):
    def q(x=A[0], dt=1, rows=1, out=A[1], sc=A[2], M=4, K=32):
        return capi.lib.pararnn_fp8_quantize(x, dt, rows, out, sc, M, K, None)

    for bad in (dict(x=None), dict(out=None), dict(sc=None), dict(dt=2), dict(rows=2), dict(rows=0), dict(M=0), dict(K=0),
                dict(out=A[0]), dict(sc=A[1]), dict(out=A[1] + 8)):
        assert q(**bad) == capi.ERR_INVALID_ARG, bad
    assert q(K=24) == capi.ERR_UNSUPPORTED

    def p(x=A[0], xs=A[1], w=A[2], ws=A[3], b=None, u=A[4], ud=1, M=4, N=16, K=32, work=256, wb=1 << 10):
        return capi.lib.pararnn_fp8_project(x, xs, w, ws, b, u, ud, M, N, K, work, wb, None)

    for bad in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(u=None), dict(ud=2), dict(M=0), dict(N=0),
                dict(K=-16), dict(b=A[5] + 4), dict(u=A[0]), dict(u=A[2] - 16), dict(M=1 << 31)):
        assert p(**bad) == capi.ERR_INVALID_ARG, bad
    assert p(K=24) == capi.ERR_UNSUPPORTED
    assert p(N=12) == capi.ERR_UNSUPPORTED
    assert p(work=None) == capi.ERR_WORKSPACE
    assert p(wb=255) == capi.ERR_WORKSPACE


def test_workspace_sizes(capi):
    for f in (capi.pararnn_glr_workspace_size, capi.pararnn_glr_adjoint_workspace_size):
        assert f(100, 3, 64) > 0 and f(100, 3, 64) % 256 == 0
        assert f(0, 3, 64) == 0 and f(100, 0, 64) == 0 and f(100, 3, 60) == 0 and f(1 << 31, 1, 64) == 0
    f = capi.pararnn_fp8_project_workspace_size
    assert f(5, 16, 32) == 256 and f(0, 16, 32) == 0 and f(5, 12, 32) == 0 and f(5, 16, 24) == 0
    f = capi.pararnn_rms_norm_adjoint_workspace_size
    assert f(100, 64) > 0 and f(100, 64) % 256 == 0
    assert f(0, 64) == 0 and f(100, 60) == 0 and f(100, 16392) == 0


def test_no_device_is_reported(capi):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = capi.lib
    assert lib.pararnn_glr_scan(A[0], 1, A[1], None, None, A[9], None, 8, 2, 16, 256, 1 << 20, None) == capi.ERR_CUDA
    assert lib.pararnn_glr_step(A[0], 1, A[1], A[2], A[2], 2, 16, None) == capi.ERR_CUDA  # in place
    assert lib.pararnn_rms_norm(A[0], 1, A[1], 1, A[2], 1e-6, A[1], A[4], 1, None, None, 4, 32, None) == capi.ERR_CUDA
    assert lib.pararnn_fp8_project(A[0], A[1], A[2], A[3], None, A[4], 1, 4, 16, 32, 256, 256, None) == capi.ERR_CUDA


# ----------------------------------------------------- the binding's refusals

def test_binding_refusals(capi):
    P = capi
    u, rate = torch.zeros(2, 3, 3, 16), torch.zeros(16)
    starts = torch.tensor([0, 3, 6], dtype=torch.int32)
    e8 = torch.zeros(4, 32).to(torch.float8_e4m3fn)
    one = torch.ones
    for error, call in (
            (ValueError, lambda: P.pararnn_glr_scan(u, rate)),  # not on a GPU
            (ValueError, lambda: P.pararnn_glr_scan(u[:, :, :2], rate)),
            (ValueError, lambda: P.pararnn_glr_scan(u, rate, seq_starts=starts)),  # packed rows are [T,3,D]
            (ValueError, lambda: P.pararnn_glr_scan(u[0], rate)),
            (ValueError, lambda: P.pararnn_glr_scan(u.transpose(0, 1), rate)),
            (TypeError, lambda: P.pararnn_glr_scan(u.half(), rate)),
            (TypeError, lambda: P.pararnn_glr_scan(u, rate.double())),
            (ValueError, lambda: P.pararnn_glr_scan(u, rate[:8])),
            (ValueError, lambda: P.pararnn_glr_scan(u, rate, torch.zeros(3, 16))),
            (TypeError, lambda: P.pararnn_glr_scan(u.view(6, 3, 16), rate, seq_starts=starts.long())),
            (ValueError, lambda: P.pararnn_glr_scan(u.view(6, 3, 16), rate, seq_starts=starts[:1])),
            (ValueError, lambda: P.pararnn_glr_adjoint(u, rate, None, u[:, :, 0], u[:, :, 0])),
            (ValueError, lambda: P.pararnn_glr_step(u, rate)),
            (ValueError, lambda: P.pararnn_rms_norm(one(16), one(16))),
            (TypeError, lambda: P.pararnn_rms_norm(one(2, 16), one(16), out_dtype=torch.float16)),
            (TypeError, lambda: P.pararnn_rms_norm(one(2, 16).half(), one(16))),
            (ValueError, lambda: P.pararnn_rms_norm(one(2, 16), one(16), sum=one(2, 16))),
            (ValueError, lambda: P.pararnn_rms_norm(one(2, 16), one(16), residual=one(3, 16))),
            (ValueError, lambda: P.pararnn_rms_norm_adjoint(one(2, 16), one(3, 16), one(16), one(3))),
            (ValueError, lambda: P.pararnn_fp8_quantize(one(2, 16), block_rows=64)),
            (ValueError, lambda: P.pararnn_fp8_quantize(one(2, 2, 16), block_rows=128)),
            (TypeError, lambda: P.pararnn_fp8_project(one(4, 32), one(4, 1), e8, one(1, 1))),
            (ValueError, lambda: P.pararnn_fp8_project(e8, one(4, 2), e8, one(1, 1))),
            (ValueError, lambda: P.pararnn_fp8_project(e8, one(4, 1), e8, one(1, 1)))):  # not on a GPU
        with pytest.raises(error):
            call()
