"""GPU parity of the layer operators where their dispatch and their arithmetic
change: few CTAs a slab, fast decays, saturated gates, scales at the ends of
fp32.  Bounds as in tests/layer_cases.py, or derived beside the test."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as O
from tests import layer_cases as C
from tests.test_gpu_layer_ops import BF16, E4M3, F32, P, check_adjoint, check_scan, near

pytestmark = pytest.mark.gpu

# rows of a tile (scan, adjoint)
TILE = {BF16: (120, 40), F32: (60, 30)}


def ends(T, packed):
    return [1, T // 3, T // 3, T // 3 + 1, T - 3] if packed else [0, T]


# CTAs a slab on 148 SMs: 1, 2, 3, 4
@pytest.mark.parametrize("D,ctas", [(4800, 1), (4096, 2), (3000, 3), (2048, 4)])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_recurrence_few_ctas_a_slab(cuda, D, ctas, tiles, dtype):
    """`tiles` tiles a CTA, the last one short; one sequence or several."""
    packed = tiles % 2 == 0
    for k, check in enumerate((check_scan, check_adjoint)):
        T = TILE[dtype][k] * ctas * tiles - 7
        starts = ends(T, packed)
        u, rate, h0, _ = C.glr_inputs(T, len(starts) - 1, D, dtype, seed=D + tiles, starts=starts, fast=tiles < 4)
        if k == 0:
            check_scan(cuda, u, rate, h0, starts, True)
        else:
            check_adjoint(cuda, u, rate, h0, starts, u.to(cuda), torch.tensor(starts, dtype=torch.int32, device=cuda), D)


@pytest.mark.parametrize("D,T", [(4800, 233), (4800, 1201), (2048, 957), (64, 9000)])
def test_adjoint_repeats_bit_for_bit(cuda, D, T):
    u, rate, h0, _ = C.glr_inputs(T, 1, D, BF16, 1)
    ud, rd, hd = u[None].to(cuda), rate.to(cuda), h0.to(cuda)
    h, dh = torch.randn(1, T, D, device=cuda), torch.randn(1, T, D, device=cuda)
    first = P().pararnn_glr_adjoint(ud, rd, hd, h, dh)
    for _ in range(30):
        assert all(torch.equal(x, y) for x, y in zip(first, P().pararnn_glr_adjoint(ud, rd, hd, h, dh)))


def glr_gradient_bounds(u, rate, h0, starts, h, dh, dh_last):
    """Bounds of (du, drate, dh0) relative to the decays and to the gates'
    slopes, in EPS, with g the larger |r| or |i| of the row:
      e^-x: its argument x log2 e is rounded twice (the constant, the product),
      2 |x|, and ex2's 4; s = 1 / (1 + e^-x): 2 |x| + 7; 1 - s = e^-x s: 4 |x| + 12;
      l = rate s: 2 |x| + 8, so a = e^-l: l (2 |x| + 10) + 4, and where it is
      1 + expm1(-l) with l < 1/8: 1 + (2 |x| + 12) / 8: both below
      A = l (2 g + 10) + g / 4 + 4;
      1 - a: a A / (1 - a) + 1, where a l / (1 - a) <= 1 and (l >= 1/8) a / (1 - a)
      <= 7.6: below 4 g + 45 (series: 2 g + 13); 1 - a^2: 4 more; m and 1 / m: half
      of that and 6: Q = 2 g + 31.
    lam adds up and is multiplied by a: A and 4 for the maps a row.  The outputs
    multiply lam, s(i), x, m or 1 / m, a^2 (2 A), h, l and 1 - s: their own factors'
    errors and 2 a product."""
    a, m, sr, si, x, left = O.glr_coefficients(u, rate)
    T, _, D = u.shape
    g = np.maximum(np.abs(u[:, 0]), np.abs(u[:, 1]))
    A, Q = left * (2 * g + 10) + g / 4 + 4, 2 * g + 31
    not_r, not_i = O.sigmoid(-u[:, 0]), O.sigmoid(-u[:, 1])
    du, drate, dh0 = np.zeros((T, 3, D)), np.zeros(D), np.zeros_like(dh_last)
    size, rows = np.zeros(D), 0
    for s in range(len(starts) - 1):
        lo, hi = starts[s], starts[s + 1]
        e, env = np.zeros(D), np.abs(dh_last[s])
        for t in range(hi - 1, lo - 1, -1):
            env = env + np.abs(dh[t])
            e = e + 3 * C.EPS * env
            before = np.abs(h0[s] if t == lo else h[t - 1])
            into = si[t] * np.abs(x[t]) * a[t] ** 2 / m[t] + a[t] * before
            fresh = m[t] * si[t]
            dl = into * (e + (2 * A[t] + Q[t] + 2 * g[t] + 17) * C.EPS * env)
            du[t, 0] = left[t] * not_r[t] * (dl + into * (6 * g[t] + 26) * C.EPS * env)
            du[t, 2] = fresh * (e + (Q[t] + 2 * g[t] + 13) * C.EPS * env)
            du[t, 1] = np.abs(x[t]) * not_i[t] * (du[t, 2] + fresh * (4 * g[t] + 16) * C.EPS * env)
            drate += sr[t] * (dl + into * (2 * g[t] + 9) * C.EPS * env)
            size += into * sr[t] * env
            rows += 1
            e = a[t] * (e + (A[t] + 5) * C.EPS * env)
            env = a[t] * env
        dh0[s] = e
    return du + 1e-36, drate + rows * C.EPS * size + 1e-36, dh0 + 1e-36


def check_gradients(dev, u, rate, h0, starts, seed):
    T, _, D = u.shape
    g = torch.Generator().manual_seed(seed)
    h, dh = torch.randn(T, D, generator=g), torch.randn(T, D, generator=g)
    dl = torch.randn(len(starts) - 1, D, generator=g)
    sd = torch.tensor(starts, dtype=torch.int32, device=dev)
    got = P().pararnn_glr_adjoint(u.to(dev), rate.to(dev), h0.to(dev), h.to(dev), dh.to(dev), dh_last=dl.to(dev),
                                  seq_starts=sd)
    args = [C.f64(t) for t in (u, rate, h0)] + [starts] + [C.f64(t) for t in (h, dh, dl)]
    du, drate, dh0, lam = O.glr_adjoint(*args)
    # the oracle's 1 - s is a difference, 0 from x = 37 on: the logistic of -x keeps its digits
    a, m, _, si, x, left = O.glr_coefficients(*args[:2])
    before = np.concatenate([args[4][:1], args[4][:-1]])
    for s, first in enumerate(starts[:-1]):
        before[first] = args[2][s]
    du[:, 0] = lam * (si * x * a * a / m - a * before) * left * O.sigmoid(-args[0][:, 0])
    du[:, 1] = lam * m * x * si * O.sigmoid(-args[0][:, 1])
    bounds = glr_gradient_bounds(*args)
    for name, x, y, b in zip(("du", "drate", "dh0"), got, (du, drate, dh0), bounds):
        near(x, y, b, name)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("starts", [[0, 200], [0, 1, 2, 90, 200]], ids=["one", "several"])
def test_gradients_of_fast_decays(cuda, starts, dtype):
    """Decays down to e^-28: what is multiplied by a keeps a's own digits."""
    T, D = 200, 72
    g = torch.Generator().manual_seed(21)
    u = torch.randn(T, 3, D, generator=g).to(dtype)
    u[:, :2] = u[:, :2].clamp(-2.5, 2.5)
    rate = torch.tensor([0.05, 0.2, 1.0, 3.0, 6.0, 10.0, 15.0, 20.0, 30.0]).repeat(8)
    h0 = torch.randn(len(starts) - 1, D, generator=g)
    check_gradients(cuda, u, rate, h0, starts, 22)


@pytest.mark.parametrize("T,D", [(1, 16), (3, 128), (50, 1040), (9, 2048), (5, 4112), (2, 16384), (1000, 512)])
@pytest.mark.parametrize("x,res", [(F32, BF16), (BF16, BF16), (BF16, None), (F32, F32)],
                         ids=lambda t: "none" if t is None else str(t)[6:])
def test_norm_in_8_bits_is_the_norm_quantised(cuda, T, D, x, res):
    """The 8-bit output is what the quantiser makes of the fp32 output, bit for
    bit: the rounded quotient by the scale decides."""
    g = torch.Generator().manual_seed(T + D)
    xs = torch.randn(T, D, generator=g).to(x).to(cuda)
    rs = None if res is None else (2 * torch.randn(T, D, generator=g)).to(res).to(cuda)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(cuda)
    y, scale, _, _ = P().pararnn_rms_norm(xs, w, residual=rs, out_dtype=E4M3)
    wide, _, _, _ = P().pararnn_rms_norm(xs, w, residual=rs, out_dtype=F32)
    q, s = P().pararnn_fp8_quantize(wide)
    assert torch.equal(scale, s)
    assert torch.equal(y.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("M", [5, 40, 100, 300, 1000])
@pytest.mark.parametrize("total", [-20, -118, -142, -155])
def test_project_of_small_scales(cuda, M, total):
    """Scales from 2^-115 to 2^115 whose product is about 2^total, however the
    exponent is split: exact to fp32 while the product is a normal number, and
    off by 2^-125 a block at most where it is not."""
    N, K = 264, 1104
    KB = (K + 127) // 128
    g = torch.Generator().manual_seed(M)
    x = (64 * torch.randn(M, K, generator=g)).clamp(-448, 448).to(E4M3)
    w = (64 * torch.randn(N, K, generator=g)).clamp(-448, 448).to(E4M3)
    split = torch.linspace(-115, total + 115, KB).round()
    xs = torch.exp2(split).repeat(M, 1) * (0.5 + torch.rand(M, KB, generator=g))
    ws = torch.exp2(total - split).repeat((N + 127) // 128, 1) * (0.5 + torch.rand((N + 127) // 128, KB, generator=g))
    got = P().pararnn_fp8_project(x.to(cuda), xs.to(cuda), w.to(cuda), ws.to(cuda), out_dtype=F32)
    want, size = O.fp8_project(C.f64(x.float()), C.f64(xs), C.f64(w.float()), C.f64(ws), None)
    # a block's 128 products, the blocks' terms and sums; the products of scales
    # are 1/4 to 9/4 of 2^total
    rel = (2 * 128 + 4 * KB + 4) * C.EPS
    small = KB * 2.0 ** -125 if total < -124 else 0.0
    near(got, want, rel * size + 2 * C.EPS * np.abs(want) + small, "u")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("slow", [True, False], ids=["slow", "fast"])
def test_gradients_of_saturated_gates(cuda, slow, dtype):
    """Gates from -50 to 50.  1 - s is a difference, so dr and di keep the
    absolute error that they have at an open gate: the bounds of layer_cases
    take 1 - s as 1, and s(x) of |x| <= 50 has up to 2 50 + 7 EPS where theirs
    of |x| <= 8 has up to 23, hence five times these."""
    T, D = 130, 72
    g = torch.Generator().manual_seed(31)
    u = torch.randn(T, 3, D, generator=g)
    u[:, :2] = 100 * torch.rand(T, 2, D, generator=g) - 50
    u = u.to(dtype)
    rate = (0.001 + 0.12 * torch.rand(D, generator=g)) * (1 if slow else 20)
    h0, dl = torch.randn(1, D, generator=g), torch.randn(1, D, generator=g)
    h, dh = torch.randn(1, T, D, generator=g), torch.randn(1, T, D, generator=g)
    got = P().pararnn_glr_adjoint(u[None].to(cuda), rate.to(cuda), h0.to(cuda), h.to(cuda), dh.to(cuda),
                                  dh_last=dl.to(cuda))
    args = [C.f64(t) for t in (u, rate, h0)] + [[0, T]] + [C.f64(t) for t in (h[0], dh[0], dl)]
    want = O.glr_adjoint(*args)
    for name, x, y, b in zip(("du", "drate", "dh0"), got, want, C.glr_adjoint_bounds(*args)):
        near(x.view(y.shape), y, 5 * b, name)


def test_rate_gradient_of_many_equal_rows(cuda):
    """Every row adds the same to drate, so roundings of a running sum would
    all fall to one side: -s(r) a row, T times.  s(r) has the logistic's error;
    a thread's sum 2 EPS, then ten warps' and 33 CTAs' at most are added."""
    T, D = 8000, 4800  # 800 rows a thread
    g = torch.Generator().manual_seed(0)
    r = torch.randn(D, generator=g).clamp(-4, 4).to(BF16)
    u = torch.zeros(1, T, 3, D, dtype=BF16, device=cuda)
    u[:, :, 0] = r.to(cuda)
    one = torch.ones(1, T, D, device=cuda)
    # no decay: lam = 1 and h = 1 in every row
    _, drate, dh0 = P().pararnn_glr_adjoint(u, torch.zeros(D, device=cuda), one[:, 0].contiguous(), one,
                                            torch.zeros_like(one), dh_last=one[:, 0].contiguous())
    assert torch.equal(dh0, one[:, 0])
    want = -T * O.sigmoid(C.f64(r))
    near(drate, want, (2 * np.abs(C.f64(r)) + 7 + 2 + 43) * C.EPS * np.abs(want), "drate")


def test_look_up_gives_up(cuda):
    """The wait for other CTAs' tiles ends by itself and is reported."""
    from nonlinear_rnn_newton_b200 import capi
    ws = torch.zeros(16384, dtype=torch.uint8, device=cuda)
    assert P().pararnn_selftest_wait_timeout(3, 5_000_000, ws) == capi.ERR_TIMEOUT
    torch.zeros(1, device=cuda).add_(1)
    torch.cuda.synchronize()  # the context is still usable


@pytest.mark.parametrize("which", [2, 3])
def test_failures_are_seen_without_a_workspace(cuda, which):
    """A wait that ran out is told once, by a look that knows no workspace, and
    the calls after it are as before."""
    from nonlinear_rnn_newton_b200 import capi
    u, rate, h0, starts = C.glr_inputs(600, 1, 64, BF16, 0)
    call = lambda: P().pararnn_glr_scan(u[None].to(cuda), rate.to(cuda), h0.to(cuda))[0]
    want = call()
    try:
        P().pararnn_take_failure()  # whatever came before
    except capi.PararnnError:
        pass
    P().pararnn_take_failure(cuda)
    ws = torch.zeros(16384, dtype=torch.uint8, device=cuda)
    assert P().pararnn_selftest_wait_timeout(which, 5_000_000, ws) == capi.ERR_TIMEOUT
    with pytest.raises(capi.PararnnError) as e:
        P().pararnn_take_failure()
    assert e.value.status == capi.ERR_TIMEOUT
    assert torch.equal(call(), want)
    P().pararnn_take_failure(stream=torch.cuda.Stream())


def test_infinite_rate_gradients_stay_infinite(cuda):
    """One infinite gradient, and rows that all add to drate with one sign:
    it is infinite and not NaN, and other channels do not notice."""
    T, D = 3000, 72
    u = torch.randn(1, T, 3, D, device=cuda)
    u[:, :, 2] = -1
    rate, h = 0.05 + 0.1 * torch.rand(D, device=cuda), torch.ones(1, T, D, device=cuda)
    dh = torch.ones(1, T, D, device=cuda)
    want = P().pararnn_glr_adjoint(u, rate, h[:, 0].contiguous(), h, dh)[1]
    dh[0, 1700, 5] = float("inf")
    got = P().pararnn_glr_adjoint(u, rate, h[:, 0].contiguous(), h, dh)[1]
    assert got[5] == -float("inf")
    got[5] = want[5]
    assert torch.equal(got, want) and torch.isfinite(want).all()
