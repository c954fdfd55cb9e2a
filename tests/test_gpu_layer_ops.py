"""GPU parity of the layer operators (gated linear recurrence, RMS norm, 8-bit
product) with the float64 oracle, at the sizes and masks where they can go
wrong.  Tolerances are derived in tests/layer_cases.py or beside the test."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as O
from tests import layer_cases as C

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def P():
    import nonlinear_rnn_newton_b200 as pkg
    return pkg


def near(got, want, bound, what=""):
    got = C.f64(got) if torch.is_tensor(got) else got
    off = np.abs(got - want)
    assert not np.isnan(got).any(), what
    worst = np.unravel_index(np.argmax(off - bound), off.shape)
    assert (off <= bound).all(), f"{what}: off by {off[worst]:.3g} at {worst}, {bound[worst]:.3g} allowed"


# ------------------------------------------------ gated linear recurrence

UNIFORM = [(1, 1, 8), (1, 2, 64), (3, 31, 72), (2, 127, 136), (1, 128, 64), (2, 129, 8), (1, 300, 264), (5, 257, 64),
           (1, 1100, 72), (300, 1, 16), (70, 9, 64), (1, 9000, 8)]
PACKED = [
    (8, 20, [0, 0, 1, 1, 20, 20]),                     # empty ones before, between and behind
    (72, 200, [0, 127, 128, 129, 200]),                # ends on both sides of a tile's
    (64, 700, [5, 6, 6, 300, 301, 640, 690]),          # rows before the first and behind the last
    (136, 520, [0, 64, 128, 256, 384, 512]),
    (64, 1500, [700, 1400]),
    (264, 40, [3, 3, 3]),                              # nothing but empty ones
    (8, 600, list(range(0, 601, 2))),                  # a start in every other row
    (16, 900, [min(900, k // 2) for k in range(0, 2400)]),  # more than are searched in shared memory, half of them empty
]


def check_scan(dev, u, rate, h0, starts, packed, L=None):
    T, _, D = u.shape
    n = len(starts) - 1
    ud = u.to(dev) if packed else u.view(n, L, 3, D).to(dev)
    sd = torch.tensor(starts, dtype=torch.int32, device=dev) if packed else None
    h = torch.full(ud.shape[:-2] + (D,), 7.5, device=dev)
    got, last = P().pararnn_glr_scan(ud, rate.to(dev), h0.to(dev), seq_starts=sd, h=h)
    want, wlast = O.glr_scan(C.f64(u), C.f64(rate), C.f64(h0), starts, h=np.full((T, D), 7.5))
    bound, blast = C.glr_bounds(C.f64(u), C.f64(rate), C.f64(h0), starts)
    near(got.view(T, D), want, bound, "h")  # bound 1e-30 where no sequence is: as it was
    near(last, wlast, blast, "h_last")
    return ud, sd, got


def check_adjoint(dev, u, rate, h0, starts, ud, sd, seed):
    T, _, D = u.shape
    n = len(starts) - 1
    g = torch.Generator().manual_seed(seed + 1)
    h, dh = torch.randn(T, D, generator=g), torch.randn(T, D, generator=g)
    dl = torch.randn(n, D, generator=g)
    du = torch.full(ud.shape, 7.5, device=dev)
    shape = ud.shape[:-2] + (D,)
    gu, gr, g0 = P().pararnn_glr_adjoint(ud, rate.to(dev), h0.to(dev), h.to(dev).view(shape), dh.to(dev).view(shape),
                                         dh_last=dl.to(dev), seq_starts=sd, du=du)
    args = (C.f64(u), C.f64(rate), C.f64(h0), starts, C.f64(h), C.f64(dh), C.f64(dl))
    wu, wr, w0, _ = O.glr_adjoint(*args)
    out = np.ones(T, bool)
    out[starts[0]:starts[-1]] = False
    wu[out] = 7.5
    bu, br, b0 = C.glr_adjoint_bounds(*args)
    near(gu.view(T, 3, D), wu, bu, "du")
    near(gr, wr, br, "drate")
    near(g0, w0, b0, "dh0")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,L,D", UNIFORM)
def test_recurrence_uniform(cuda, n, L, D, dtype):
    u, rate, h0, starts = C.glr_inputs(n * L, n, D, dtype, seed=n + L + D)
    ud, _, _ = check_scan(cuda, u, rate, h0, starts, False, L)
    check_adjoint(cuda, u, rate, h0, starts, ud, None, n + L + D)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("k", range(len(PACKED)))
def test_recurrence_packed(cuda, k, dtype):
    D, T, starts = PACKED[k]
    u, rate, h0, _ = C.glr_inputs(T, len(starts) - 1, D, dtype, seed=k, starts=starts)
    ud, sd, _ = check_scan(cuda, u, rate, h0, starts, True)
    check_adjoint(cuda, u, rate, h0, starts, ud, sd, k)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,T,starts", [(72, 700, [0, 700]), (64, 1500, [0, 1100, 1100, 1101, 1490]), PACKED[3]])
def test_recurrence_slow_rates(cuda, D, T, starts, dtype):
    """Every rate below 1/8: the decays come from the series alone."""
    u, rate, h0, _ = C.glr_inputs(T, len(starts) - 1, D, dtype, seed=T, starts=starts, fast=False)
    ud, sd, _ = check_scan(cuda, u, rate, h0, starts, True)
    check_adjoint(cuda, u, rate, h0, starts, ud, sd, T)


def test_recurrence_optional_arguments(cuda):
    u, rate, h0, starts = C.glr_inputs(60, 2, 16, BF16, 0)
    ud, rd = u.view(2, 30, 3, 16).to(cuda), rate.to(cuda)
    h, last = P().pararnn_glr_scan(ud, rd)
    z = torch.zeros(2, 16, device=cuda)
    h2, last2 = P().pararnn_glr_scan(ud, rd, z)
    assert torch.equal(h, h2) and torch.equal(last, last2) and torch.equal(last, h[:, -1])
    h3, none = P().pararnn_glr_scan(ud, rd, want_last=False)
    assert none is None and torch.equal(h, h3)
    dh = torch.randn(h.shape, device=cuda)
    a = P().pararnn_glr_adjoint(ud, rd, None, h, dh)
    b = P().pararnn_glr_adjoint(ud, rd, z, h, dh, dh_last=z)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = P().pararnn_glr_adjoint(ud, rd, None, h, dh, want_dh0=False)
    assert c[2] is None and torch.equal(c[0], a[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_recurrence_other_sequences_do_not_matter(cuda, bad):
    """NaN, infinities and the type's lowest value in other sequences, and in rows of none, change nothing."""
    starts = [40, 300, 301, 640, 690]
    T, D = 700, 64
    u, rate, h0, _ = C.glr_inputs(T, 4, D, BF16, 1, starts)
    g = torch.Generator().manual_seed(2)
    h, dh, dl = (torch.randn(s, D, generator=g) for s in (T, T, 4))
    value = torch.finfo(BF16).min if bad == "lowest" else bad
    for s in range(4):
        lo, hi = starts[s], starts[s + 1]
        v = [x.clone() for x in (u, h0, h, dh, dl)]
        for x in v[0], v[2], v[3]:
            x[:lo], x[hi:] = value, value
        for x in v[1], v[4]:
            x[:s], x[s + 1:] = value, value
        got = []
        for x in ((u, h0, h, dh, dl), v):
            a, b, c, d, e = (t.to(cuda) for t in x)
            sd = torch.tensor(starts, dtype=torch.int32, device=cuda)
            y, last = P().pararnn_glr_scan(a, rate.to(cuda), b, seq_starts=sd)
            du, _, dh0 = P().pararnn_glr_adjoint(a, rate.to(cuda), b, c, d, dh_last=e, seq_starts=sd)
            got.append((y[lo:hi], last[s], du[lo:hi], dh0[s]))
        assert all(torch.equal(x, y) for x, y in zip(*got)), s


@pytest.mark.parametrize("gate", ["lowest", "-inf"])
def test_recurrence_shut_gate_holds_the_state(cuda, gate):
    u, rate, h0, starts = C.glr_inputs(300, 1, 64, BF16, 5)
    u[100:250, 0] = torch.finfo(BF16).min if gate == "lowest" else -float("inf")
    h, _ = P().pararnn_glr_scan(u[None].to(cuda), rate.to(cuda), h0.to(cuda))
    # the shut rows' maps are (1, 0) exactly, and folding with those is exact: each
    # of their states is row 99's up to how the rows before were folded, which
    # leaves every one of them within row 99's bound of the same number
    want, _ = O.glr_scan(C.f64(u), C.f64(rate), C.f64(h0), starts)
    bound, _ = C.glr_bounds(C.f64(u), C.f64(rate), C.f64(h0), starts)
    near(h[0, 100:250], np.repeat(want[99:100], 150, 0), np.repeat(bound[99:100], 150, 0))
    dh = torch.randn(1, 300, 64, device=cuda)
    du, drate, dh0 = P().pararnn_glr_adjoint(u[None].to(cuda), rate.to(cuda), h0.to(cuda), h, dh)
    assert torch.isfinite(du).all() and torch.isfinite(drate).all() and torch.isfinite(dh0).all()
    assert not du[0, 100:250].any()
    zero = P().pararnn_glr_adjoint(u[None].to(cuda), torch.zeros_like(rate).to(cuda), h0.to(cuda), h, dh)
    assert all(torch.isfinite(x).all() for x in zero)


def test_recurrence_adjoint_is_the_slope_of_the_scan(cuda):
    """Against differences of the 64-bit recurrence: along a direction v the
    loss changes by (gradient . v), up to the 1e-6 that the differences have
    and the gradient's own bound."""
    starts = [0, 50, 50, 51, 180]
    u, rate, h0, _ = C.glr_inputs(180, 4, 8, F32, 11, starts)
    g = torch.Generator().manual_seed(12)
    dh, dl = torch.randn(180, 8, generator=g), torch.randn(4, 8, generator=g)
    sd = torch.tensor(starts, dtype=torch.int32, device=cuda)
    h, _ = P().pararnn_glr_scan(u.to(cuda), rate.to(cuda), h0.to(cuda), seq_starts=sd)
    grads = P().pararnn_glr_adjoint(u.to(cuda), rate.to(cuda), h0.to(cuda), h, dh.to(cuda), dh_last=dl.to(cuda),
                                    seq_starts=sd)
    x = [C.f64(t) for t in (u, rate, h0)]
    bounds = C.glr_adjoint_bounds(*x, starts, C.f64(h), C.f64(dh), C.f64(dl))
    hb, _ = C.glr_bounds(*x, starts)

    def loss(u, rate, h0):
        h, last = O.glr_scan(u, rate, h0, starts)
        return (h * C.f64(dh)).sum() + (last * C.f64(dl)).sum()

    r = np.random.default_rng(0)
    for k in range(3):
        v = r.standard_normal(x[k].shape) * (x[k] if k == 1 else 1)
        hi, lo = list(x), list(x)
        hi[k], lo[k] = x[k] + 1e-6 * v, x[k] - 1e-6 * v
        slope = (loss(*hi) - loss(*lo)) / 2e-6
        # the adjoint reads the states as the scan rounded them
        extra = np.abs(hb).sum() * np.abs(C.f64(dh)).max() * np.abs(v).max()
        assert abs(slope - (C.f64(grads[k]) * v).sum()) <= 1e-6 * abs(slope) + 1e-6 + (bounds[k] * np.abs(v)).sum() + extra


@pytest.mark.parametrize("B,D,dtype", [(1, 8, F32), (3, 136, BF16), (256, 64, BF16), (5, 1000, F32)])
def test_step_matches_scan_of_one_row(cuda, B, D, dtype):
    u, rate, h0, starts = C.glr_inputs(B, B, D, dtype, 3)
    want, _ = O.glr_scan(C.f64(u), C.f64(rate), C.f64(h0), starts)
    bound, _ = C.glr_bounds(C.f64(u), C.f64(rate), C.f64(h0), starts)
    state = h0.to(cuda)
    near(P().pararnn_glr_step(u.to(cuda), rate.to(cuda), state), want, bound)
    out = P().pararnn_glr_step(u.to(cuda), rate.to(cuda), state, h_next=state)
    assert out is state
    near(state, want, bound)
    none = P().pararnn_glr_step(u.to(cuda), rate.to(cuda))
    assert torch.equal(none, P().pararnn_glr_step(u.to(cuda), rate.to(cuda), torch.zeros_like(state)))


def test_prefill_then_steps(cuda):
    """A prompt through the scan, then tokens one by one, is the scan of both."""
    B, L, D = 3, 140, 72
    u, rate, h0, _ = C.glr_inputs(B * L, B, D, BF16, 8)
    starts = [L * k for k in range(B + 1)]
    want, _ = O.glr_scan(C.f64(u), C.f64(rate), C.f64(h0), starts)
    bound, _ = C.glr_bounds(C.f64(u), C.f64(rate), C.f64(h0), starts)
    ud, rd = u.view(B, L, 3, D).to(cuda), rate.to(cuda)
    _, state = P().pararnn_glr_scan(ud[:, :130].contiguous(), rd, h0.to(cuda))
    for t in range(130, L):
        P().pararnn_glr_step(ud[:, t].contiguous(), rd, state, h_next=state)
        near(state, want.reshape(B, L, D)[:, t], bound.reshape(B, L, D)[:, t])


def test_recurrence_repeats_bit_for_bit(cuda):
    u, rate, h0, _ = C.glr_inputs(6000, 2, 136, BF16, 1)
    ud, rd, hd = u.view(2, 3000, 3, 136).to(cuda), rate.to(cuda), h0.to(cuda)
    dh = torch.randn(2, 3000, 136, device=cuda)
    first = None
    for _ in range(5):
        h, last = P().pararnn_glr_scan(ud, rd, hd)
        now = (h, last) + P().pararnn_glr_adjoint(ud, rd, hd, h, dh)
        first = first or now
        assert all(torch.equal(x, y) for x, y in zip(first, now))


# --------------------------------------------------------------- RMS norm

@pytest.mark.parametrize("T,D", [(1, 8), (1, 2048), (3, 16), (50, 120), (2, 128), (37, 1000), (5, 2064), (3, 4104),
                                 (2, 16384), (3000, 272)])
@pytest.mark.parametrize("x,res,y", [(F32, BF16, E4M3), (BF16, BF16, BF16), (BF16, None, F32), (F32, F32, F32),
                                     (BF16, F32, E4M3), (F32, None, E4M3)],
                         ids=lambda t: "none" if t is None else str(t)[6:])
def test_norm(cuda, T, D, x, res, y):
    if y == E4M3 and D % 16:
        pytest.skip("8 bits need a multiple of 16")
    g = torch.Generator().manual_seed(T + D)
    xs = torch.randn(T, D, generator=g).to(x)
    rs = None if res is None else (2 * torch.randn(T, D, generator=g)).to(res)
    w = 1 + 0.1 * torch.randn(D, generator=g)
    if T > 1:
        xs[1] = 0  # a row of nothing
        if res is not None:
            rs[1] = 0
    got, scale, total, rstd = P().pararnn_rms_norm(xs.to(cuda), w.to(cuda), residual=None if rs is None else rs.to(cuda),
                                                   eps=1e-5, out_dtype=y)
    want, v, wr = O.rms_norm(C.f64(xs), None if rs is None else C.f64(rs), C.f64(w), 1e-5)
    # v rounded (EPS, twice that in its square), the square, a thread's 32 sums
    # and 9 more over threads: 45 EPS of the mean, half of it in rstd, the
    # division, the root and the sum with eps 4
    rel = 30 * C.EPS
    near(rstd, wr, rel * wr, "rstd")
    if res is None:
        assert total is None
    else:
        # v is rounded to 32 bits, then to the residual's type
        near(total, v, (C.HALF[res] + (C.EPS if res == BF16 else 0)) * np.abs(v) * 1.01, "sum")
    size = np.abs(want) * (rel + 4 * C.EPS) + 2 * C.EPS * np.abs(w.double().numpy()) * wr[:, None] * (
        np.abs(C.f64(xs)) + (0 if rs is None else np.abs(C.f64(rs))))
    if y != E4M3:
        near(got, want, size + C.HALF[y] * np.abs(want) * 1.01, "y")
        return
    ws = O.block_scales(want, 1)
    near(scale, ws, O.block_scales(size + np.abs(want), 1) - ws + 2 * C.EPS * ws, "scale")
    sc = O.spread(C.f64(scale), 1, T, D)
    # half a step of the value, or of the smallest numbers' (2^-9)
    near(C.f64(got) * sc, want, size * 1.1 + np.maximum(C.HALF[y] * np.abs(want) * 1.001, 2.0 ** -10 * sc), "y")


def test_norm_in_place_and_given_outputs(cuda):
    x, r, w = torch.randn(5, 64, device=cuda), torch.randn(5, 64, device=cuda), torch.randn(64, device=cuda)
    y, _, s, rstd = P().pararnn_rms_norm(x, w, residual=r, out_dtype=BF16)
    r2 = r.clone()
    y2, _, s2, _ = P().pararnn_rms_norm(x, w, residual=r2, out_dtype=BF16, sum=r2)
    assert s2 is r2 and torch.equal(s, s2) and torch.equal(y, y2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_bad_values_stay_in_their_row(cuda, bad):
    x, w = torch.randn(9, 256, device=cuda), torch.ones(256, device=cuda)
    y, scale, _, _ = P().pararnn_rms_norm(x, w, out_dtype=E4M3)
    x[4, 200] = bad
    y2, scale2, _, _ = P().pararnn_rms_norm(x, w, out_dtype=E4M3)
    rows = [k for k in range(9) if k != 4]
    assert torch.equal(y.float()[rows], y2.float()[rows]) and torch.equal(scale[rows], scale2[rows])
    assert torch.isnan(y2.float()[4, 128:] * scale2[4, 1]).all()


@pytest.mark.parametrize("T,D", [(1, 8), (3, 16), (40, 120), (37, 1000), (5, 2064), (3, 4104), (2, 16384), (3000, 272),
                                 (700, 2048)])
@pytest.mark.parametrize("y,v,with_dv", [(BF16, BF16, True), (F32, F32, False), (F32, BF16, False), (BF16, F32, True)],
                         ids=lambda t: str(t)[6:] if isinstance(t, torch.dtype) else "dsum" if t else "alone")
def test_norm_adjoint(cuda, T, D, y, v, with_dv):
    g = torch.Generator().manual_seed(T + D)
    dy, vs = torch.randn(T, D, generator=g).to(y), (2 * torch.randn(T, D, generator=g)).to(v)
    dv = torch.randn(T, D, generator=g).to(v) if with_dv else None
    w = 1 + 0.1 * torch.randn(D, generator=g)
    rstd = (1 / (vs.double().square().mean(1) + 1e-5).sqrt()).float()
    args = [t.to(cuda) for t in (dy, vs, w, rstd)]
    dx, dw = P().pararnn_rms_norm_adjoint(*args, dsum=None if dv is None else dv.to(cuda))
    a = [C.f64(t) for t in (dy, vs, w, rstd)]
    wx, ww = O.rms_norm_adjoint(a[0], a[1], a[2], a[3], None if dv is None else C.f64(dv))
    n, gg = a[1] * a[3][:, None], a[0] * a[2]
    mean = (np.abs(gg * n)).mean(1, keepdims=True)
    # the mean of g n: two roundings a term, then 32 + 9 sums; three more at the end
    size = a[3][:, None] * (np.abs(gg) * 4 + np.abs(n) * mean * 50) * C.EPS + 2 * C.EPS * np.abs(wx)
    near(dx, wx, size + C.HALF[v] * np.abs(wx) * 1.01, "dx")
    # a column's sum: a thread's rows, the CTAs' parts: at most T additions, and two roundings a term
    near(dw, ww, (T + 20) * C.EPS * np.abs(a[0] * n).sum(0), "dw")
    if with_dv:
        place = dv.to(cuda)
        again, _ = P().pararnn_rms_norm_adjoint(*args, dsum=place, dx=place)
        assert again is place and torch.equal(again, dx)


# ---------------------------------------------------------- 8-bit product

@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K,rows", [(1, 16, 1), (3, 128, 1), (50, 144, 1), (37, 1040, 1), (300, 272, 1), (1, 16, 128),
                                      (128, 128, 128), (129, 144, 128), (300, 1040, 128)])
def test_quantize_is_exact(cuda, M, K, rows, dtype):
    """Scales and values bit for bit: the largest magnitude is exact, the two
    divisions are IEEE's, and the rounding is to nearest even."""
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(4 * torch.randn(M, 1, generator=g))).to(dtype)
    x[0, :16] = 0
    if M > 2:
        x[2] = 0  # an empty row
        x[1, :] *= 1e-30
    q, scale = P().pararnn_fp8_quantize(x.to(cuda), block_rows=rows)
    pad = torch.nn.functional.pad(x.float(), (0, -K % 128, 0, -M % rows))
    b = pad.view(pad.shape[0] // rows, rows, -1, 128)
    want = torch.clamp(b.abs().amax((1, 3)) / torch.tensor(448.0), min=2.0 ** -126)
    z = (b / want[:, None, :, None]).reshape(pad.shape)[:M, :K]
    assert torch.equal(scale.cpu(), want)
    assert torch.equal(q.cpu().float(), z.to(E4M3).float())
    assert np.array_equal(C.f64(q.float()), O.e4m3(C.f64(z)))


def test_quantize_is_exact_beside_the_middles(cuda):
    """Numbers at the middle between two e4m3 values times the scale, and up to
    six steps of fp32 to both sides of it, at scales of any mantissa: the value
    is that of the rounded quotient, bit for bit."""
    g = torch.Generator().manual_seed(3)
    grid = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double()
    middles = (grid[1:] + grid[:-1]) / 2
    scale = (1 + torch.rand(600, generator=g)) * torch.exp2(torch.randint(-120, 118, (600,), generator=g).float())
    x = (middles[None] * scale.double()[:, None]).float()
    x = (x.view(torch.int32) + torch.randint(-6, 7, x.shape, generator=g, dtype=torch.int32)).view(torch.float32)
    x = torch.cat([448 * scale[:, None], x, -x[:, :1]], 1)  # the first column sets the scale
    want = x.abs().amax(1) / torch.tensor(448.0)
    q, s = P().pararnn_fp8_quantize(x.contiguous().to(cuda))
    assert x.shape[1] == 128 and torch.equal(s.cpu()[:, 0], want)
    assert torch.equal(q.cpu().float(), (x / want[:, None]).to(E4M3).float())


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_bad_values_stay_in_their_block(cuda, rows, bad):
    x = torch.randn(256, 384, device=cuda)
    q, s = P().pararnn_fp8_quantize(x, block_rows=rows)
    x[130, 140] = bad
    q2, s2 = P().pararnn_fp8_quantize(x, block_rows=rows)
    full = lambda q, s: q.float() * s.repeat_interleave(rows, 0).repeat_interleave(128, 1)
    y, y2 = full(q, s), full(q2, s2)
    lo, hi = (130, 131) if rows == 1 else (128, 256)
    assert torch.isnan(y2[lo:hi, 128:256]).all()
    y2[lo:hi, 128:256] = y[lo:hi, 128:256]
    assert torch.equal(y, y2)


SIZES = [(1, 8, 16), (1, 200, 128), (3, 136, 144), (16, 256, 512), (17, 264, 1040), (64, 1304, 272), (65, 128, 128),
         (100, 392, 2048), (127, 256, 640), (128, 128, 384), (129, 264, 400), (200, 1000, 1104), (300, 520, 4096),
         (513, 2056, 656), (1000, 768, 256), (300, 8200, 1040), (2570, 2056, 400)]


@pytest.mark.parametrize("u", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_project(cuda, M, N, K, u):
    check_project(cuda, M, N, K, u, bias=(M + N) % 16 != 0)


def check_project(cuda, M, N, K, u, bias):
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    w = torch.randn(N, K, generator=g) * K ** -0.5
    xq, xs = P().pararnn_fp8_quantize(x.to(cuda), block_rows=1)
    wq, ws = P().pararnn_fp8_quantize(w.to(cuda), block_rows=128)
    # scales of any size, not those of one quantiser alone
    xs, ws = xs * (0.5 + torch.rand(xs.shape, generator=g)).to(cuda), ws * (0.5 + torch.rand(ws.shape, generator=g)).to(cuda)
    b = torch.randn(N, generator=g) if bias else None
    out = torch.full((M, N), 7.5, dtype=u, device=cuda)
    got = P().pararnn_fp8_project(xq, xs, wq, ws, bias=None if b is None else b.to(cuda), out_dtype=u, u=out)
    want, size = O.fp8_project(C.f64(xq.float()), C.f64(xs), C.f64(wq.float()), C.f64(ws), None if b is None else C.f64(b))
    # a block's 128 products (exact in fp32) added in any order, each sum
    # rounded or cut: 2 EPS a sum; then the blocks' (a scale's product, the
    # term's, the sum's rounding each) and the bias
    rel = (2 * 128 + 4 * ((K + 127) // 128) + 4) * C.EPS
    near(got, want, rel * size + C.EPS * np.abs(want) + C.HALF[u] * np.abs(want) * 1.01, "u")


def test_project_bad_values_stay_in_their_row(cuda):
    x, w = torch.randn(140, 256, device=cuda), torch.randn(136, 256, device=cuda)
    wq, ws = P().pararnn_fp8_quantize(w, block_rows=128)
    xq, xs = P().pararnn_fp8_quantize(x)
    u = P().pararnn_fp8_project(xq, xs, wq, ws)
    x[77, 3], x[130, 200] = float("nan"), float("inf")
    xq, xs = P().pararnn_fp8_quantize(x)
    u2 = P().pararnn_fp8_project(xq, xs, wq, ws)
    assert torch.isnan(u2[77]).all() and torch.isnan(u2[130]).all()
    rows = [k for k in range(140) if k not in (77, 130)]
    assert torch.equal(u[rows], u2[rows])


def test_project_of_nothing_is_the_bias(cuda):
    xq, xs = P().pararnn_fp8_quantize(torch.zeros(5, 128, device=cuda))
    wq, ws = P().pararnn_fp8_quantize(torch.zeros(16, 128, device=cuda), block_rows=128)
    b = torch.randn(16, device=cuda)
    assert torch.equal(P().pararnn_fp8_project(xq, xs, wq, ws, bias=b, out_dtype=F32), b.expand(5, 16))


# ----------------------------------------------------- together, and streams

def layer(x, res, w, wq, ws, bias, rate, h0, state=None):
    """One layer of a residual stream: norm, projection, recurrence (the scan,
    or the decode step from `state`)."""
    y, sc, res, rstd = P().pararnn_rms_norm(x, w, residual=res, out_dtype=E4M3)
    u = P().pararnn_fp8_project(y, sc, wq, ws, bias=bias)
    u = u.view(u.shape[:-1] + (3, rate.shape[0]))
    if state is None:
        return P().pararnn_glr_scan(u, rate, h0) + (res, u, rstd)
    return P().pararnn_glr_step(u, rate, state), res, u


def test_layers_together(cuda):
    """Two layers over a prompt, then token by token: the decode path gives the
    states of the whole run.  Rows do not depend on their neighbours in the norm
    and the product, so the gates are equal but for the order of the product's
    sums (other tile shapes): one bf16 step of the gates at most."""
    B, L, D = 2, 70, 128
    g = torch.Generator().manual_seed(0)
    x = torch.randn(B, L, D, generator=g).to(cuda)
    layers = []
    for _ in range(2):
        wq, ws = P().pararnn_fp8_quantize((torch.randn(3 * D, D, generator=g) * D ** -0.5).to(cuda), block_rows=128)
        layers.append((torch.ones(D, device=cuda), wq, ws, torch.randn(3 * D, generator=g).to(cuda),
                       torch.rand(D, generator=g).to(cuda) * 0.1))
    h0 = torch.zeros(B, D, device=cuda)

    def prompt(n):
        h, res, out, ends = x[:, :n].contiguous(), torch.zeros(B, n, D, dtype=BF16, device=cuda), [], []
        for w, wq, ws, b, rate in layers:
            h, last, res, u, _ = layer(h, res, w, wq, ws, b, rate, h0)
            out.append(u)
            ends.append(last)
        return out, ends

    whole, whole_ends = prompt(L)
    _, states = prompt(60)
    for t in range(60, L):
        h, res = x[:, t].contiguous(), torch.zeros(B, D, dtype=BF16, device=cuda)
        for k, (w, wq, ws, b, rate) in enumerate(layers):
            h, res, u = layer(h, res, w, wq, ws, b, rate, None, states[k])
            states[k] = h
            if k == 0:
                off = (u.float() - whole[0][:, t].float()).abs()
                assert (off <= 2 ** -7 * whole[0][:, t].float().abs() + 1e-5).all()
    assert torch.allclose(states[0], whole_ends[0], rtol=0, atol=2 ** -6)


def test_other_stream_and_graph(cuda):
    """On a stream of its own and replayed from a graph, twice, with new inputs in the same buffers."""
    B, L, D = 2, 900, 64
    w = torch.ones(D, device=cuda)
    wq, ws = P().pararnn_fp8_quantize(torch.randn(3 * D, D, device=cuda) * D ** -0.5, block_rows=128)
    rate, h0 = torch.rand(D, device=cuda) * 0.1, torch.randn(B, D, device=cuda)
    x, res = torch.randn(B, L, D, device=cuda), torch.randn(B, L, D, device=cuda).to(BF16)
    dh = torch.randn(B, L, D, device=cuda)

    def run():
        y, sc, s, rstd = P().pararnn_rms_norm(x, w, residual=res, out_dtype=E4M3)
        u = P().pararnn_fp8_project(y, sc, wq, ws).view(B, L, 3, D)
        h, last = P().pararnn_glr_scan(u, rate, h0)
        du, dr, d0 = P().pararnn_glr_adjoint(u, rate, h0, h, dh)
        dx, dw = P().pararnn_rms_norm_adjoint(du.view(B, L, 3 * D)[..., :D].contiguous(), s, w, rstd, dsum=res)
        return s, u, h, last, du, dr, d0, dx, dw

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(2):
        torch.manual_seed(seed)
        x.normal_()
        dh.normal_()
        want = run()
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_explicit_stream(cuda):
    """A call on a given stream: its outputs and workspace are that stream's, so
    work of the current stream that starts meanwhile does not meet them."""
    B, L, D = 1, 20000, 256
    u, rate, h0, _ = C.glr_inputs(B * L, B, D, BF16, 3)
    ud, rd, hd = u.view(B, L, 3, D).to(cuda), rate.to(cuda), h0.to(cuda)
    x, w = torch.randn(L, D, device=cuda), torch.ones(D, device=cuda)
    wq, ws = P().pararnn_fp8_quantize(torch.randn(136, D, device=cuda), block_rows=128)
    dh = torch.randn(B, L, D, device=cuda)

    def run(stream):
        y, sc, _, rstd = P().pararnn_rms_norm(x, w, out_dtype=E4M3, stream=stream)
        q, qs = P().pararnn_fp8_quantize(x, stream=stream)
        g = P().pararnn_fp8_project(y, sc, wq, ws, stream=stream)
        h, last = P().pararnn_glr_scan(ud, rd, hd, stream=stream)
        du, dr, d0 = P().pararnn_glr_adjoint(ud, rd, hd, h, dh, stream=stream)
        dx, dw = P().pararnn_rms_norm_adjoint(x, x, w, rstd, stream=stream)
        n = P().pararnn_glr_step(ud[:, 0].contiguous(), rd, hd, stream=stream)
        return y.float(), sc, rstd, q.float(), qs, g, h, last, du, dr, d0, dx, dw, n

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = run(side)
        for n in (256, L * D * 4, 1 << 20):  # what the current stream does meanwhile
            torch.full((n,), 255, dtype=torch.uint8, device=cuda)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del got


def test_outcome_is_read_from_the_workspace(cuda):
    u, rate, h0, _ = C.glr_inputs(4000, 1, 64, BF16, 0)
    ws = torch.full((P().pararnn_glr_adjoint_workspace_size(4000, 1, 64),), 255, dtype=torch.uint8, device=cuda)
    ud, rd, hd = u[None].to(cuda), rate.to(cuda), h0.to(cuda)
    h, _ = P().pararnn_glr_scan(ud, rd, hd, workspace=ws)
    assert P().pararnn_read_result(ws)[0] == 0
    ws.fill_(255)
    P().pararnn_glr_adjoint(ud, rd, hd, h, h, workspace=ws)
    assert P().pararnn_read_result(ws)[0] == 0
    q, s = P().pararnn_fp8_quantize(torch.randn(300, 128, device=cuda))
    wq, wsc = P().pararnn_fp8_quantize(torch.randn(136, 128, device=cuda), block_rows=128)
    for rows in (3, 300):  # both forms of the product
        ws.fill_(255)
        P().pararnn_fp8_project(q[:rows], s[:rows], wq, wsc, workspace=ws[:256])
        assert P().pararnn_read_result(ws[:256])[0] == 0


@pytest.mark.slow
def test_offsets_beyond_32_bits(cuda):
    """Arrays of more than 2^31 elements: their ends are what a call on the ends
    alone gives."""
    T, D = 800_000, 1024  # 2.46e9 gates
    u = torch.empty(1, T, 3, D, dtype=BF16, device=cuda)
    for k in range(0, T, 100_000):
        u[:, k:k + 100_000].normal_()
    rate, dh = torch.rand(D, device=cuda) * 0.1 + 0.01, torch.randn(1, T, D, device=cuda)
    h, last = P().pararnn_glr_scan(u, rate)
    cut = T - 5000
    want, wlast = P().pararnn_glr_scan(u[:, cut:].contiguous(), rate, h[:, cut - 1].contiguous())
    # the same rows folded from other tile bounds: both within the recurrence's
    # bound, 8 EPS of the state's envelope (below 30 here) a row over 1 / (1 - a)
    # <= 200 rows' memory
    assert (h[:, cut:] - want).abs().max() <= 2 * 8 * C.EPS * 30 * 200 and torch.equal(last, h[:, -1])
    du, drate, dh0 = P().pararnn_glr_adjoint(u, rate, None, h, dh)
    wu, _, wg = P().pararnn_glr_adjoint(u[:, cut:].contiguous(), rate, h[:, cut - 1].contiguous(),
                                        h[:, cut:].contiguous(), dh[:, cut:].contiguous())
    scale = wu.abs().amax((0, 1))
    assert ((du[:, cut:] - wu).abs().amax((0, 1)) <= 1e-3 * scale).all()
    assert torch.isfinite(du[:, :1000]).all() and torch.isfinite(drate).all() and torch.isfinite(dh0).all()
    del du, wu, dh, want
    flat = u.view(T * 3, D)
    # 4000 rows: fewer are spread over more threads a row (and, in the product,
    # over other tiles), which sums in another order; from 1184 rows of this
    # width on the rows do not depend on how many there are
    y, sc, _, rstd = P().pararnn_rms_norm(flat, torch.ones(D, device=cuda), out_dtype=E4M3)
    y2, sc2, _, rstd2 = P().pararnn_rms_norm(flat[-4000:].contiguous(), torch.ones(D, device=cuda), out_dtype=E4M3)
    assert torch.equal(y[-4000:].float(), y2.float()) and torch.equal(sc[-4000:], sc2)
    q, qs = P().pararnn_fp8_quantize(flat)
    q2, qs2 = P().pararnn_fp8_quantize(flat[-4000:].contiguous())
    assert torch.equal(q[-4000:].float(), q2.float()) and torch.equal(qs[-4000:], qs2)
    del u, flat, h, y
    wq, ws = P().pararnn_fp8_quantize(torch.randn(1024, 1024, device=cuda), block_rows=128)
    g = P().pararnn_fp8_project(q, qs, wq, ws)  # 2.46e9 outputs
    assert torch.equal(g[-4000:], P().pararnn_fp8_project(q2, qs2, wq, ws))


def test_barrier_wait_gives_up(cuda):
    """The waits of the scans and the product end by themselves and are reported."""
    from nonlinear_rnn_newton_b200 import capi
    ws = torch.zeros(16384, dtype=torch.uint8, device=cuda)
    st = capi.lib.pararnn_selftest_wait_timeout(2, 5_000_000, ws.data_ptr(), ws.numel(), None)
    assert st == capi.ERR_TIMEOUT
    torch.zeros(1, device=cuda).add_(1)
    torch.cuda.synchronize()  # the context is still usable


def test_two_streams_at_once(cuda):
    """Two recurrences at the same time, each with a workspace of its own."""
    ins = []
    for k in range(2):
        u, rate, h0, _ = C.glr_inputs(20000, 1, 264, BF16, k)
        ins.append((u[None].to(cuda), rate.to(cuda), h0.to(cuda)))
    want = [P().pararnn_glr_scan(*a) for a in ins]
    dh = torch.randn_like(want[0][0])
    back = [P().pararnn_glr_adjoint(*a, h[0], dh) for a, h in zip(ins, want)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got, gback = [None, None], [None, None]
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = P().pararnn_glr_scan(*ins[k])
                gback[k] = P().pararnn_glr_adjoint(*ins[k], want[k][0], dh)
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(want[k] + back[k], got[k] + gback[k]))
