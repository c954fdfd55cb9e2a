"""What is measured of the layer operators: the gated linear recurrence (scan,
adjoint, decode step), the RMS norm with the residual's addition and its
adjoint, and the 8-bit product with a scale for each block of 128.

`run` computes each operator from elementary torch operations in 32 bits, or,
where `own` is true, through the package's entry points."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
BLOCK = 128      # columns that share a scale (and rows, for a weight)
TOP = 448.0      # largest e4m3 value
LEAST = 2.0 ** -126


def listed():
    return [
        # one generated token for 256 sequences
        {"name": "step_B256_D2048", "kind": "step", "B": 256, "D": 2048, "u": "bf16"},
        # a short prompt batch of unequal lengths (some empty, some of one token), fp32 gates
        {"name": "scan_packed_small", "kind": "scan", "T": 1501, "seqs": 9, "packed": True, "D": 264, "u": "f32"},
        # the framework's batch of eight sequences
        {"name": "scan_B8_L4096_D1024", "kind": "scan", "T": 8 * 4096, "seqs": 8, "packed": False, "D": 1024, "u": "bf16"},
        # the framework's longest sequence
        {"name": "scan_B1_L65536_D2048", "kind": "scan", "T": 65536, "seqs": 1, "packed": False, "D": 2048, "u": "bf16"},
        # documents packed into one training batch
        {"name": "adjoint_packed_T16384_D1024", "kind": "adjoint", "T": 16384, "seqs": 37, "packed": True, "D": 1024,
         "u": "bf16"},
        # the framework's training batch
        {"name": "adjoint_B4_L16384_D2048", "kind": "adjoint", "T": 4 * 16384, "seqs": 4, "packed": False, "D": 2048,
         "u": "bf16"},
        # the norm before a projection while generating: eight tokens
        {"name": "norm_T8_D2048_e4m3", "kind": "norm", "T": 8, "D": 2048, "x": "f32", "res": "bf16", "y": "e4m3"},
        # the norm before a projection over a whole batch, fp32 states joining a bf16 stream
        {"name": "norm_T32768_D2048_e4m3", "kind": "norm", "T": 32768, "D": 2048, "x": "f32", "res": "bf16", "y": "e4m3"},
        # its backward pass in training
        {"name": "norm_adjoint_T32768_D2048", "kind": "norm_adjoint", "T": 32768, "D": 2048, "x": "bf16", "y": "bf16"},
        # the gates of sixteen generated tokens: the weight is read once
        {"name": "product_M16_N6144_K2048", "kind": "product", "M": 16, "N": 6144, "K": 2048, "bias": True, "u": "bf16"},
        # a training step's forward product at odd sizes, weights just updated: both operands quantised in the call
        {"name": "quantized_product_odd", "kind": "quantized_product", "M": 4133, "N": 1304, "K": 1104, "bias": False,
         "u": "f32", "x": "bf16"},
        # the gates of a whole batch
        {"name": "product_M32768_N6144_K2048", "kind": "product", "M": 32768, "N": 6144, "K": 2048, "bias": True,
         "u": "bf16"},
    ]


def draw(rng):
    def log(lo, hi, of=1):
        return max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / of)) * of

    kind = rng.choice(["step", "scan", "adjoint", "norm", "norm_adjoint", "product", "quantized_product"])
    if kind == "step":
        return {"kind": kind, "B": log(1, 512), "D": log(64, 4096, 8), "u": rng.choice(["bf16", "f32"])}
    if kind in ("scan", "adjoint"):
        D = log(64, 2048, 8)
        most = min(65536, 65536 * 1024 // D)
        packed = rng.random() < 0.5
        seqs = log(1, 64)
        length = max(1, log(64, most) // seqs)
        T = seqs * length + (rng.randrange(seqs + 1) if packed else 0)
        return {"kind": kind, "T": T, "seqs": seqs, "packed": packed, "D": D, "u": rng.choice(["bf16", "bf16", "f32"])}
    if kind == "norm":
        y = rng.choice(["e4m3", "e4m3", "bf16", "f32"])
        return {"kind": kind, "T": log(1, 16384), "D": log(64, 4096, 16), "x": rng.choice(["bf16", "f32"]),
                "res": rng.choice(["bf16", "f32", "none"]), "y": y}
    if kind == "norm_adjoint":
        return {"kind": kind, "T": log(16, 16384), "D": log(64, 4096, 8), "x": rng.choice(["bf16", "f32"]),
                "y": rng.choice(["bf16", "f32"])}
    case = {"kind": kind, "M": log(1, 16384), "N": log(64, 6144, 8), "K": log(128, 4096, 16),
            "bias": rng.random() < 0.5, "u": rng.choice(["bf16", "f32"])}
    return case | ({"x": rng.choice(["bf16", "f32"])} if kind == "quantized_product" else {})


# ------------------------------------------------------------------- inputs

def starts_of(case, seed):
    """Offsets of a packed batch: lengths of an exponential law, a few of them nought or one."""
    n, T = case["seqs"], case["T"]
    g = torch.Generator().manual_seed(seed + 7)
    part = torch.empty(n, dtype=torch.float64).exponential_(generator=g)
    ends = (part.cumsum(0) / part.sum() * T).round().to(torch.int32)
    if n >= 8:
        ends[2] = ends[1]
        ends[4] = ends[3] + 1
        ends = ends.cummax(0).values.clamp_(max=T)
    ends[-1] = T
    return torch.cat([torch.zeros(1, dtype=torch.int32), ends])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    kind = case["kind"]
    s = {"case": case}
    if kind in ("step", "scan", "adjoint"):
        D = case["D"]
        rows = case["B"] if kind == "step" else case["T"]
        seqs = case["B"] if kind == "step" else case["seqs"]
        s["u"] = normal(rows, 3, D, dtype=DTYPES[case["u"]])
        # decays between 0.9 and 0.999 where the gate is open
        s["rate"] = -torch.log(0.9 + 0.099 * torch.rand(D, generator=g, device=dev))
        s["h0"] = normal(seqs, D, std=0.5)
        if kind == "step":
            return s
        s["starts"] = None
        if case["packed"]:
            s["starts"] = starts_of(case, seed).to(dev)
        else:
            s["u"] = s["u"].view(seqs, rows // seqs, 3, D)
        if kind == "adjoint":
            shape = s["u"].shape[:-2] + (D,)
            # states of the size that the forward pass reaches
            s["h"] = normal(*shape)
            s["dh"] = normal(*shape)
            s["dh_last"] = normal(seqs, D)
    elif kind == "norm":
        T, D = case["T"], case["D"]
        s["x"] = normal(T, D, dtype=DTYPES[case["x"]])
        s["res"] = None if case["res"] == "none" else normal(T, D, std=2.0, dtype=DTYPES[case["res"]])
        s["w"] = 1.0 + normal(D, std=0.1)
    elif kind == "norm_adjoint":
        T, D = case["T"], case["D"]
        s["sum"] = normal(T, D, std=2.0, dtype=DTYPES[case["x"]])
        s["dsum"] = normal(T, D, dtype=DTYPES[case["x"]])
        s["dy"] = normal(T, D, dtype=DTYPES[case["y"]])
        s["w"] = 1.0 + normal(D, std=0.1)
        s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(1) + 1e-6)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        kept = DTYPES[case.get("x", "f32")]
        # activations with a few large columns, as norms leave them
        x = (normal(M, K) * (1.0 + 4.0 * (torch.rand(K, generator=g, device=dev) < 0.02))).to(kept)
        w = normal(N, K, std=K ** -0.5, dtype=kept)
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        if kind == "product":
            s["x"], s["x_scale"] = quantize(x, 1)
            s["w"], s["w_scale"] = quantize(w, BLOCK)
        else:
            s["x"], s["w"] = x, w
    return s


# -------------------------------------------------------------- plain forms

def row_sequences(u, starts, seqs):
    """(first, last, owner) of every row: whether it begins or ends a sequence, and which one's it is."""
    T = u.shape[0]
    if starts is None:
        starts = torch.arange(seqs + 1, device=u.device) * (T // seqs)
    t = torch.arange(T, device=u.device)
    owner = torch.searchsorted(starts.long(), t, right=True) - 1
    return t == starts[owner], t + 1 == starts[owner + 1], owner


def doubled(a, b):
    """y_t = a_t y_{t-1} + b_t along dimension 0, from y = 0, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def gates(u, rate):
    r, i, x = u.unbind(-2)
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    decay = rate * sr
    left = -torch.expm1(-decay)
    return sr, si, x, decay, torch.exp(-decay), torch.sqrt(left * (2 - left))


def scan(u, rate, h0, starts):
    flat = u.reshape(-1, 3, u.shape[-1])
    first, last, owner = row_sequences(flat, starts, h0.shape[0])
    _, si, x, _, a, m = gates(flat.float(), rate)
    b = m * si * x
    b = torch.where(first[:, None], b + a * h0[owner], b)
    h = doubled(torch.where(first[:, None], 0.0, a), b)
    h_last = h0.clone()
    h_last[owner[last]] = h[last]
    return h.view(u.shape[:-2] + (u.shape[-1],)), h_last


def adjoint(u, rate, h0, h, dh, dh_last, starts):
    shape, D = u.shape, u.shape[-1]
    flat, h, dh = u.reshape(-1, 3, D), h.reshape(-1, D), dh.reshape(-1, D)
    first, last, owner = row_sequences(flat, starts, h0.shape[0])
    # in 64 bits: the rates' gradients are long sums of terms of either sign
    h0, h, dh, dh_last = h0.double(), h.double(), dh.double(), dh_last.double()
    sr, si, x, decay, a, m = gates(flat.double(), rate.double())
    before = torch.where(first[:, None], h0[owner], torch.cat([h[:1], h[:-1]]))
    up = torch.where(last[:, None], dh + dh_last[owner], dh)
    back = doubled(torch.where(last[:, None], 0.0, a).flip(0), (a * up).flip(0)).flip(0)
    lam = up + torch.where(last[:, None], 0.0, torch.cat([back[1:], back[:1]]))
    dx = lam * m * si
    di = dx * x * (1 - si)
    dl = lam * (a * a / m * si * x - a * before)
    du = torch.stack([dl * decay * (1 - sr), di, dx], 1)
    drate = (dl * sr).sum(0)
    dh0 = dh_last.clone()
    dh0[owner[first]] = back[first]
    return du.view(shape).float(), drate.float(), dh0.float()


def step(u, rate, h):
    _, si, x, _, a, m = gates(u.float(), rate)
    return a * h + m * si * x


def blocks(v, rows):
    """v [M, K] filled up with noughts to whole blocks: [M/rows, rows, K/128, 128]."""
    M, K = v.shape
    v = torch.nn.functional.pad(v, (0, -K % BLOCK, 0, -M % rows))
    return v.view(v.shape[0] // rows, rows, v.shape[1] // BLOCK, BLOCK)


def quantize(v, rows):
    """(e4m3 values, scales) with a scale for each `rows` x 128 block."""
    M, K = v.shape
    v = blocks(v.float(), rows)
    # divided by a tensor: by a plain number the device would multiply by its rounded inverse
    scale = (v.abs().amax((1, 3)) / torch.full((), TOP, device=v.device)).clamp(min=LEAST)
    q = (v / scale[:, None, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return q.reshape(q.shape[0] * rows, -1)[:M, :K].contiguous(), scale


def norm(x, w, res, eps, y_dtype):
    v = x.float() if res is None else x.float() + res.float()
    rstd = torch.rsqrt(v.square().mean(1) + eps)
    y = v * rstd[:, None] * w
    y, scale = quantize(y, 1) if y_dtype == torch.float8_e4m3fn else (y.to(y_dtype), None)
    return y, scale, None if res is None else v.to(res.dtype), rstd


def norm_adjoint(dy, total, w, rstd, dsum):
    n = total.float() * rstd[:, None]
    gw = dy.float() * w
    dx = dsum.float() + rstd[:, None] * (gw - n * (gw * n).mean(1, keepdim=True))
    return dx.to(total.dtype), (dy.float() * n).sum(0, dtype=torch.float64).float()


def product(x, x_scale, w, w_scale, bias, dtype):
    wide = (blocks(x.float(), 1) * x_scale[:, None, :, None]).flatten(2).flatten(0, 1)[:, :x.shape[1]]
    deep = (blocks(w.float(), BLOCK) * w_scale[:, None, :, None]).flatten(2).flatten(0, 1)[:w.shape[0], :w.shape[1]]
    u = wide @ deep.T
    return (u if bias is None else u + bias).to(dtype)


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import nonlinear_rnn_newton_b200 as P
    if kind == "step":
        return P.pararnn_glr_step(s["u"], s["rate"], s["h0"]) if own else step(s["u"], s["rate"], s["h0"])
    if kind == "scan":
        if own:
            return P.pararnn_glr_scan(s["u"], s["rate"], s["h0"], seq_starts=s["starts"])
        return scan(s["u"], s["rate"], s["h0"], s["starts"])
    if kind == "adjoint":
        if own:
            return P.pararnn_glr_adjoint(s["u"], s["rate"], s["h0"], s["h"], s["dh"], dh_last=s["dh_last"],
                                         seq_starts=s["starts"])
        return adjoint(s["u"], s["rate"], s["h0"], s["h"], s["dh"], s["dh_last"], s["starts"])
    if kind == "norm":
        y = DTYPES[case["y"]]
        if own:
            out = P.pararnn_rms_norm(s["x"], s["w"], residual=s["res"], eps=1e-6, out_dtype=y)
        else:
            out = norm(s["x"], s["w"], s["res"], 1e-6, y)
        return [v for v in out if v is not None]
    if kind == "norm_adjoint":
        if own:
            return P.pararnn_rms_norm_adjoint(s["dy"], s["sum"], s["w"], s["rstd"], dsum=s["dsum"])
        return norm_adjoint(s["dy"], s["sum"], s["w"], s["rstd"], s["dsum"])
    u = DTYPES[case["u"]]
    if kind == "product":
        if own:
            return P.pararnn_fp8_project(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=u)
        return product(s["x"], s["x_scale"], s["w"], s["w_scale"], s["bias"], u)
    if own:
        x, x_scale = P.pararnn_fp8_quantize(s["x"], block_rows=1)
        w, w_scale = P.pararnn_fp8_quantize(s["w"], block_rows=BLOCK)
        out = P.pararnn_fp8_project(x, x_scale, w, w_scale, bias=s["bias"], out_dtype=u)
    else:
        x, x_scale = quantize(s["x"], 1)
        w, w_scale = quantize(s["w"], BLOCK)
        out = product(x, x_scale, w, w_scale, s["bias"], u)
    return x, x_scale, w, w_scale, out


# --------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    if kind in ("step", "scan", "adjoint"):
        D, es = case["D"], BYTES[case["u"]]
        if kind == "step":
            return {"bytes": case["B"] * D * (3 * es + 8) + 4 * D, "flops": 20 * case["B"] * D}
        ends = case["seqs"] * D * 4 + 4 * D
        if kind == "scan":
            return {"bytes": case["T"] * D * (3 * es + 4) + 2 * ends, "flops": 20 * case["T"] * D}
        return {"bytes": case["T"] * D * (3 * es + 8 + 12) + 3 * ends, "flops": 40 * case["T"] * D}
    if kind == "norm":
        T, D = case["T"], case["D"]
        res = 0 if case["res"] == "none" else 2 * BYTES[case["res"]]
        scales = 4 * T * -(-D // BLOCK) if case["y"] == "e4m3" else 0
        return {"bytes": T * D * (BYTES[case["x"]] + res + BYTES[case["y"]]) + scales + 4 * T + 4 * D, "flops": 6 * T * D}
    if kind == "norm_adjoint":
        T, D = case["T"], case["D"]
        return {"bytes": T * D * (3 * BYTES[case["x"]] + BYTES[case["y"]]) + 4 * T + 8 * D, "flops": 10 * T * D}
    M, N, K = case["M"], case["N"], case["K"]
    scales = 4 * -(-K // BLOCK) * (M + -(-N // BLOCK))
    total = (M + N) * K + scales + M * N * BYTES[case["u"]] + (4 * N if case["bias"] else 0)
    if kind == "quantized_product":
        total += (M + N) * K * BYTES[case["x"]]
    return {"bytes": total, "flops": 2 * M * N * K}


# -------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() and v.dtype != torch.float8_e4m3fn else v
         for k, v in s.items()}
    if kind in ("step", "scan", "adjoint"):
        return exact_recurrence(case, d)
    if kind == "norm":
        v = d["x"] if d["res"] is None else d["x"] + d["res"]
        mean = (v * v).sum(1) / case["D"] + 1e-6
        y = v / mean.sqrt()[:, None] * d["w"]
        out = [y]
        if case["y"] == "e4m3":
            out = list(exact_quantized(y, 1))
        return out + ([] if d["res"] is None else [v]) + [mean ** -0.5]
    if kind == "norm_adjoint":
        v = d["sum"].requires_grad_(True)
        w = d["w"].requires_grad_(True)
        # the norm with rstd as given: its own derivative joins through the row's mean
        n = v.detach() * d["rstd"][:, None]
        inner = (d["dy"] * d["w"].detach() * n).sum(1, keepdim=True) / case["D"]
        value = (d["dy"] * w * v * d["rstd"][:, None]).sum() - (v * (n * inner * d["rstd"][:, None])).sum()
        dv, dw = torch.autograd.grad(value, (v, w))
        return dv + d["dsum"], dw
    lead = ()
    if kind == "quantized_product":
        lead = exact_quantized(d["x"], 1) + exact_quantized(d["w"], BLOCK)
        x, x_scale, w, w_scale = lead
    else:
        x, x_scale, w, w_scale = s["x"].double(), d["x_scale"], s["w"].double(), d["w_scale"]
    K = case["K"]
    u = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=x.device)
    for k in range(0, K, BLOCK):
        rows = w_scale[:, k // BLOCK].repeat_interleave(BLOCK)[:case["N"]]
        u += (x[:, k:k + BLOCK] @ w[:, k:k + BLOCK].T) * x_scale[:, k // BLOCK, None] * rows
    if d["bias"] is not None:
        u += d["bias"]
    return u if kind == "product" else lead + (u,)


def exact_quantized(v, rows):
    """e4m3 values (8 steps to an octave, 2^-9 below 2^-6) and scales, block by block. The scale that is kept has
    32 bits, and the value that is rounded to e4m3 is the 32-bit quotient by it: bf16 inputs often lie halfway
    between two e4m3 values, and which one is theirs goes by that."""
    M, K = v.shape
    q = torch.empty_like(v)
    scale = torch.empty(-(-M // rows), -(-K // BLOCK), dtype=torch.float64, device=v.device)
    for j in range(scale.shape[1]):
        part = v[:, j * BLOCK:(j + 1) * BLOCK]
        most = part.abs().amax(1)
        if rows > 1:
            most = torch.nn.functional.pad(most, (0, -M % rows)).view(-1, rows).amax(1)
        scale[:, j] = torch.clamp(most / TOP, min=LEAST).float()
        z = (part.float() / scale[:, j].float().repeat_interleave(rows)[:M, None]).double()
        grid = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, j * BLOCK:(j + 1) * BLOCK] = (torch.round(z / grid) * grid).clamp(-TOP, TOP)
    return q, scale


def exact_recurrence(case, d):
    """One row after another, every sequence by itself; gradients of the gates from autograd of one row's formula."""
    u, rate, D = d["u"].reshape(-1, 3, case["D"]), d["rate"], case["D"]

    def formula(u, rate, before):
        open_ = 1 / (1 + torch.exp(-u[..., 0, :]))
        a = torch.exp(-rate * open_)
        fresh = torch.sqrt(-torch.expm1(-2 * rate * open_))
        return a * before + fresh * u[..., 2, :] / (1 + torch.exp(-u[..., 1, :]))

    if case["kind"] == "step":
        return formula(u, rate, d["h0"])
    T, n = case["T"], case["seqs"]
    ends = d["starts"].tolist() if case["packed"] else [T // n * k for k in range(n + 1)]
    a = torch.exp(-rate / (1 + torch.exp(-u[:, 0])))
    if case["kind"] == "scan":
        b = formula(u, rate, torch.zeros(D, dtype=torch.float64, device=u.device))
        h = torch.empty_like(b)
        h_last = d["h0"].clone()
        for k in range(n):
            y = d["h0"][k]
            for t in range(ends[k], ends[k + 1]):
                y = torch.addcmul(b[t], a[t], y, out=h[t])
            h_last[k] = y
        return h.view(d["u"].shape[:-2] + (D,)), h_last
    h, dh = d["h"].reshape(-1, D), d["dh"].reshape(-1, D)
    before, lam, dh0 = torch.empty_like(h), torch.empty_like(h), d["dh_last"].clone()
    for k in range(n):
        lo, hi = ends[k], ends[k + 1]
        if lo == hi:
            continue
        before[lo] = d["h0"][k]
        before[lo + 1:hi] = h[lo:hi - 1]
        y = torch.add(dh[hi - 1], d["dh_last"][k], out=lam[hi - 1])
        for t in range(hi - 2, lo - 1, -1):
            y = torch.addcmul(dh[t], a[t + 1], y, out=lam[t])
        dh0[k] = a[lo] * y
    du, drate = torch.empty_like(u), torch.empty_like(rate)
    for c in range(0, D, 256):
        part = u[..., c:c + 256].clone().requires_grad_(True)
        speed = rate[c:c + 256].clone().requires_grad_(True)
        value = (formula(part, speed, before[:, c:c + 256]) * lam[:, c:c + 256]).sum()
        du[..., c:c + 256], drate[c:c + 256] = torch.autograd.grad(value, (part, speed))
    return du.view(d["u"].shape), drate, dh0
