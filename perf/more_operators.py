"""The selective scan with its causal convolution, RMS norm with the residual's addition, and the matrix
product of 8-bit numbers with a scale for each block of 128, as cases to measure.

The selective scan keeps a state h [dstate] for every channel d, with keys B_t and C_t [dstate] shared by
the channels of a group:

    Delta_t = softplus(dt_t + dt_bias)          (or dt_t + dt_bias)
    h_t = exp(Delta_t A) h_{t-1} + Delta_t x_t B_t
    y_t = (C_t . h_t + D x_t) SiLU(z_t)

The convolution in front of it is v_t = SiLU(bias + sum_k weight_k x_{t-width+1+k}) for every channel.
RMS norm: r = x + residual rounded to the residual's type, y = r weight / sqrt(mean(r^2) + eps), or y in e4m3
with the scale max|y| / 448 for each 128 values of a row.  The product: out[m][n] = sum over blocks kb of
a_scale[m][kb] w_scale[n/128][kb] sum over k in kb of a[m][k] w[n][k].

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits; where it is
true it calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-5
BLOCK = 128       # values that share a scale
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
LEAST = 2.0 ** -126   # the least scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _scan(op, batch, seqlen, dim, dstate=16, ngroups=1, dtype="bf16", init=False, gate=True, softplus=True, nseq=0, lo=0, hi=0):
    return {"op": op, "batch": batch, "seqlen": seqlen, "dim": dim, "dstate": dstate, "ngroups": ngroups, "dtype": dtype,
            "init": init, "gate": gate, "softplus": softplus, "nseq": nseq, "lo": lo, "hi": hi}


def _conv(op, batch, seqlen, dim, width=4, dtype="bf16", init=False, silu=True, nseq=0, lo=0, hi=0):
    return {"op": op, "batch": batch, "seqlen": seqlen, "dim": dim, "width": width, "dtype": dtype, "init": init, "silu": silu,
            "nseq": nseq, "lo": lo, "hi": hi}


def _norm(op, rows, dim, dtype="bf16", residual="fp32"):
    return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": residual}


def _product(rows, cols, inner, dtype="bf16", bias=False):
    return {"op": "product", "rows": rows, "cols": cols, "inner": inner, "dtype": dtype, "bias": bias}


def listed():
    cases = {
        # a short prompt that continues a carried state, at the inner width of the small workload; latency counts
        "scan_fwd short_turn": _scan("scan_fwd", 1, 77, 1536, init=True),
        # a serving batch of prompts of different lengths packed into one stream, each with its carried state
        "scan_fwd packed_prompts": _scan("scan_fwd", 1, 0, 5120, init=True, nseq=16, lo=128, hi=2048),
        # gradients in 32 bits at odd sizes: packed sequences down to one token, carried states, their gradients
        "scan_bwd odd_fp32": _scan("scan_bwd", 1, 0, 291, dstate=13, ngroups=3, dtype="fp32", init=True, nseq=9, lo=1, hi=301),
        # gradients of one training step at the 2.7B-scale inner width
        "scan_bwd train_2.7B": _scan("scan_bwd", 8, 2048, 5120),
        # one token of each of 64 sequences (the decode workload's batch)
        "scan_step decode_b64": _scan("scan_step", 64, 1, 5120, init=True),
        # the convolution of the packed prompts, each with its carried window
        "conv_fwd packed_prompts": _conv("conv_fwd", 1, 0, 5120, init=True, nseq=16, lo=128, hi=2048),
        # the convolution's gradients in the training step
        "conv_bwd train_2.7B": _conv("conv_bwd", 8, 2048, 5120),
        # the norm before a decode step's projection: one token of each of 64 sequences, to 8 bits
        "norm_quant decode_rows": _norm("norm_quant", 64, 2560),
        # the norm before a prompt batch's projection, to 8 bits, the residual stream in 32 bits
        "norm_quant prompt_rows": _norm("norm_quant", 16384, 2560),
        # gradients of a training step's norm, the residual stream in 32 bits
        "norm_bwd train_rows": _norm("norm_bwd", 16384, 2560),
        # the projection of a decode step: 64 rows against the 2.7B-scale weights (2560 to 2 x 5120)
        "product decode_rows": _product(64, 10240, 2560),
        # the same of a prompt batch of 16K tokens
        "product prompt_rows": _product(16384, 10240, 2560),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd", "conv_step", "norm_fwd",
                     "norm_quant", "norm_bwd", "product", "product"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "product":
        rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 16, 10240)
        return _product(rows, cols, 16 * _log_int(rng, 1, 640), dtype, rng.random() < 0.3)
    if op.startswith("norm"):
        dim = _log_int(rng, 16, 8192)
        return _norm(op, _log_int(rng, 1, min(16384, (32 << 20) // dim)), dim, dtype, rng.choice(["none", dtype, "fp32"]))
    packed = rng.random() < 0.5 and not op.endswith("step")
    nseq = _log_int(rng, 2, 40) if packed else 0
    most = 2048 if op == "scan_bwd" else 4096
    seqlen = 1 if op.endswith("step") else _log_int(rng, 1, most)
    lo = hi = 0
    if packed:
        hi = max(2, seqlen // 2)
        lo, seqlen = rng.randint(1, hi), 0
    batch = _log_int(rng, 1, 128) if op.endswith("step") else 1 if packed else rng.randint(1, max(1, min(4, most // seqlen)))
    if op.startswith("conv"):
        return _conv(op, batch, seqlen, _log_int(rng, 16, 5120), rng.randint(2, 4), dtype, rng.random() < 0.5 or op == "conv_step",
                     rng.random() < 0.8, nseq, lo, hi)
    ngroups = rng.choice([1, 1, 2, 3, 4])
    dim = ngroups * _log_int(rng, 16, 4096 // ngroups)
    dstate = rng.choice([16, 16, rng.randint(1, 64)])
    if dim * dstate > 1 << 16:
        dstate = 16
    return _scan(op, batch, seqlen, dim, dstate, ngroups, dtype, rng.random() < 0.5 or op == "scan_step", rng.random() < 0.7,
                 rng.random() < 0.8, nseq, lo, hi)


def _lengths(case):
    """The lengths of a packed case's sequences: spread over its range, the shortest and the longest among them."""
    n, lo, hi = case["nseq"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((7 * i) % n) // max(1, n - 1) for i in range(n)]


def _tokens(case):
    return sum(_lengths(case)) if case["nseq"] else case["batch"] * case["seqlen"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    el, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    if op == "product":
        m, n, k = case["rows"], case["cols"], case["inner"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        # activations of rows and columns of different size, weights of a linear layer; both as their
        # quantisation leaves them: the largest of a block at 448
        a, a_scale = _to_8bit(normal(m, k) * (0.3 + normal(1, k).abs()))
        w = normal(n, k) / math.sqrt(k)
        wide = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(nb, BLOCK, kb, BLOCK)
        w_scale = (wide.abs().amax((1, 3)) / F8_MAX).clamp(min=LEAST)
        w = (wide / w_scale[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous().to(F8)
        return {"op": op, "a": a, "a_scale": a_scale, "w": w, "w_scale": w_scale, "el": el,
                "bias": 0.1 * normal(n) if case["bias"] else None}

    if op.startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        s = {"op": op, "x": normal(rows, dim).to(el), "weight": 1 + 0.1 * normal(dim), "residual": None}
        if case["residual"] != "none":
            # a residual stream: rows of different size, a few large channels
            s["residual"] = (normal(rows, dim) * (0.5 + 2 * normal(rows, 1).abs()) * (1 + 9 * (uniform(1, dim) < 0.01))).to(TYPES[case["residual"]])
        if op == "norm_bwd":
            s["dy"] = normal(rows, dim).to(el)
            # what the forward pass of the same step left, and the gradient of the residual stream
            s["stream"] = s["x"] if s["residual"] is None else s["residual"]
            s["rstd"] = (s["stream"].double().square().mean(1) + EPS).rsqrt().float()
            s["dres"] = None if s["residual"] is None else normal(rows, dim).to(s["stream"].dtype)
        return s

    packed = case["nseq"] > 0
    B, T, D = (1, _tokens(case), case["dim"]) if packed else (case["batch"], case["seqlen"], case["dim"])
    step = op.endswith("step")
    lead = (B,) if step else (B, T)
    rows = case["nseq"] if packed else B
    s = {"op": op, "seq_idx": None, "nseq": None, "lengths": None, "init": None}
    if packed:
        s["lengths"], s["nseq"] = _lengths(case), case["nseq"]
        s["seq_idx"] = torch.repeat_interleave(torch.arange(s["nseq"], device="cuda", dtype=torch.int32),
                                               torch.tensor(s["lengths"], device="cuda"), output_size=T)
    # the projection into the block gives x and z side by side
    xz = normal(*lead, 2 * D).to(el)
    if op.startswith("conv"):
        K = case["width"]
        s["x"], s["silu"] = xz[..., :D], case["silu"]
        s["weight"], s["bias"] = normal(D, K) / math.sqrt(K), 0.1 * normal(D)
        if case["init"]:
            s["init"] = normal(rows, K - 1, D).to(el)
        if op == "conv_bwd":
            s["dy"] = normal(*lead, D).to(el)
            s["dfinal"] = normal(rows, K - 1, D).to(el) if case["init"] else None
        if step:
            s["window"] = s["init"].clone()
        return s

    N, G = case["dstate"], case["ngroups"]
    s["softplus"] = case["softplus"]
    s["x"] = normal(*lead, D).to(el)
    s["z"] = xz[..., D:] if case["gate"] else None
    # B and C stand behind the low-rank part of dt in one projection's output
    low = -(-D // 32)
    bc = normal(*lead, low + 2 * G * N).to(el)
    s["B"] = bc[..., low:low + G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., low + G * N:].unflatten(-1, (G, N))
    # step sizes from 0.001 to 0.1 around which the tokens vary, rates 1 to N, as these layers start from
    step0 = torch.exp(uniform(D) * math.log(100.0)) * 1e-3
    raw = step0 + torch.log(-torch.expm1(-step0))
    if case["softplus"]:
        s["dt"], s["dt_bias"] = (0.5 * normal(*lead, D)).to(el), raw
    else:
        s["dt"], s["dt_bias"] = torch.nn.functional.softplus(0.5 * normal(*lead, D) + raw).to(el), None
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * normal(D, N))
    s["D"] = 1 + 0.1 * normal(D)
    if case["init"]:
        s["init"] = 0.3 * normal(rows, D, N)
    if op == "scan_bwd":
        s["dy"] = normal(*lead, D).to(el)
        s["dfinal"] = 0.3 * normal(rows, D, N) if case["init"] else None
    if step:
        s["state"] = s["init"].clone()
    return s


def _to_8bit(y):
    """[rows, dim] in 32 bits as e4m3 with a scale for each 128 values of a row."""
    rows, dim = y.shape
    nb = -(-dim // BLOCK)
    b = torch.nn.functional.pad(y, (0, nb * BLOCK - dim)).view(rows, nb, BLOCK)
    scale = (b.abs().amax(2) / F8_MAX).clamp(min=LEAST)
    q = (b / scale[..., None]).clamp(-F8_MAX, F8_MAX).to(F8)
    return q.view(rows, nb * BLOCK)[:, :dim].contiguous(), scale


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rows_of(s):
    """Packed streams as a batch: the index [nseq, longest] of every sequence's tokens, and which of them are real."""
    if s["nseq"] is None:
        return None
    dev = s["x"].device
    n = torch.tensor(s["lengths"], device=dev)
    at = torch.arange(max(s["lengths"]), device=dev)
    real = at < n[:, None]
    return torch.where(real, (n.cumsum(0) - n)[:, None] + at, 0), real


def _batched(x, rows):
    """[batch, tokens, ...] -> [sequences, longest, ...] in 32 bits, zero behind the last token."""
    x = x.float()
    if rows is None:
        return x
    return x[0][rows[0]] * rows[1].view(rows[1].shape + (1,) * (x.dim() - 2))


def _flat(x, like, rows):
    return (x if rows is None else x[rows[1]][None]).to(like.dtype)


def _plain_steps(s, dt):
    dt = dt if s["dt_bias"] is None else dt + s["dt_bias"]
    return torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs())) if s["softplus"] else dt


def _plain_scan(s):
    """What both directions need: everything in 32 bits, and the state before every token."""
    rows = _rows_of(s)
    c = {n: _batched(s[n], rows) for n in ("x", "dt", "B", "C")}
    if rows is not None:
        c["keep"] = rows[1][:, :, None]
    c["delta"] = _plain_steps(s, c["dt"])
    if rows is not None:
        c["delta"] = c["delta"] * c["keep"]
    b, T, D = c["x"].shape
    G, N = s["B"].shape[2:]
    c["grouped"] = (b, G, D // G, N)
    h = torch.zeros(b, D, N, device=s["x"].device) if s["init"] is None else s["init"]
    c["dx"] = c["delta"] * c["x"]
    before = []
    for t in range(T):
        before.append(h)
        add = c["dx"][:, t].view(b, G, D // G, 1) * c["B"][:, t, :, None]
        h = torch.exp(c["delta"][:, t, :, None] * s["A"]) * h + add.view(b, D, N)
    return rows, c, before, h


def _gated(s, c, y, rows):
    if s["z"] is None:
        return y
    z = _batched(s["z"], rows)
    return y * (z / (1 + torch.exp(-z)))


def _plain_y(s, c, before, last):
    b, G, per, N = c["grouped"]
    hs = before[1:] + [last]
    y = torch.stack([(hs[t].view(b, G, per, N) * c["C"][:, t, :, None]).sum(-1).view(b, G * per) for t in range(len(hs))], 1)
    return y + s["D"] * c["x"]


def _plain_scan_fwd(s):
    rows, c, before, last = _plain_scan(s)
    return _flat(_gated(s, c, _plain_y(s, c, before, last), rows), s["x"], rows), last


def _plain_scan_bwd(s):
    rows, c, before, last = _plain_scan(s)
    b, G, per, N = c["grouped"]
    D = G * per
    dy = _batched(s["dy"], rows)
    out = {}
    if s["z"] is not None:
        y = _plain_y(s, c, before, last)
        z = _batched(s["z"], rows)
        sig = 1 / (1 + torch.exp(-z))
        out["dz"] = _flat(dy * y * sig * (1 + z * (1 - sig)), s["x"], rows)
        dy = dy * z * sig
    else:
        out["dz"] = None
    g = torch.zeros_like(last) if s["dfinal"] is None else s["dfinal"].clone()
    dA = torch.zeros_like(s["A"])
    ddelta, ddx, dB, dC = [], [], [], []
    h = last
    for t in range(len(before) - 1, -1, -1):
        yt = dy[:, t].view(b, G, per, 1)
        dC.append((h.view(b, G, per, N) * yt).sum(2))
        g = g + (yt * c["C"][:, t, :, None]).view(b, D, N)
        g4 = g.view(b, G, per, N)
        dB.append((g4 * c["dx"][:, t].view(b, G, per, 1)).sum(2))
        ddx.append((g4 * c["B"][:, t, :, None]).sum(-1).view(b, D))
        step = c["delta"][:, t, :, None]
        g = g * torch.exp(step * s["A"])
        gh = g * before[t]
        ddelta.append((gh * s["A"]).sum(-1))
        dA = dA + (gh * step).sum(0)
        h = before[t]
    ddelta, ddx, dB, dC = (torch.stack(v[::-1], 1) for v in (ddelta, ddx, dB, dC))
    ddelta = ddelta + ddx * c["x"]
    out["dx"] = _flat(ddx * c["delta"] + dy * s["D"], s["x"], rows)
    out["dD"] = (dy * c["x"]).sum((0, 1))
    if s["softplus"]:
        raw = c["dt"] if s["dt_bias"] is None else c["dt"] + s["dt_bias"]
        ddelta = ddelta / (1 + torch.exp(-raw))
    if rows is not None:
        ddelta = ddelta * c["keep"]
    out["ddt"] = _flat(ddelta, s["x"], rows)
    out["ddt_bias"] = ddelta.sum((0, 1)) if s["dt_bias"] is not None else None
    out["dA"] = dA
    out["dB"], out["dC"] = _flat(dB, s["x"], rows), _flat(dC, s["x"], rows)
    out["dinitial_states"] = g if s["init"] is not None else None
    return out


def _plain_scan_step(s):
    delta = _plain_steps(s, s["dt"].float())
    x = s["x"].float()
    b, D = x.shape
    B, C = (s[n].float().repeat_interleave(D // s[n].shape[1], dim=1) for n in ("B", "C"))
    h = torch.exp(delta[..., None] * s["A"]) * s["state"] + (delta * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1 + torch.exp(-z)))
    # the state moves on in place: the next pass is the next token
    return y.to(s["x"].dtype), s["state"].copy_(h)


def _windowed(s, rows):
    """The inputs with width - 1 of their past in front."""
    x = _batched(s["x"], rows)
    past = s["weight"].shape[1] - 1
    front = x.new_zeros(x.shape[0], past, x.shape[2]) if s["init"] is None else s["init"].float()
    return torch.cat([front, x], 1)


def _plain_conv(s, xs, T):
    v = s["bias"].expand(xs.shape[0], T, -1)
    for k in range(s["weight"].shape[1]):
        v = v + xs[:, k:k + T] * s["weight"][:, k]
    return v


def _last_window(s, xs, rows, past):
    if rows is None:
        return xs[:, xs.shape[1] - past:]
    at = torch.tensor(s["lengths"], device=xs.device)[:, None] + torch.arange(past, device=xs.device)
    return xs.gather(1, at[:, :, None].expand(-1, -1, xs.shape[2]))


def _plain_conv_fwd(s):
    rows = _rows_of(s)
    xs, past = _windowed(s, rows), s["weight"].shape[1] - 1
    v = _plain_conv(s, xs, xs.shape[1] - past)
    y = v / (1 + torch.exp(-v)) if s["silu"] else v
    return _flat(y, s["x"], rows), _last_window(s, xs, rows, past).to(s["x"].dtype)


def _plain_conv_bwd(s):
    rows = _rows_of(s)
    xs, past = _windowed(s, rows), s["weight"].shape[1] - 1
    T = xs.shape[1] - past
    dv = _batched(s["dy"], rows)
    if s["silu"]:
        v = _plain_conv(s, xs, T)
        sig = 1 / (1 + torch.exp(-v))
        dv = dv * sig * (1 + v * (1 - sig))
    dxs, dw = torch.zeros_like(xs), []
    for k in range(past + 1):
        dxs[:, k:k + T] += dv * s["weight"][:, k]
        dw.append((dv * xs[:, k:k + T]).sum((0, 1)))
    if s["dfinal"] is not None:
        n = torch.tensor(s["lengths"] if rows is not None else [T] * xs.shape[0], device=xs.device)
        at = n[:, None] + torch.arange(past, device=xs.device)
        dxs.scatter_add_(1, at[:, :, None].expand(-1, -1, xs.shape[2]), s["dfinal"].float())
    return {"dx": _flat(dxs[:, past:], s["x"], rows), "dweight": torch.stack(dw, 1), "dbias": dv.sum((0, 1)),
            "dinitial_window": dxs[:, :past].to(s["x"].dtype) if s["init"] is not None else None}


def _plain_conv_step(s):
    xs = torch.cat([s["window"], s["x"][:, None]], 1)
    v = s["bias"] + (xs.float() * s["weight"].t()).sum(1)
    y = v / (1 + torch.exp(-v)) if s["silu"] else v
    return y.to(s["x"].dtype), s["window"].copy_(xs[:, 1:])


def _plain_stream(s):
    if s["residual"] is None:
        return s["x"]
    return (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)


def _plain_norm(s):
    stream = _plain_stream(s)
    r = stream.float()
    rstd = 1 / torch.sqrt((r * r).mean(1) + EPS)
    return r * rstd[:, None] * s["weight"], stream, rstd


def _plain_norm_bwd(s):
    r, dy = s["stream"].float(), s["dy"].float()
    hat = r * s["rstd"][:, None]
    w = dy * s["weight"]
    dr = (w - hat * (w * hat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dr = dr + s["dres"].float()
    return {"dx": dr.to(s["dy"].dtype), "dresidual": None if s["dres"] is None else dr.to(s["dres"].dtype), "dweight": (dy * hat).sum(0)}


def _plain_product(s):
    m, k = s["a"].shape
    n = s["w"].shape[0]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, dim=1)[:, :k]
    w = s["w"].float() * s["w_scale"].repeat_interleave(BLOCK, dim=0)[:n].repeat_interleave(BLOCK, dim=1)[:, :k]
    out = a @ w.t()
    return (out if s["bias"] is None else out + s["bias"]).to(s["el"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own_scan(s, op):
    from ssd_chunked_scan_amd import ssd
    kw = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "dt_softplus": s["softplus"]}
    if op == "scan_step":
        return ssd.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], **kw), s["state"]
    kw.update(initial_states=s["init"], seq_idx=s["seq_idx"], nseq=s["nseq"])
    if op == "scan_fwd":
        return ssd.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], **kw)
    return ssd.selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], dfinal_states=s["dfinal"],
                                  want_dinit=s["init"] is not None, **kw)


def _own_conv(s, op):
    from ssd_chunked_scan_amd import ssd
    if op == "conv_step":
        return ssd.causal_conv_step(s["x"], s["window"], s["weight"], bias=s["bias"], silu=s["silu"]), s["window"]
    kw = {"bias": s["bias"], "silu": s["silu"], "initial_window": s["init"], "seq_idx": s["seq_idx"], "nseq": s["nseq"]}
    if op == "conv_fwd":
        return ssd.causal_conv_fwd(s["x"], s["weight"], **kw)
    return ssd.causal_conv_bwd(s["x"], s["weight"], s["dy"], dfinal_window=s["dfinal"], want_dinit=s["init"] is not None, **kw)


def _own_norm(s, op):
    from ssd_chunked_scan_amd import ssd
    if op == "norm_fwd":
        return ssd.rms_norm_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    if op == "norm_quant":
        return ssd.rms_norm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    return ssd.rms_norm_bwd(s["stream"], s["dy"], s["rstd"], s["weight"], dresidual=s["dres"])


def _own_product(s):
    from ssd_chunked_scan_amd import ssd
    return ssd.matmul_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=s["el"])


def run(state):
    s, op = state, state["op"]
    if own:
        if op.startswith("scan"):
            return _own_scan(s, op)
        if op.startswith("conv"):
            return _own_conv(s, op)
        return _own_product(s) if op == "product" else _own_norm(s, op)
    if op == "scan_fwd":
        return _plain_scan_fwd(s)
    if op == "scan_bwd":
        return _plain_scan_bwd(s)
    if op == "scan_step":
        return _plain_scan_step(s)
    if op == "conv_fwd":
        return _plain_conv_fwd(s)
    if op == "conv_bwd":
        return _plain_conv_bwd(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "product":
        return _plain_product(s)
    y, stream, rstd = _plain_norm(s)
    if op == "norm_quant":
        return (*_to_8bit(y), None if s["residual"] is None else stream)
    return y.to(s["x"].dtype), None if s["residual"] is None else stream, rstd


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op == "product":
        m, n, k = case["rows"], case["cols"], case["inner"]
        kb = -(-k // BLOCK)
        return {"bytes": (m + n) * k + 4 * kb * (m + -(-n // BLOCK)) + m * n * e + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op.startswith("norm"):
        n, d = case["rows"] * case["dim"], case["dim"]
        r = 0 if case["residual"] == "none" else SIZE[case["residual"]]
        if op == "norm_fwd":
            return {"bytes": n * (2 * e + 2 * r) + 4 * case["rows"] + 4 * d, "flops": 5 * n}
        if op == "norm_quant":
            return {"bytes": n * (e + 1 + 2 * r) + 4 * case["rows"] * -(-d // BLOCK) + 4 * d, "flops": 7 * n}
        # the stream, dy and the stream's gradient in, dx and (of another type) the stream's gradient out
        other = r if r and case["residual"] != case["dtype"] else 0
        return {"bytes": n * ((r or e) + e + r + e + other) + 4 * case["rows"] + 8 * d, "flops": 9 * n}
    T, D = _tokens(case), case["dim"]
    ids = 4 * T if case["nseq"] else 0
    rows = case["nseq"] or case["batch"]
    if op.startswith("conv"):
        K = case["width"]
        window = rows * (K - 1) * D * e
        par = 4 * D * (K + 1)
        if op == "conv_step":
            return {"bytes": 2 * T * D * e + 2 * window + par, "flops": 2 * K * T * D}
        if op == "conv_fwd":
            return {"bytes": 2 * T * D * e + window * (2 if case["init"] else 1) + par + ids, "flops": 2 * K * T * D}
        return {"bytes": 3 * T * D * e + window * (3 if case["init"] else 0) + 2 * par + ids, "flops": 6 * K * T * D}
    N, G = case["dstate"], case["ngroups"]
    states = 4 * rows * D * N
    par = 4 * D * (N + 1 + (1 if case["softplus"] else 0))
    token = (2 * D + 2 * G * N + (D if case["gate"] else 0)) * e   # x, dt, B, C, z
    if op == "scan_step":
        return {"bytes": T * (token + D * e) + 2 * states + par, "flops": 7 * T * D * N}
    # the recurrence itself: the decay's exponent, the update and the sum of every token, channel and state
    if op == "scan_fwd":
        return {"bytes": T * (token + D * e) + states * (2 if case["init"] else 1) + par + ids, "flops": 7 * T * D * N}
    return {"bytes": T * (2 * token + D * e) + states * (3 if case["init"] else 0) + 2 * par + ids, "flops": 20 * T * D * N}


# ---------------------------------------------------------------------------
# the definition, token by token in 64 bits
# ---------------------------------------------------------------------------

class _Sequences:
    """The sequences of a state, packed or not, token by token: those that have a t-th token, and its row."""

    def __init__(self, s):
        B, T = s["x"].shape[:2]
        self.n = s["lengths"] if s["nseq"] is not None else [T] * B
        self.length = torch.tensor(self.n, device=s["x"].device)
        self.first = self.length.cumsum(0) - self.length
        self.steps, self.count = max(self.n), len(self.n)

    def at(self, t):
        live = torch.nonzero(self.length > t)[:, 0]
        return self.first[live] + t, live


def _exact_inputs(s):
    """x, dt, z [tokens, D] and B, C [tokens, D, N] a token at a time, the step sizes and their slope."""
    D = s["x"].shape[-1]
    flat = {n: None if s[n] is None else s[n].reshape(-1, D).double() for n in ("x", "dt", "z")}
    for n in ("B", "C"):
        flat[n] = s[n].reshape(-1, *s[n].shape[-2:]).double()
    raw = flat["dt"] if s["dt_bias"] is None else flat["dt"] + s["dt_bias"].double()
    flat["delta"] = torch.logaddexp(raw, torch.zeros_like(raw)) if s["softplus"] else raw
    flat["slope"] = torch.sigmoid(raw) if s["softplus"] else torch.ones_like(raw)
    return flat


def _spread(k, D):
    return k.repeat_interleave(D // k.shape[1], dim=1)


def _exact_scan_fwd(s):
    f, seqs, A = _exact_inputs(s), _Sequences(s), s["A"].double()
    D, N = A.shape
    h = torch.zeros(seqs.count, D, N, device=A.device, dtype=torch.float64) if s["init"] is None else s["init"].double()
    y = torch.zeros_like(f["x"])
    for t in range(seqs.steps):
        rows, live = seqs.at(t)
        step = f["delta"][rows]
        new = torch.exp(step[..., None] * A) * h[live] + (step * f["x"][rows])[..., None] * _spread(f["B"][rows], D)
        h = h.index_copy(0, live, new)
        y[rows] = torch.matmul(new[:, :, None], _spread(f["C"][rows], D)[..., None])[..., 0, 0]
    y = y + s["D"].double() * f["x"]
    if f["z"] is not None:
        y = y * torch.nn.functional.silu(f["z"])
    return y.view(s["x"].shape), h


def _exact_scan_bwd(s):
    f, seqs, A = _exact_inputs(s), _Sequences(s), s["A"].double()
    D, N = A.shape
    G = s["B"].shape[-2]
    skip = s["D"].double()
    h = torch.zeros(seqs.count, D, N, device=A.device, dtype=torch.float64) if s["init"] is None else s["init"].double()
    gate = torch.ones_like(f["x"]) if f["z"] is None else torch.nn.functional.silu(f["z"])
    dout = s["dy"].reshape(-1, D).double()
    dy = dout * gate

    def token(rows, h0):
        step = f["delta"][rows]
        decay = torch.exp(step[..., None] * A)
        B, C = _spread(f["B"][rows], D), _spread(f["C"][rows], D)
        return step, decay, B, C, decay * h0 + (step * f["x"][rows])[..., None] * B

    kept, every = [], 64
    for t in range(seqs.steps):
        if t % every == 0:
            kept.append(h)
        rows, live = seqs.at(t)
        h = h.index_copy(0, live, token(rows, h[live])[-1])
    g = torch.zeros_like(h) if s["dfinal"] is None else s["dfinal"].double()
    like = {"dx": f["x"], "ddt": f["x"], "dB": f["B"], "dC": f["C"], "dz": f["x"]}
    out = {n: torch.zeros_like(v) for n, v in like.items()}
    dA = torch.zeros_like(A)
    for c in range(len(kept) - 1, -1, -1):
        last = min(seqs.steps, (c + 1) * every)
        hs = [kept[c]]
        for t in range(c * every, last):
            rows, live = seqs.at(t)
            hs.append(hs[-1].index_copy(0, live, token(rows, hs[-1][live])[-1]))
        for t in range(last - 1, c * every - 1, -1):
            rows, live = seqs.at(t)
            h0 = hs[t - c * every][live]
            step, decay, B, C, h1 = token(rows, h0)
            x, e = f["x"][rows], dy[rows]
            adj = g[live] + e[..., None] * C
            out["dz"][rows] = dout[rows] * ((h1 * C).sum(-1) + skip * x)
            out["dC"][rows] = (e[..., None] * h1).unflatten(1, (G, -1)).sum(2)
            out["dB"][rows] = ((step * x)[..., None] * adj).unflatten(1, (G, -1)).sum(2)
            along = (adj * B).sum(-1)
            out["dx"][rows] = step * along + skip * e
            back = decay * adj
            out["ddt"][rows] = (x * along + (back * h0 * A).sum(-1)) * f["slope"][rows]
            dA += (back * h0 * step[..., None]).sum(0)
            g = g.index_copy(0, live, back)
    res = {n: v.view(s[n[1:]].shape) for n, v in out.items() if n != "dz"}
    if f["z"] is None:
        res["dz"] = None
    else:
        sig = torch.sigmoid(f["z"])
        res["dz"] = (out["dz"] * (sig + f["z"] * sig * (1 - sig))).view(s["x"].shape)
    res["dA"], res["dD"] = dA, (dy * f["x"]).sum(0)
    res["ddt_bias"] = None if s["dt_bias"] is None else out["ddt"].sum(0)
    res["dinitial_states"] = None if s["init"] is None else g
    return res


def _exact_scan_step(s):
    A, x = s["A"].double(), s["x"].double()
    D = A.shape[0]
    raw = s["dt"].double() if s["dt_bias"] is None else s["dt"].double() + s["dt_bias"].double()
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if s["softplus"] else raw
    h = s["init"].double() * torch.exp(step[..., None] * A) + (step * x)[..., None] * _spread(s["B"].double(), D)
    y = torch.matmul(h[:, :, None], _spread(s["C"].double(), D)[..., None])[..., 0, 0] + s["D"].double() * x
    return y if s["z"] is None else y * torch.nn.functional.silu(s["z"].double()), h


def _exact_conv(s):
    """A sequence at a time: each tap as a row of one padded signal."""
    D, K = s["weight"].shape
    seqs, w = _Sequences(s), s["weight"].double()
    x = s["x"].reshape(-1, D).double()
    for i in range(seqs.count):
        at = slice(int(seqs.first[i]), int(seqs.first[i]) + seqs.n[i])
        past = torch.zeros(K - 1, D, device=x.device, dtype=torch.float64) if s["init"] is None else s["init"][i].double()
        sig = torch.cat([past, x[at]])
        taps = sig.unfold(0, K, 1) if seqs.n[i] else sig.new_zeros(0, D, K)   # [tokens, D, K]
        yield i, at, sig, taps, s["bias"].double() + (taps * w).sum(-1)


def _exact_conv_fwd(s):
    D, K = s["weight"].shape
    y = torch.zeros(s["x"].shape, device=s["x"].device, dtype=torch.float64)
    ends = []
    for i, at, sig, _, v in _exact_conv(s):
        y.view(-1, D)[at] = torch.nn.functional.silu(v) if s["silu"] else v
        ends.append(sig[sig.shape[0] - (K - 1):])
    return y, torch.stack(ends)


def _exact_conv_bwd(s):
    D, K = s["weight"].shape
    dev, w = s["x"].device, s["weight"].double()
    dx, firsts = torch.zeros(s["x"].shape, device=dev, dtype=torch.float64), []
    dw, db = torch.zeros_like(w), torch.zeros_like(s["bias"], dtype=torch.float64)
    for i, at, sig, taps, v in _exact_conv(s):
        dv = s["dy"].reshape(-1, D)[at].double()
        if s["silu"]:
            g = torch.sigmoid(v)
            dv = dv * (g + v * g * (1 - g))
        dw += (dv[..., None] * taps).sum(0)
        db += dv.sum(0)
        ds = torch.zeros_like(sig)
        if s["dfinal"] is not None:
            ds[sig.shape[0] - (K - 1):] = s["dfinal"][i].double()
        for k in range(K):
            ds[k:k + dv.shape[0]] += dv * w[:, k]
        dx.view(-1, D)[at] = ds[K - 1:]
        firsts.append(ds[:K - 1])
    return {"dx": dx, "dweight": dw, "dbias": db, "dinitial_window": torch.stack(firsts) if s["init"] is not None else None}


def _exact_norm(s, op):
    x = s["x"].double()
    if s["residual"] is None:
        stream = x
    else:
        total = x + s["residual"].double()
        stream = total.to(s["residual"].dtype).double()   # the stream's own values: what is normed
    inv = (stream.pow(2).sum(1) / stream.shape[1] + EPS).pow(-0.5)
    y = stream * inv[:, None] * s["weight"].double()
    told = None if s["residual"] is None else total
    if op == "norm_fwd":
        return y, told, inv
    parts = y.split(BLOCK, dim=1)
    scale = torch.stack([p.abs().amax(1) for p in parts], 1).clamp(min=F8_MAX * LEAST) / F8_MAX
    return torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), scale, told


def _exact_norm_bwd(s):
    r, dy, inv = s["stream"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    w = dy * s["weight"].double()
    dr = inv * w - inv ** 3 / r.shape[1] * r * (w * r).sum(1, keepdim=True)
    if s["dres"] is not None:
        dr = dr + s["dres"].double()
    return {"dx": dr, "dresidual": None if s["dres"] is None else dr, "dweight": (dy * r * inv).sum(0)}


def _exact_product(s):
    m, k = s["a"].shape
    n = s["w"].shape[0]
    out = torch.zeros(m, n, device=s["a"].device, dtype=torch.float64)
    if s["bias"] is not None:
        out += s["bias"].double()
    columns = torch.arange(n, device=out.device) // BLOCK
    for i in range(s["a_scale"].shape[1]):
        at = slice(i * BLOCK, min(k, (i + 1) * BLOCK))
        left = s["a"][:, at].double() * s["a_scale"][:, i:i + 1].double()
        right = s["w"][:, at].double() * s["w_scale"][columns, i:i + 1].double()
        out.addmm_(left, right.t())
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("norm"):
        return _exact_norm_bwd(s) if op == "norm_bwd" else _exact_norm(s, op)
    if op == "product":
        return _exact_product(s)
    if op == "conv_step":   # the first pass
        sig = torch.cat([s["init"], s["x"][:, None]], 1).double()
        v = torch.matmul(sig.permute(0, 2, 1)[:, :, None], s["weight"].double()[None, :, :, None])[..., 0, 0] + s["bias"].double()
        return torch.nn.functional.silu(v) if s["silu"] else v, sig[:, 1:]
    return {"scan_fwd": _exact_scan_fwd, "scan_bwd": _exact_scan_bwd, "scan_step": _exact_scan_step, "conv_fwd": _exact_conv_fwd,
            "conv_bwd": _exact_conv_bwd}[op](s)
