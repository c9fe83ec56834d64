"""The gated delta rule (prompt, gradients, one token) and layer norm (forward, gradients), as cases to measure.

The gated delta rule keeps one state S [dstate, headdim] for every head, key k_t
and query q_t [dstate] shared by the heads of a group, value v_t [headdim], a log
decay g_t <= 0 and a step size beta_t:

    u_t = v_t - e^{g_t} S_{t-1}^T k_t
    S_t = e^{g_t} S_{t-1} + beta_t k_t u_t^T
    y_t = scale S_t^T q_t

Layer norm over the last axis of x [rows, dim]: y = (x - mean) rstd weight + bias,
rstd = 1 / sqrt(var + eps).

Where ``own`` is false ``run`` computes them with elementary torch operations in
32 bits; where it is true it calls the library.
"""
import math

import torch

own = False

CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gdr(op, batch, seqlen, nheads, headdim, dstate, ngroups, dtype="bf16", init=False, nseq=0, lo=0, hi=0):
    return {"op": op, "batch": batch, "seqlen": seqlen, "nheads": nheads, "headdim": headdim, "dstate": dstate,
            "ngroups": ngroups, "dtype": dtype, "init": init, "nseq": nseq, "lo": lo, "hi": hi}


def _norm(op, rows, dim, dtype="bf16", affine=True):
    return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "affine": affine}


def listed():
    cases = {
        # a short prompt that continues a carried state: what a chat turn prefills; latency counts
        "gdr_fwd short_turn": _gdr("gdr_fwd", 1, 77, 8, 64, 64, 8, init=True),
        # one long document at the long workload's heads (16K tokens, N = 256): few heads, a long chain
        "gdr_fwd long_document": _gdr("gdr_fwd", 1, 16384, 32, 64, 256, 1),
        # a serving batch of prompts of different lengths packed into one stream, each with its carried state
        "gdr_fwd packed_prompts": _gdr("gdr_fwd", 1, 0, 64, 64, 128, 8, init=True, nseq=16, lo=128, hi=2048),
        # gradients in 32 bits at odd sizes: packed sequences down to one token, carried states, their gradients
        "gdr_bwd odd_fp32": _gdr("gdr_bwd", 1, 0, 6, 48, 80, 3, dtype="fp32", init=True, nseq=9, lo=1, hi=301),
        # gradients of the small training workload (24 heads, N = 64) from carried states
        "gdr_bwd small_train": _gdr("gdr_bwd", 2, 2048, 24, 64, 64, 1, init=True),
        # gradients of one training step at the 2.7B-scale heads
        "gdr_bwd train_2.7B": _gdr("gdr_bwd", 8, 2048, 80, 64, 128, 1),
        # one token of one sequence, two value heads for each key head
        "gdr_step single": _gdr("gdr_step", 1, 1, 32, 128, 128, 16),
        # one token of each of 64 sequences at the 2.7B-scale heads (the decode workload)
        "gdr_step decode_b64": _gdr("gdr_step", 64, 1, 80, 64, 128, 1),
        # the norm before a decode step: one token of each of 64 sequences at the 2.7B model width
        "norm_fwd decode_rows": _norm("norm_fwd", 64, 2560),
        # the norm before a training step's block: 8 x 2048 tokens
        "norm_fwd train_rows": _norm("norm_fwd", 16384, 2560),
        # gradients at a width that no vector divides, in 32 bits
        "norm_bwd odd_fp32": _norm("norm_bwd", 1001, 1531, dtype="fp32"),
        # gradients of a training step's norm at the inner width of 80 heads of 64
        "norm_bwd train_rows": _norm("norm_bwd", 16384, 5120),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_bwd", "gdr_bwd", "gdr_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("norm"):
        dim = _log_int(rng, 16, 8192)
        return _norm(op, _log_int(rng, 1, min(65536, (32 << 20) // dim)), dim, dtype, rng.random() < 0.8)
    ngroups = rng.choice([1, 2, 3, 4, 8])
    nheads = ngroups * rng.choice([1, 2, 4, 5])
    headdim, dstate = 16 * rng.randint(1, 8), 16 * rng.randint(2, 16)
    if op == "gdr_step":
        return _gdr(op, _log_int(rng, 1, 128), 1, nheads, headdim, dstate, ngroups, dtype, True)
    most = 2048 if op == "gdr_bwd" or dtype == "fp32" else 8192
    if rng.random() < 0.5:
        nseq = _log_int(rng, 2, 40)
        hi = max(2, _log_int(rng, 2, most) // 2)
        return _gdr(op, 1, 0, nheads, headdim, dstate, ngroups, dtype, rng.random() < 0.5, nseq, rng.randint(1, hi), hi)
    seqlen = _log_int(rng, 1, most)
    return _gdr(op, rng.randint(1, max(1, min(4, most // seqlen))), seqlen, nheads, headdim, dstate, ngroups, dtype,
                rng.random() < 0.5)


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
    el = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    if case["op"].startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        # activations of a residual stream: rows of different scale, off centre
        x = (normal(rows, dim) * (0.5 + normal(rows, 1).abs()) + normal(rows, 1)).to(el)
        s = {"op": case["op"], "x": x, "weight": None, "bias": None}
        if case["affine"]:
            s["weight"], s["bias"] = 1 + 0.1 * normal(dim), 0.1 * normal(dim)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, dim).to(el)
            # what the forward pass of the same step left
            xf = x.double()
            mean = xf.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((xf - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        return s

    H, P, N, G = case["nheads"], case["headdim"], case["dstate"], case["ngroups"]
    packed = case["nseq"] > 0
    B, T = (1, _tokens(case)) if packed else (case["batch"], case["seqlen"])
    lead = (B,) if case["op"] == "gdr_step" else (B, T)

    def unit(*shape):   # keys and queries come normalised, as the layers that use the rule make them
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(el)

    s = {"op": case["op"], "scale": 1 / math.sqrt(N), "seq_idx": None, "nseq": None, "lengths": None, "init": None}
    s["q"], s["k"] = unit(*lead, G, N), unit(*lead, G, N)
    s["v"] = normal(*lead, H, P).to(el)
    # decays of e^{-A softplus(dt)}, A log-uniform over heads, as the selective state space layers draw them
    A = torch.exp(torch.rand(H, device="cuda", generator=gen) * math.log(16.0))
    s["g"] = (-A * torch.nn.functional.softplus(normal(*lead, H) * 0.5 - 3.0)).to(el)
    s["beta"] = torch.sigmoid(normal(*lead, H)).to(el)
    states = case["nseq"] if packed else B
    if case["init"] or case["op"] == "gdr_step":
        s["init"] = 0.3 * normal(states, H, P, N)
    if packed:
        s["lengths"], s["nseq"] = _lengths(case), case["nseq"]
        s["seq_idx"] = torch.repeat_interleave(torch.arange(s["nseq"], device="cuda", dtype=torch.int32),
                                               torch.tensor(s["lengths"], device="cuda"), output_size=T)
    if case["op"] == "gdr_bwd":
        s["dy"] = normal(*lead, H, P).to(el)
        s["dfinal"] = 0.3 * normal(states, H, P, N) if case["init"] else None
    if case["op"] == "gdr_step":
        s["state"] = s["init"].clone()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rows_of(s):
    """Packed streams as a batch: the index [nseq, longest] of every sequence's tokens, and which of them are real."""
    dev = s["q"].device
    n = torch.tensor(s["lengths"], device=dev)
    at = torch.arange(max(s["lengths"]), device=dev)
    real = at < n[:, None]
    return torch.where(real, (n.cumsum(0) - n)[:, None] + at, 0), real


def _batched(x, s, rows):
    """[batch, tokens, ...] -> [sequences, heads or groups, chunks, 64, width] in 32 bits, zero behind the last token."""
    x = x.float()
    if x.dim() == 3:
        x = x[..., None]
    if rows is not None:
        x = x[0][rows[0]] * rows[1][:, :, None, None]
    more = -x.shape[1] % CHUNK
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, more))
    b, t, h, d = x.shape
    return x.view(b, t // CHUNK, CHUNK, h, d).permute(0, 3, 1, 2, 4).contiguous()


def _flat(x, like, rows):
    """The inverse of _batched, rounded to the type of `like`."""
    b, h, c, q, d = x.shape
    x = x.permute(0, 2, 3, 1, 4).reshape(b, c * q, h, d)
    if rows is None:
        x = x[:, :like.shape[1]]
    else:
        x = x[:, :rows[1].shape[1]][rows[1]][None]
    return x.reshape(like.shape).to(like.dtype)


def _unit_lower_inverse(m):
    """The inverse of unit lower triangular [.., 64, 64], from blocks of 1, 2, 4 .. 32."""
    inv = torch.eye(CHUNK, device=m.device).expand_as(m).clone()
    n = 1
    while n < CHUNK:
        b = CHUNK // (2 * n)
        t = inv.unflatten(-1, (b, 2, n)).unflatten(-4, (b, 2, n))
        l = m.unflatten(-1, (b, 2, n)).unflatten(-4, (b, 2, n))
        d = torch.arange(b, device=m.device)
        # the two inverses on the diagonal of each block of 2n, and what lies below the first
        a, c, low = t[..., d, 0, :, d, 0, :], t[..., d, 1, :, d, 1, :], l[..., d, 1, :, d, 0, :]
        t[..., d, 1, :, d, 0, :] = -(c @ low @ a)
        n *= 2
    return inv


def _heads(x, H):
    return x.repeat_interleave(H // x.shape[1], dim=1)


def _chunk_terms(s, rows):
    """Everything of the chunked rule that no state enters."""
    H = s["v"].shape[2]
    q, k = (_heads(_batched(s[n], s, rows), H) for n in ("q", "k"))
    v, g, beta = (_batched(s[n], s, rows) for n in ("v", "g", "beta"))
    cs = g.double().cumsum(3)
    at = torch.arange(CHUNK, device=q.device)
    gap = cs - cs.transpose(3, 4)
    low = (at[:, None] >= at).expand_as(gap)
    gamma = torch.where(low, gap, -torch.inf).exp().float()
    kt = k.transpose(3, 4).contiguous()
    A = torch.tril(gamma * (k @ kt), -1)
    inv = _unit_lower_inverse(A * beta.transpose(3, 4) + torch.eye(CHUNK, device=q.device))
    return {"q": q, "k": k, "kt": kt, "v": v, "beta": beta, "gamma": gamma, "A": A, "inv": inv,
            "since": cs.exp().float(), "till": (cs[..., -1:, :] - cs).exp().float(), "whole": cs[..., -1:, :].exp().float()}


def _first_state(s, v):
    b, h, _, _, p = v.shape
    if s["init"] is None:
        return v.new_zeros(b, h, s["q"].shape[-1], p)
    return s["init"].transpose(2, 3).contiguous()


def _chunk_states(s, c):
    """The states that enter every chunk, the last one, and every chunk's u."""
    S = _first_state(s, c["v"])
    entering, us = [], []
    for i in range(c["v"].shape[2]):
        u = c["inv"][:, :, i] @ (c["v"][:, :, i] - c["since"][:, :, i] * (c["k"][:, :, i] @ S))
        entering.append(S)
        us.append(u)
        S = c["whole"][:, :, i] * S + c["kt"][:, :, i] @ (c["till"][:, :, i] * c["beta"][:, :, i] * u)
    return torch.stack(entering, 2), S, torch.stack(us, 2)


def _plain_fwd(s):
    rows = _rows_of(s) if s["nseq"] else None
    c = _chunk_terms(s, rows)
    S, last, u = _chunk_states(s, c)
    y = c["since"] * (c["q"] @ S) + (c["gamma"] * (c["q"] @ c["kt"])) @ (c["beta"] * u)
    return _flat(s["scale"] * y, s["v"], rows), last.transpose(2, 3).contiguous()


def _plain_bwd(s):
    rows = _rows_of(s) if s["nseq"] else None
    c = _chunk_terms(s, rows)
    S, last, u = _chunk_states(s, c)
    q, k, kt, beta, gamma = c["q"], c["k"], c["kt"], c["beta"], c["gamma"]
    dy = s["scale"] * _batched(s["dy"], s, rows)
    # gradients of beta u that come from this chunk's outputs, and of the state from its outputs
    dw0 = (gamma * (q @ kt)).transpose(3, 4).contiguous() @ dy
    qt = q.transpose(3, 4).contiguous()
    invt = c["inv"].transpose(3, 4).contiguous()
    At = c["A"].transpose(3, 4).contiguous()
    D = torch.zeros_like(last) if s["dfinal"] is None else s["dfinal"].transpose(2, 3).contiguous()
    after, dws, dus = [], [], []
    for i in range(q.shape[2] - 1, -1, -1):
        dw = dw0[:, :, i] + c["till"][:, :, i] * (k[:, :, i] @ D)
        du = invt[:, :, i] @ (beta[:, :, i] * dw)
        after.append(D)
        dws.append(dw - At[:, :, i] @ du)
        dus.append(du)
        D = c["whole"][:, :, i] * D + qt[:, :, i] @ (c["since"][:, :, i] * dy[:, :, i]) - kt[:, :, i] @ (c["since"][:, :, i] * du)
    D1, dw, du = (torch.stack(x[::-1], 2) for x in (after, dws, dus))
    w = beta * u
    ut = w.transpose(3, 4).contiguous()
    St, Dt = S.transpose(3, 4).contiguous(), D1.transpose(3, 4).contiguous()
    W = gamma * (dy @ ut)
    Z = torch.tril(gamma * (du @ ut), -1)
    dq = c["since"] * (dy @ St) + W @ k
    dk_row = -(c["since"] * (du @ St)) - Z @ k
    dk_col = c["till"] * (w @ Dt) + W.transpose(3, 4).contiguous() @ q - Z.transpose(3, 4).contiguous() @ k
    dcs = (q * dq + k * dk_row - k * dk_col).double().sum(-1, keepdim=True)
    end = c["whole"][..., 0, 0] * (D1 * S).double().sum((3, 4)) + ((k * c["till"]) * (w @ Dt)).double().sum((3, 4))
    dg = dcs.flip(3).cumsum(3).flip(3) + end[:, :, :, None, None]
    dbeta = (dw * u).sum(-1, keepdim=True)
    G = s["q"].shape[2]
    dq, dk = (x.unflatten(1, (G, -1)).sum(2) for x in (dq, dk_row + dk_col))
    return {"dq": _flat(dq, s["q"], rows), "dk": _flat(dk, s["k"], rows), "dv": _flat(du, s["v"], rows),
            "dg": _flat(dg.float(), s["g"], rows), "dbeta": _flat(dbeta, s["beta"], rows),
            "dinitial_states": D.transpose(2, 3).contiguous() if s["init"] is not None else None}


def _plain_step(s):
    H = s["v"].shape[1]
    q, k = (_heads(s[n].float(), H) for n in ("q", "k"))
    S = s["state"] * torch.exp(s["g"].float())[..., None, None]
    u = s["beta"].float()[..., None] * (s["v"].float() - (S * k[:, :, None]).sum(-1))
    S = S + u[..., None] * k[:, :, None]
    y = s["scale"] * (S * q[:, :, None]).sum(-1)
    # the state moves on in place: the next pass is the next token
    return y.to(s["v"].dtype), s["state"].copy_(S)


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy if s["weight"] is None else dy * s["weight"]
    dx = (w - w.mean(1, keepdim=True) - xhat * (w * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["weight"] is None:
        return {"dx": dx.to(s["x"].dtype)}
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if own:
        from ssd_chunked_scan_amd import ssd
        if op == "gdr_fwd":
            return ssd.gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], initial_states=s["init"],
                               seq_idx=s["seq_idx"], nseq=s["nseq"])
        if op == "gdr_bwd":
            return ssd.gdr_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], scale=s["scale"],
                               initial_states=s["init"], dfinal_states=s["dfinal"], seq_idx=s["seq_idx"],
                               nseq=s["nseq"], want_dinit=s["init"] is not None)
        if op == "gdr_step":
            return ssd.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"]), s["state"]
        if op == "norm_fwd":
            return ssd.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        return ssd.layer_norm_bwd(s["x"], s["dy"], s["mean"], s["rstd"], s["weight"])
    if op == "gdr_fwd":
        return _plain_fwd(s)
    if op == "gdr_bwd":
        return _plain_bwd(s)
    if op == "gdr_step":
        return _plain_step(s)
    return _plain_norm_fwd(s) if op == "norm_fwd" else _plain_norm_bwd(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op.startswith("norm"):
        n, d = case["rows"] * case["dim"], case["dim"]
        par = 8 * d if case["affine"] else 0
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * case["rows"] + par, "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + 3 * par // 2, "flops": 14 * n}
    H, P, N, G = case["nheads"], case["headdim"], case["dstate"], case["ngroups"]
    T = _tokens(case)
    states = 4 * H * P * N * (case["nseq"] or case["batch"])
    token = (2 * G * N + H * P + 2 * H) * e   # q, k, v, g, beta
    if op == "gdr_step":
        return {"bytes": T * (token + H * P * e) + 2 * states, "flops": 7 * T * H * P * N}
    # the recurrence itself: the decay, k S, the rank-one update and q S of every token
    if op == "gdr_fwd":
        return {"bytes": T * (token + H * P * e) + states * (2 if case["init"] else 1) + (4 * T if case["nseq"] else 0),
                "flops": 7 * T * H * P * N}
    return {"bytes": T * (2 * token + H * P * e) + states * (3 if case["init"] else 0) + (4 * T if case["nseq"] else 0),
            "flops": 20 * T * H * P * N}


# ---------------------------------------------------------------------------
# the definition, token by token in 64 bits
# ---------------------------------------------------------------------------

class _Tokens:
    """Token t of every sequence still running, in 64 bits, heads in the place of groups."""

    def __init__(self, s):
        dev = s["q"].device
        packed = s["nseq"] is not None
        B, T, H, _ = s["v"].shape
        self.n = s["lengths"] if packed else [T] * B
        off = [sum(self.n[:i]) for i in range(len(self.n))] if packed else [T * i for i in range(B)]
        self.off, self.length = torch.tensor(off, device=dev), torch.tensor(self.n, device=dev)
        self.H, self.s, self.steps = H, s, max(self.n)

    def at(self, t, names):
        """(where, which, the values of `names`): the rows of token t, and the sequences that have one."""
        which = torch.nonzero(self.length > t)[:, 0]
        rows = self.off[which] + t
        out = []
        for n in names:
            x = self.s[n].flatten(0, 1)[rows].double()
            out.append(x.repeat_interleave(self.H // x.shape[1], dim=1))
        return rows, which, out

    def first(self):
        s = self.s
        if s["init"] is not None:
            return s["init"].double().clone()
        return torch.zeros(len(self.n), self.H, s["v"].shape[3], s["q"].shape[3], device=s["q"].device, dtype=torch.float64)


def _advance(S, q, k, v, g, beta):
    """One token: the state [.., P, N] after it, and u."""
    S = S * g.exp()[..., None, None]
    u = v - torch.matmul(S, k[..., None])[..., 0]
    return S + (beta[..., None] * u)[..., None] * k[:, :, None], u


def _exact_fwd(s):
    tk = _Tokens(s)
    S = tk.first()
    y = torch.zeros(s["v"].shape, device=S.device, dtype=torch.float64)
    yf = y.flatten(0, 1)
    for t in range(tk.steps):
        rows, which, (q, k, v, g, beta) = tk.at(t, ("q", "k", "v", "g", "beta"))
        new, _ = _advance(S[which], q, k, v, g, beta)
        S[which] = new
        yf[rows] = s["scale"] * torch.matmul(new, q[..., None])[..., 0]
    return y, S


def _exact_bwd(s):
    tk = _Tokens(s)
    names = ("q", "k", "v", "g", "beta")
    S = tk.first()
    kept, every = [], 32
    for t in range(tk.steps):
        if t % every == 0:
            kept.append(S.clone())
        _, which, x = tk.at(t, names)
        S[which] = _advance(S[which], *x)[0]
    D = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double().clone()
    grads = {"d" + n: torch.zeros(s[n].shape, device=S.device, dtype=torch.float64) for n in names}
    flat = {n: x.flatten(0, 1) for n, x in grads.items()}
    G = s["q"].shape[2]
    for c in range(len(kept) - 1, -1, -1):
        S, before = kept[c], []
        for t in range(c * every, min(tk.steps, (c + 1) * every)):
            _, which, x = tk.at(t, names)
            before.append(S[which].clone())
            S[which] = _advance(S[which], *x)[0]
        for t in range(min(tk.steps, (c + 1) * every) - 1, c * every - 1, -1):
            rows, which, (q, k, v, g, beta, dy) = tk.at(t, names + ("dy",))
            S0 = before.pop()
            S1, u = _advance(S0, q, k, v, g, beta)
            a = g.exp()[..., None, None]
            dy = s["scale"] * dy
            E = D[which] + dy[..., None] * q[:, :, None]
            Ek = torch.matmul(E, k[..., None])[..., 0]
            du = beta[..., None] * Ek
            dk = torch.matmul((beta[..., None] * u)[:, :, None], E)[:, :, 0] - torch.matmul(du[:, :, None], a * S0)[:, :, 0]
            dq = torch.matmul(dy[:, :, None], S1)[:, :, 0]
            E = E - du[..., None] * k[:, :, None]
            flat["dq"][rows], flat["dk"][rows] = (x.unflatten(1, (G, -1)).sum(2) for x in (dq, dk))
            flat["dv"][rows], flat["dbeta"][rows] = du, (Ek * u).sum(-1)
            flat["dg"][rows] = (E * S0).sum((2, 3)) * a[..., 0, 0]
            D[which] = a * E
    grads["dinitial_states"] = D if s["init"] is not None else None
    return grads


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gdr_fwd":
        return _exact_fwd(s)
    if op == "gdr_bwd":
        return _exact_bwd(s)
    if op == "gdr_step":   # the first pass
        H = s["v"].shape[1]
        q, k = (s[n].double().repeat_interleave(H // s[n].shape[1], dim=1) for n in ("q", "k"))
        S, _ = _advance(s["init"].double(), q, k, *(s[n].double() for n in ("v", "g", "beta")))
        return s["scale"] * torch.matmul(S, q[..., None])[..., 0], S
    x = s["x"].double()
    if op == "norm_fwd":
        mean, var = x.mean(1), x.var(1, unbiased=False)
        y = (x - mean[:, None]) / (var + EPS).sqrt()[:, None]
        y = y if s["weight"] is None else y * s["weight"].double() + s["bias"].double()
        return y, mean, 1 / (var + EPS).sqrt()
    dim, dy = x.shape[1], s["dy"].double()
    mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xc = x - mean
    w = dy if s["weight"] is None else dy * s["weight"].double()
    dx = rstd * w - rstd / dim * w.sum(1, keepdim=True) - rstd ** 3 / dim * xc * (w * xc).sum(1, keepdim=True)
    if s["weight"] is None:
        return {"dx": dx}
    return {"dx": dx, "dweight": (dy * xc * rstd).sum(0), "dbias": dy.sum(0)}
