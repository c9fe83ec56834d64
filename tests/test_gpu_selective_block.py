"""The selective scan, its convolution, RMS norm and the 8-bit product as a block uses them: a prompt and then single
tokens, a training step captured and replayed, calls on two streams at once; and sizes between the other tests'.

Bars as in each operator's own tests: 1e-5 in norm for the scan and the convolution in fp32, 1e-6 for the norm and
the product with fp32 outputs.  Two ways of forming the same fp32 tensor differ by at most the sum of their bars.
"""
import numpy as np
import pytest
import torch

from oracle import selective as sel
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def near(got, ref, bar, size=None):
    got, ref = sel.f64(got), sel.f64(ref) if isinstance(ref, torch.Tensor) else np.asarray(ref)
    assert got.shape == ref.shape and np.isfinite(got).all()
    err, tol = np.linalg.norm(got - ref), bar * np.linalg.norm(ref if size is None else size) + 1e-30
    assert err <= tol, (err, tol)


def normal(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen)


class Block:
    """norm to 8 bits -> product to [x | z | dt | B | C] -> convolution of x -> scan -> norm to 8 bits -> product."""

    def __init__(self, width, dim, N, G, K):
        t = normal(0)
        self.dim, self.N, self.G = dim, N, G
        cols = 3 * dim + 2 * G * N
        c = lambda v: v.cuda()
        self.norm, self.norm2 = c(1 + 0.1 * t(width)), c(1 + 0.1 * t(dim))
        self.w_in, self.s_in = c(t(cols, width)).to(F8), c(0.5 + torch.rand(-(-cols // 128), -(-width // 128))) / width ** 0.5
        self.w_out, self.s_out = c(t(width, dim)).to(F8), c(0.5 + torch.rand(-(-width // 128), -(-dim // 128))) / dim ** 0.5
        self.taps, self.bias = c(t(dim, K)), c(t(dim))
        self.A, self.D, self.dt_bias = c(-torch.exp(0.3 * t(dim, N)) * (1 + torch.arange(N))), c(t(dim)), c(t(dim) - 3)

    def split(self, p):
        dim, n = self.dim, self.G * self.N
        keys = lambda at: p[..., at:at + n].unflatten(-1, (self.G, self.N))
        return p[..., :dim], p[..., dim:2 * dim], p[..., 2 * dim:3 * dim], keys(3 * dim), keys(3 * dim + n)

    def prompt(self, h, res, window, state):
        q, s, res = ssd.rms_norm_quant(h, self.norm, residual=res)
        p = ssd.matmul_fp8(q, s, self.w_in, self.s_in, out_dtype=torch.float32)
        x, z, dt, B, C = self.split(p)
        xc, window = ssd.causal_conv_fwd(x, self.taps, bias=self.bias, initial_window=window)
        y, state = ssd.selective_scan_fwd(xc, dt, self.A, B, C, D=self.D, z=z, dt_bias=self.dt_bias, initial_states=state)
        q2, s2, _ = ssd.rms_norm_quant(y, self.norm2)
        out = ssd.matmul_fp8(q2, s2, self.w_out, self.s_out, out_dtype=torch.float32)
        return dict(q=q, s=s, res=res, p=p, xc=xc, y=y, q2=q2, s2=s2, out=out, window=window, state=state)

    def token(self, h, res, window, state):
        q, s, res = ssd.rms_norm_quant(h, self.norm, residual=res)
        p = ssd.matmul_fp8(q, s, self.w_in, self.s_in, out_dtype=torch.float32)
        x, z, dt, B, C = self.split(p)
        xc = ssd.causal_conv_step(x, window, self.taps, bias=self.bias)
        y = ssd.selective_scan_step(xc, dt, self.A, B, C, state, D=self.D, z=z, dt_bias=self.dt_bias)
        q2, s2, _ = ssd.rms_norm_quant(y, self.norm2)
        return y, ssd.matmul_fp8(q2, s2, self.w_out, self.s_out, out_dtype=torch.float32)


def test_prompt_then_tokens():
    b, T, more, width, dim, N, G, K = 2, 150, 6, 160, 96, 16, 2, 4
    m, t = Block(width, dim, N, G, K), normal(1)
    h, res = t(b, T + more, width).cuda(), t(b, T + more, width).cuda()
    cut = lambda v, a, e: v[:, a:e].contiguous()
    whole = m.prompt(h, res, None, None)
    torch.cuda.synchronize()
    # every stage from what it was given
    near(whole["res"], h.double() + res.double(), 2.0 ** -24)
    near(whole["p"], sel.matmul_fp8(whole["q"].view(-1, width), whole["s"].view(b * (T + more), -1), m.w_in, m.s_in)[0].reshape(b, T + more, -1), 1e-6)
    x, z, dt, B, C = m.split(whole["p"])
    xc, win = sel.conv_forward(x, m.taps, m.bias, True)
    near(whole["xc"], xc, 1e-5)
    y, fin = sel.scan_forward(whole["xc"], dt, m.A, B, C, D=m.D, z=z, dt_bias=m.dt_bias)
    near(whole["y"], y, 1e-5)
    near(whole["state"], fin, 1e-5)
    near(whole["out"], sel.matmul_fp8(whole["q2"].view(-1, dim), whole["s2"].view(b * (T + more), -1), m.w_out, m.s_out)[0].reshape(b, T + more, -1), 1e-6)
    # a prompt, then tokens one by one.  A row's norm does not depend on the other rows; the product's sums do,
    # in their order (1e-6 each way), and the scan's and the convolution's (1e-5 each way, twice)
    first = m.prompt(cut(h, 0, T), cut(res, 0, T), None, None)
    window, state = first["window"], first["state"]
    assert torch.equal(first["q"].view(torch.uint8), cut(whole["q"], 0, T).view(torch.uint8)) and torch.equal(first["s"], cut(whole["s"], 0, T))
    ys = [m.token(h[:, i].contiguous(), res[:, i].contiguous(), window, state)[0] for i in range(T, T + more)]
    torch.cuda.synchronize()
    near(torch.stack(ys, 1), whole["y"][:, T:], 4.2e-5)
    near(state, whole["state"], 4.2e-5)
    near(window, whole["window"], 2e-6)


def test_tokens_captured():
    """Single tokens in a graph: the states move on at every replay as they do eagerly."""
    b, width, dim, N, G, K = 3, 128, 64, 16, 1, 4
    m, t = Block(width, dim, N, G, K), normal(2)
    h, res, window, state = t(b, width).cuda(), t(b, width).cuda(), t(b, K - 1, dim).cuda(), t(b, dim, N).cuda()
    w0, s0 = window.clone(), state.clone()
    m.token(h, res, window, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, out = m.token(h, res, window, state)
    window.copy_(w0), state.copy_(s0)
    we, se = w0.clone(), s0.clone()
    for i in range(4):
        h.copy_(normal(10 + i)(b, width))
        graph.replay()
        ye, oe = m.token(h, res, we, se)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(out, oe) and torch.equal(state, se) and torch.equal(window, we), i


def train(p):
    """norm -> convolution -> scan, and back."""
    y, r, rstd = ssd.rms_norm_fwd(p["h"], p["norm"], residual=p["res"])
    xc, _ = ssd.causal_conv_fwd(y, p["taps"], bias=p["bias"], want_window=False)
    kw = dict(D=p["D"], z=p["z"], dt_bias=p["dt_bias"])
    ins = (xc, p["dt"], p["A"], p["B"], p["C"])
    out, _ = ssd.selective_scan_fwd(*ins, want_final=False, **kw)
    gs = ssd.selective_scan_bwd(*ins, p["dy"], want_dinit=False, **kw)
    gc = ssd.causal_conv_bwd(y, p["taps"], gs["dx"], bias=p["bias"], want_dinit=False)
    gn = ssd.rms_norm_bwd(r, gc["dx"], rstd, p["norm"], dresidual=p["dr"])
    grads = {**{"scan." + k: v for k, v in gs.items()}, **{"conv." + k: v for k, v in gc.items()}, "norm.dx": gn["dx"], "norm.dweight": gn["dweight"]}
    return dict(out=out, y=y, xc=xc, r=r, **{k: v for k, v in grads.items() if v is not None})


def train_case(b, T, dim, N, G, K, dtype):
    t = normal(3)
    c = lambda v, d=torch.float32: v.to(d).cuda()
    return dict(h=c(t(b, T, dim), dtype), res=c(t(b, T, dim)), norm=c(1 + 0.1 * t(dim)), taps=c(t(dim, K)), bias=c(t(dim)), D=c(t(dim)),
                z=c(t(b, T, dim), dtype), dt=c(0.5 * t(b, T, dim), dtype), dt_bias=c(t(dim) - 3), A=c(-torch.exp(0.3 * t(dim, N)) * (1 + torch.arange(N))),
                B=c(t(b, T, G, N), dtype), C=c(t(b, T, G, N), dtype), dy=c(t(b, T, dim), dtype), dr=c(t(b, T, dim)))


def test_training_gradients():
    p = train_case(2, 130, 72, 16, 2, 4, torch.float32)
    g = train(p)
    torch.cuda.synchronize()
    y, rstd = sel.rms_norm(sel.f64(p["h"]) + sel.f64(p["res"]), sel.f64(p["norm"]))[:2]
    xc, _ = sel.conv_forward(y, p["taps"], p["bias"], True)
    ins = dict(x=xc, dt=p["dt"], A=p["A"], B=p["B"], C=p["C"], D=p["D"], z=p["z"], dt_bias=p["dt_bias"])
    out, _ = sel.scan_forward(**ins)
    near(g["out"], out, 3e-5)
    rs = sel.scan_backward(**ins, dy=p["dy"])
    rc = sel.conv_backward(y, p["taps"], rs["dx"], p["bias"], True)
    rn = sel.rms_norm_backward(sel.f64(p["h"]) + sel.f64(p["res"]), rc["dx"], rstd, sel.f64(p["norm"]), sel.f64(p["dr"]))
    # a chain's bar is its operators' together: norm, convolution and scan forward, then back; what comes in off by
    # a part of itself goes out so, against the size of the terms
    for k in ("dx", "ddt", "dB", "dC", "dA", "dD", "ddt_bias", "dz"):
        near(g["scan." + k], rs[k], 4e-5, rs["sizes"].get(k))
    near(g["conv.dx"], rc["dx"], 6e-5)
    near(g["conv.dweight"], rc["dweight"], 6e-5, rc["sizes"]["dweight"])
    near(g["norm.dx"], rn[0], 8e-5)
    near(g["norm.dweight"], rn[1], 8e-5, rn[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_step_captured(dtype):
    p = train_case(2, 300, 136, 16, 1, 4, dtype)
    want = {k: v.clone() for k, v in train(p).items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train(p)
    for i in range(3):
        for v in got.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), i
        assert all(torch.equal(v, want[k]) for k, v in train(p).items())
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls in flight together, each with its own workspace: the shares of a product's k, a scan in chunks, gradients."""
    p = train_case(1, 900, 64, 16, 1, 4, torch.float32)
    t = normal(4)
    a, sa = t(5, 2048).cuda().to(F8), torch.rand(5, 16).cuda()
    w, sw = t(192, 2048).cuda().to(F8), torch.rand(2, 16).cuda()
    assert ssd.matmul_fp8(a, sa, w, sw).shape == (5, 192)
    one, two = train(p), ssd.matmul_fp8(a, sa, w, sw)
    want = {k: v.clone() for k, v in one.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append((train(p), ssd.matmul_fp8(a, sa, w, sw)))
    torch.cuda.synchronize()
    for g, o in got:
        assert all(torch.equal(g[k], want[k]) for k in want) and torch.equal(o, two)


@pytest.mark.parametrize("dim", [4, 12, 20, 36])
@pytest.mark.parametrize("b", [1, 3])
def test_convolution_of_fours_that_are_not_eights(dim, b):
    """Rows of whole fours but not eights, in buffers with something behind them."""
    t, K, T = normal(dim), 4, 9
    x, w, bias, win, dy = t(b, T, dim).bfloat16(), t(dim, K), t(dim), t(b, K - 1, dim).bfloat16(), t(b, T, dim).bfloat16()
    def behind(shape, fill=None):
        n = int(np.prod(shape))
        buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        if fill is not None:
            buf[:n] = fill.reshape(-1).cuda()
        return buf, buf[:n].view(shape)
    wb, window = behind((b, K - 1, dim), win)
    ys, bufs = [], [wb]
    for i in range(T):
        yb, y = behind((b, dim))
        bufs.append(yb)
        ys.append(ssd.causal_conv_step(x.cuda()[:, i], window, w.cuda(), bias=bias.cuda(), y=y))
    yb, y = behind((b, T, dim))
    fb, fin = behind((b, K - 1, dim))
    ssd.causal_conv_fwd(x.cuda(), w.cuda(), bias=bias.cuda(), initial_window=win.cuda(), y=y, final_window=fin)
    db, dx = behind((b, T, dim))
    g = ssd.causal_conv_bwd(x.cuda(), w.cuda(), dy.cuda(), bias=bias.cuda(), initial_window=win.cuda(), grads=dict(dx=dx))
    torch.cuda.synchronize()
    assert all((v[-64:] == 7).all() for v in [*bufs, yb, fb, db])
    yr, fr = sel.conv_forward(x, w, bias, True, win)
    bar = 2.0 ** -8 + 1e-5
    near(torch.stack(ys, 1), yr, bar)
    near(y, yr, bar)
    assert np.array_equal(sel.f64(window), fr) and np.array_equal(sel.f64(fin), fr)
    r = sel.conv_backward(x, w, dy, bias, True, win)
    near(g["dx"], r["dx"], bar)
    near(g["dweight"], r["dweight"], 1e-5, r["sizes"]["dweight"])


@pytest.mark.parametrize("nseq", [1023, 1024, 1025, 1700])
def test_many_short_segments(nseq):
    """More segments than are put in order by length, some without tokens, and the gradients of them all."""
    rng = np.random.default_rng(nseq)
    lengths = rng.integers(0, 4, nseq).tolist()
    T, dim, N = sum(lengths), 9, 4
    t = normal(nseq)
    ids = torch.repeat_interleave(torch.arange(nseq, dtype=torch.int32), torch.tensor(lengths)).cuda()
    p = dict(x=t(1, T, dim), dt=t(1, T, dim) - 2, A=-torch.exp(t(dim, N)), B=t(1, T, 1, N), C=t(1, T, 1, N))
    s0, dy, df = t(nseq, dim, N), t(1, T, dim), t(nseq, dim, N)
    g = {k: v.cuda() for k, v in p.items()}
    kw = dict(initial_states=s0.cuda(), seq_idx=ids, nseq=nseq)
    y, f = ssd.selective_scan_fwd(**g, **kw)
    gr = ssd.selective_scan_bwd(**g, dy=dy.cuda(), dfinal_states=df.cuda(), **kw)
    torch.cuda.synchronize()
    yr, fr = sel.scan_forward(**p, init=s0, lengths=lengths)
    near(y, yr, 1e-5)
    near(f, fr, 1e-5)
    r = sel.scan_backward(**p, dy=dy, init=s0, dfinal=df, lengths=lengths)
    near(gr["dx"], r["dx"], 1e-5)
    near(gr["ddt"], r["ddt"], 1e-5, r["sizes"]["ddt"])
    near(gr["dA"], r["dA"], 1e-5, r["sizes"]["dA"])
    near(gr["dinitial_states"], r["dinitial_states"], 1e-5)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_states_at_any_element(off):
    """States and A that start at any fp32 element, with rows of whole fours."""
    b, T, dim, N = 2, 33, 20, 16
    t = normal(off)
    def at(v):
        buf = torch.zeros(v.numel() + 8, device="cuda")
        o = buf[off:off + v.numel()].view(v.shape)
        o.copy_(v)
        return o
    p = dict(x=t(b, T, dim), dt=t(b, T, dim) - 2, A=-torch.exp(t(dim, N)), B=t(b, T, 1, N), C=t(b, T, 1, N))
    s0, df, dy = t(b, dim, N), t(b, dim, N), t(b, T, dim)
    g = {k: v.cuda() for k, v in p.items()}
    g["A"] = at(p["A"])
    fin = at(torch.zeros(b, dim, N))
    y, f = ssd.selective_scan_fwd(**g, initial_states=at(s0), final_states=fin)
    gr = ssd.selective_scan_bwd(**g, dy=dy.cuda(), initial_states=at(s0), dfinal_states=at(df))
    state = at(s0)
    for i in range(T):
        ys = ssd.selective_scan_step(g["x"][:, i], g["dt"][:, i], g["A"], g["B"][:, i], g["C"][:, i], state)
    torch.cuda.synchronize()
    yr, fr = sel.scan_forward(**p, init=s0)
    near(y, yr, 1e-5)
    near(ys, yr[:, -1], 1e-5, yr)
    near(f, fr, 1e-5)
    near(state, fr, 1e-5)
    r = sel.scan_backward(**p, dy=dy, init=s0, dfinal=df)
    near(gr["dinitial_states"], r["dinitial_states"], 1e-5)
    near(gr["dA"], r["dA"], 1e-5, r["sizes"]["dA"])
