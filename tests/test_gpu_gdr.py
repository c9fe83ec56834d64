"""GPU parity of the gated delta rule (ssd_gdr_fwd, ssd_gdr_bwd, ssd_gdr_step) against
the fp64 recurrence, through the Python binding.

Errors are relative L2 norms per (batch row or segment, head) of y, the states and
the gradients (q, k per group).  Bars, counted before the first run:

  fp32   1e-4, the framework's bar.
  bf16   operands of 8 bits are off by at most 2^-8 of themselves.  y takes three such
         roundings (S or U, the pair matrix, y itself), dq and dk as many, dbeta three
         (U, H, itself), dg three: 3 * 2^-8 = 1.2e-2, and the parts of one sum add in
         norm: the framework's bar of 2e-2.  dv takes one rounding, of itself: 2^-8.
  states (fp32, also of bf16 problems) a chain value is handed over as two numbers of
         8 bits, off by at most 2^-16 of itself, and a product drops the product of the
         two small parts, again 2^-16; a chunk takes three such products and old errors
         decay with the state: 6 * 2^-16 = 9e-5, bar 1e-4.
"""
import numpy as np
import pytest
import torch

from oracle import delta
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

TOL = {"fp32": 1e-4, "bf16": 2e-2}
STATE = 1e-4
DV = {"fp32": 1e-4, "bf16": 2.0 ** -8}
EL = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rel(a, b):
    n = np.linalg.norm(b)
    return np.linalg.norm(a - b) / n if n > 0 else float(np.linalg.norm(a))


def draw(seed, b, T, H, P, N, G, dtype, lengths=None, init=True, gate=1.0, beta=None, decay=True):
    """Inputs on the CPU in the case's type; lengths: a packed stream's (zeros allowed)."""
    rng = np.random.default_rng(seed)
    nseq = None
    if lengths is not None:
        b, T, nseq = 1, sum(lengths), len(lengths)
    el = EL[dtype]
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)
    x = dict(q=t(unit(rng.standard_normal((b, T, G, N)))).to(el), k=t(unit(rng.standard_normal((b, T, G, N)))).to(el),
             v=t(rng.standard_normal((b, T, H, P))).to(el),
             g=t(-gate * rng.uniform(0, 0.3, (b, T, H)) * (1 if decay else 0)).to(el),
             beta=t(rng.uniform(0, 1, (b, T, H)) if beta is None else np.full((b, T, H), beta)).to(el))
    n = nseq or b
    x["initial_states"] = t(0.3 * rng.standard_normal((n, H, P, N))) if init else None
    x["seq_idx"] = None if lengths is None else torch.from_numpy(np.repeat(np.arange(nseq), lengths).astype(np.int32))
    x["nseq"] = nseq
    x["scale"] = N ** -0.5
    dy = t(rng.standard_normal((b, T, H, P))).to(el)
    dfin = t(0.3 * rng.standard_normal((n, H, P, N))) if init else None
    return x, dy, dfin


def gpu(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def spans(x):
    if x["seq_idx"] is None:
        return [(i, 0, x["v"].shape[1]) for i in range(x["v"].shape[0])]
    return [(0, lo, hi) for lo, hi in delta._segments(x["v"].shape[1], x["seq_idx"], x["nseq"]) if hi > lo]


def worst_tokens(got, ref, x, pooled=False):
    """max over (row or segment, head or group) of the relative error over its tokens.
    pooled: a slice of fewer than 64 tokens is held to the tensor's average size where
    that is larger than its own.  A gradient of one token is one dot product (of a fresh
    one-token sequence dq = scale beta (dy.u) k): its terms are off by 2^-8 of their
    sizes |dy_i u_i|, while the sum may cancel to nothing."""
    w, rms = 0.0, np.linalg.norm(ref) / np.sqrt(ref.size)
    for r, lo, hi in spans(x):
        for h in range(ref.shape[2]):
            a, b = got[r, lo:hi, h], ref[r, lo:hi, h]
            n = np.linalg.norm(b)
            if pooled and hi - lo < 64:
                n = max(n, rms * np.sqrt(b.size))
            w = max(w, np.linalg.norm(a - b) / max(n, 1e-30))
    return w


def worst_states(got, ref):
    return max(rel(got[i, h], ref[i, h]) for i in range(ref.shape[0]) for h in range(ref.shape[1]))


def check_fwd(x, dtype, label=""):
    g = gpu(x)
    y, fin = ssd.gdr_fwd(**g)
    torch.cuda.synchronize()
    yr, fr = delta.gdr_forward(**x)
    ey, ef = worst_tokens(f64(y), yr, x), worst_states(f64(fin), fr)
    print(f"[gdr fwd] {label} y={ey:.2e} states={ef:.2e}", flush=True)
    assert np.isfinite(f64(y)).all()
    assert ey <= TOL[dtype] and ef <= STATE, (ey, ef)


def check_bwd(x, dy, dfin, dtype, label=""):
    g = gpu(x)
    got = ssd.gdr_bwd(**g, dy=dy.cuda(), dfinal_states=None if dfin is None else dfin.cuda())
    torch.cuda.synchronize()
    ref = delta.gdr_backward(**x, dy=dy, dfinal_states=dfin)
    e = {}
    for n in ("dq", "dk", "dv", "dbeta", "dg"):
        r, a = ref[n], f64(got[n])
        assert np.isfinite(a).all(), n
        e[n] = worst_tokens(a, r, x, pooled=n != "dv")
    e["dinit"] = worst_states(f64(got["dinitial_states"]), ref["dinitial_states"])
    print(f"[gdr bwd] {label} " + " ".join(f"{k}={v:.2e}" for k, v in e.items()), flush=True)
    for n, v in e.items():
        assert v <= (STATE if n == "dinit" else DV[dtype] if n == "dv" else TOL[dtype]), (n, v)


# (b, T, H, P, N, G): every state width of the kernels (64, 128, 256) and ragged ones, one
# and several column tiles of a head (P = 16 .. 144), head sharing, lengths around the chunk
SHAPES = [(1, 1, 1, 16, 16, 1), (2, 63, 2, 32, 64, 1), (1, 64, 3, 48, 48, 3), (2, 65, 4, 64, 128, 2),
          (1, 130, 2, 80, 80, 1), (1, 257, 4, 64, 256, 4), (2, 200, 6, 144, 112, 2), (1, 320, 5, 128, 208, 1)]
IDS = lambda s: "b%d_T%d_H%d_P%d_N%d_G%d" % s


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(dtype, shape):
    b, T, H, P, N, G = shape
    check_fwd(draw(sum(shape), b, T, H, P, N, G, dtype)[0], dtype, str(shape))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(dtype, shape):
    b, T, H, P, N, G = shape
    x, dy, dfin = draw(sum(shape), b, T, H, P, N, G, dtype)
    check_bwd(x, dy, dfin, dtype, str(shape))


LENGTHS = {"mixed": [70, 1, 0, 64, 129, 2], "ones": [1] * 70, "one_empty": [0, 0, 5, 0], "long_first": [200, 3, 3]}


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("which", LENGTHS)
@pytest.mark.parametrize("init", [True, False], ids=["carried", "fresh"])
def test_packed(dtype, which, init):
    x, dy, dfin = draw(5, 1, 0, 4, 48, 64, 2, dtype, lengths=LENGTHS[which], init=init)
    check_fwd(x, dtype, which)
    check_bwd(x, dy, dfin, dtype, which)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("variant", ["fresh", "beta_zero", "beta_one", "beta_two", "no_decay", "strong_decay"])
def test_gates(dtype, variant):
    kw = dict(fresh=dict(init=False), beta_zero=dict(beta=0.0), beta_one=dict(beta=1.0), beta_two=dict(beta=2.0),
              no_decay=dict(decay=False), strong_decay=dict(gate=30.0))[variant]
    x, dy, dfin = draw(7, 2, 150, 2, 32, 64, 1, dtype, **kw)
    check_fwd(x, dtype, variant)
    check_bwd(x, dy, dfin, dtype, variant)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_same_key_in_every_token(dtype):
    """The triangular system at its stiffest: every pair of tokens shares its key, beta =
    1, no decay.  Then S returns the newest value, exactly: u_t = v_t - v_{t-1}."""
    x, _, _ = draw(8, 1, 130, 2, 32, 64, 1, dtype, init=False, beta=1.0, decay=False)
    key = torch.zeros_like(x["k"])
    key[..., 3] = 1
    x["k"], x["q"], x["scale"] = key, key.clone(), 1.0
    y, _ = ssd.gdr_fwd(**gpu(x))
    torch.cuda.synchronize()
    # y = v: the pair matrix and U are rounded once each before they are summed over up to
    # 64 tokens whose sum telescopes; |u| <= 2 |v|, in norm 64^(1/2) * 2 * 2 * 2^-9
    assert rel(f64(y), f64(x["v"])) <= (1e-4 if dtype == "fp32" else 2.0 ** -4)
    check_fwd_states_only(x)


def check_fwd_states_only(x):
    _, fin = ssd.gdr_fwd(**gpu(x))
    torch.cuda.synchronize()
    assert worst_states(f64(fin), delta.gdr_forward(**x)[1]) <= STATE


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_minus_infinite_gates_reset_the_state(dtype):
    x, _, _ = draw(9, 1, 100, 2, 32, 64, 1, dtype)
    cut = 37
    x["g"][:, cut] = -float("inf")
    y, fin = ssd.gdr_fwd(**gpu(x))
    tail = {n: (x[n][:, cut:].contiguous() if n in "qkv" or n in ("g", "beta") else x[n]) for n in x}
    tail["g"] = tail["g"].clone()
    tail["g"][:, 0] = 0
    tail["initial_states"] = None
    y2, fin2 = delta.gdr_forward(**tail)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()
    assert worst_tokens(f64(y[:, cut:]), y2, tail) <= TOL[dtype]
    assert worst_states(f64(fin), fin2) <= STATE


def test_nan_of_one_sequence_stays_there():
    x, dy, _ = draw(10, 1, 0, 2, 32, 64, 1, "bf16", lengths=[70, 30, 65])
    clean, cf = ssd.gdr_fwd(**gpu(x))
    cg = ssd.gdr_bwd(**gpu(x), dy=dy.cuda())
    for n in "qkv":
        x[n][0, 70:100] = float("nan")
    x["g"][0, 80] = float("nan")
    dy[0, 75] = float("inf")
    y, f = ssd.gdr_fwd(**gpu(x))
    gr = ssd.gdr_bwd(**gpu(x), dy=dy.cuda())
    torch.cuda.synchronize()
    for a, b in ((clean, y), *((cg[n], gr[n]) for n in ("dq", "dk", "dv", "dg", "dbeta"))):
        assert torch.equal(a[0, :70], b[0, :70]) and torch.equal(a[0, 100:], b[0, 100:])
    assert torch.equal(cf[[0, 2]], f[[0, 2]]) and torch.isnan(f[1]).any()
    assert torch.isnan(y[0, 70:100]).any()


# ---------------------------------------------------------------------------
# one token
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 16, 16, 1), (3, 4, 64, 128, 2), (2, 2, 48, 48, 1), (2, 8, 128, 256, 4),
                                   (5, 6, 80, 112, 3), (2, 3, 32, 32, 1)], ids=lambda s: "b%d_H%d_P%d_N%d_G%d" % s)
def test_step(dtype, shape):
    b, H, P, N, G = shape
    x, _, _ = draw(sum(shape), b, 1, H, P, N, G, dtype)
    tok = [x[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    state = x["initial_states"].cuda()
    y = ssd.gdr_step(*(t.cuda() for t in tok), state, scale=x["scale"])
    torch.cuda.synchronize()
    yr, sr = delta.gdr_step(*tok, x["initial_states"], x["scale"])
    # fp32 arithmetic throughout; y is rounded once
    assert rel(f64(y), yr) <= (1e-5 if dtype == "fp32" else 2.0 ** -8)
    assert worst_states(f64(state), sr) <= 1e-5


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prompt_then_steps_is_the_whole_prompt(dtype):
    """A prompt's first part through gdr_fwd, its rest token by token through gdr_step,
    and the same in two calls of gdr_fwd: the whole prompt's y and state."""
    x, _, _ = draw(11, 2, 150, 4, 64, 64, 2, dtype)
    g = gpu(x)
    y, fin = ssd.gdr_fwd(**g)
    part = lambda lo, hi, init: {n: (g[n][:, lo:hi].contiguous() if n in ("q", "k", "v", "g", "beta") else g[n])
                                 for n in g} | {"initial_states": init}
    y1, s1 = ssd.gdr_fwd(**part(0, 128, g["initial_states"]))
    y2, s2 = ssd.gdr_fwd(**part(128, 150, s1))
    assert torch.equal(y, torch.cat([y1, y2], 1)) and torch.equal(fin, s2)   # chunk boundaries agree
    state = s1.clone()
    steps = [ssd.gdr_step(*(g[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), state, scale=g["scale"])
             for t in range(128, 150)]
    torch.cuda.synchronize()
    assert rel(f64(torch.stack(steps, 1)), f64(y2)) <= TOL[dtype]
    assert worst_states(f64(state), f64(fin)) <= STATE


# ---------------------------------------------------------------------------
# gradients against differences, determinism, streams, graphs, sizes
# ---------------------------------------------------------------------------

def test_gradients_against_differences_of_the_kernel():
    """fp32: a directional difference of ssd_gdr_fwd's own loss against its gradients.
    The loss is a sum of about 1e4 terms in fp32 outputs (1e-4 of its size at worst),
    the step 1e-2 moves it by about that share: bar 2e-2 of the larger of both."""
    x, dy, dfin = draw(12, 1, 100, 2, 32, 32, 1, "fp32")
    gr = ssd.gdr_bwd(**gpu(x), dy=dy.cuda(), dfinal_states=dfin.cuda())
    rng = np.random.default_rng(13)

    def loss(x):
        y, f = ssd.gdr_fwd(**gpu(x))
        return float((y.double() * dy.cuda().double()).sum() + (f.double() * dfin.cuda().double()).sum())

    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("initial_states", "dinitial_states")):
        d = torch.from_numpy(rng.standard_normal(tuple(x[n].shape)).astype(np.float32))
        h = 2e-3
        num = (loss(dict(x, **{n: x[n] + h * d})) - loss(dict(x, **{n: x[n] - h * d}))) / (2 * h)
        ana = float((gr[gn].double().cpu() * d.double()).sum())
        scale = float(gr[gn].double().norm())
        assert abs(num - ana) <= 2e-2 * max(abs(ana), scale), (n, num, ana, scale)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_results_do_not_change_from_call_to_call(dtype):
    x, dy, dfin = draw(14, 1, 0, 8, 64, 128, 1, dtype, lengths=[100, 300, 1])
    g = gpu(x)
    runs = []
    for fill in (0, 255):
        ws = torch.full((ssd.gdr_fwd_workspace_bytes(*(g[n] for n in ("q", "k", "v", "g", "beta")), g["seq_idx"], 3),),
                        fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((ssd.gdr_bwd_workspace_bytes(*(g[n] for n in ("q", "k", "v", "g", "beta")), g["seq_idx"], 3),),
                        fill, dtype=torch.uint8, device="cuda")
        y, f = ssd.gdr_fwd(**g, workspace=ws)
        gr = ssd.gdr_bwd(**g, dy=dy.cuda(), dfinal_states=dfin.cuda(), workspace=wb)
        runs.append([y, f, *(gr[n] for n in sorted(gr))])
    torch.cuda.synchronize()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_another_stream():
    x, dy, _ = draw(15, 2, 200, 4, 64, 64, 2, "bf16")
    g = gpu(x)
    y, f = ssd.gdr_fwd(**g)
    gr = ssd.gdr_bwd(**g, dy=dy.cuda())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    d = dy.cuda()
    s.wait_stream(torch.cuda.current_stream())
    y2, f2 = ssd.gdr_fwd(**g, stream=s.cuda_stream)
    gr2 = ssd.gdr_bwd(**g, dy=d, stream=s.cuda_stream)
    junk = [torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]   # current stream
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(f, f2)
    assert all(torch.equal(gr[n], gr2[n]) for n in gr) and len(junk) == 8


def test_captured_and_replayed():
    x, dy, _ = draw(16, 1, 0, 4, 64, 64, 2, "bf16", lengths=[90, 40])
    g, d = gpu(x), dy.cuda()
    tok = [g[n][0, :2].contiguous() for n in ("q", "k", "v", "g", "beta")]
    st0 = g["initial_states"].clone()
    state = st0.clone()

    def all_three():
        y, f = ssd.gdr_fwd(**g)
        gr = ssd.gdr_bwd(**g, dy=d)
        return [y, f, *(gr[n] for n in sorted(gr)), ssd.gdr_step(*tok, state, scale=g["scale"])]

    want = [t.clone() for t in all_three()]
    s1 = state.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        all_three()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_three()
    for i in range(3):
        state.copy_(st0)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(state, s1), i
        ssd.gdr_fwd(**g)   # eager work between replays


def test_offsets_past_32_bits():
    """A stream whose v and y pass 2^32 bytes: its second half from the first half's
    state gives the same bits as the whole (the halves meet at a chunk boundary)."""
    T, H, P, N = 1 << 20, 34, 64, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(17)
    el = torch.bfloat16
    k = torch.nn.functional.normalize(torch.randn(1, T, 1, N, device="cuda", generator=gen), dim=-1).to(el)
    q = k.flip(1).contiguous()
    v = torch.empty(1, T, H, P, dtype=el, device="cuda")
    for i in range(0, T, 1 << 17):
        v[:, i:i + (1 << 17)] = torch.randn(1, 1 << 17, H, P, device="cuda", generator=gen).to(el)
    g = (-0.1 * torch.rand(1, T, H, device="cuda", generator=gen)).to(el)
    beta = torch.rand(1, T, H, device="cuda", generator=gen).to(el)
    assert v.numel() * 2 > 1 << 32
    y, f = ssd.gdr_fwd(q, k, v, g, beta)
    half = T // 2
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()
    _, s1 = ssd.gdr_fwd(*(cut(t, 0, half) for t in (q, k, v, g, beta)))
    y2, s2 = ssd.gdr_fwd(*(cut(t, half, T) for t in (q, k, v, g, beta)), initial_states=s1)
    torch.cuda.synchronize()
    assert torch.equal(s2, f) and torch.equal(y[:, half:], y2)


def test_no_tokens():
    x, dy, dfin = draw(18, 2, 4, 2, 32, 32, 1, "bf16")
    g = gpu(x)
    e = {n: (g[n][:, :0].contiguous() if n in ("q", "k", "v", "g", "beta") else g[n]) for n in g}
    y, f = ssd.gdr_fwd(**e)
    gr = ssd.gdr_bwd(**e, dy=y.clone(), dfinal_states=dfin.cuda())
    torch.cuda.synchronize()
    assert y.shape[1] == 0 and torch.equal(f, g["initial_states"])
    assert torch.equal(gr["dinitial_states"].cpu(), dfin)
