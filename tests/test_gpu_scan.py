"""GPU parity of the selective scan (ssd_selective_scan_fwd, _bwd, _step) against fp64.

Bars, counted before the first run.  Everything is computed in fp32 from exact inputs.  A decay over a stretch of
steps is the exponential of s = sum of Delta A: Delta is good to 1.8e-6 at worst (softplus from the hardware's
exponential and logarithm) and each exponential to 2^-22 of its own; stretches of s > 12 have decayed to 6e-6 of
themselves, so what counts is off by up to 12 * 1.8e-6 = 2.2e-5 if every error had one sign, and by a fraction of
that as they have not: the bar is 1e-5 in norm.  Sums over tokens or channels (dA, dB, dC, dD, ddt_bias) and ddt, whose two
terms may cancel, are held to 1e-5 of their terms' sizes.  Outputs in bf16 are rounded once: 2^-8 of themselves.
"""
import numpy as np
import pytest
import torch

from oracle import selective as sel
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

EL = {"fp32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"fp32": 0.0, "bf16": 2.0 ** -8}
BAR = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def near(got, ref, dtype=None, size=None):
    """Whether a tensor is its reference, rounded to its type, up to the bar."""
    got, ref = sel.f64(got), np.asarray(ref)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    half = ROUND[dtype] if dtype else 0.0
    assert np.isfinite(got).all()
    err = np.linalg.norm(got - ref)
    bar = half * np.linalg.norm(ref) + BAR * np.linalg.norm(ref if size is None else size) + 1e-30
    assert err <= bar, (err, bar, np.linalg.norm(ref))


def draw(seed, b, T, dim, N, G=1, dtype="fp32", lengths=None, init=True, gate=True, skip=True, bias=True, softplus=True, wide=False):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    el = EL[dtype]
    rows = b if lengths is None else len(lengths)
    p = {}
    # columns of one projection's rows, or tensors of their own
    xz = t(b, T, 2 * dim + 3).to(el)
    p["x"], p["z"] = xz[..., :dim], xz[..., dim + 3:]
    bc = t(b, T, 5 + 2 * G * N).to(el)
    p["B"], p["C"] = bc[..., 5:5 + G * N].unflatten(-1, (G, N)), bc[..., 5 + G * N:].unflatten(-1, (G, N))
    p["dt"] = (0.5 * t(b, T, dim) - (0 if bias else 3)).to(el)
    if not softplus:
        p["dt"] = torch.nn.functional.softplus(p["dt"].float() - 3).to(el)
    p["dt_bias"] = (t(dim) - 3 if softplus else 0.01 * t(dim).abs()) if bias else None
    p["A"] = -torch.exp(0.5 * t(dim, N)) * (1 + torch.arange(N))
    p["D"] = t(dim) if skip else None
    if not gate:
        p["z"] = None
    if not wide:
        for n in ("x", "z", "B", "C"):
            p[n] = None if p[n] is None else p[n].contiguous()
    s0 = 0.5 * t(rows, dim, N) if init else None
    return p, s0, t(b, T, dim).to(el), 0.5 * t(rows, dim, N) if init else None


def on_gpu(p):
    return {k: None if v is None else (v.cuda() if v.is_contiguous() else columns(v)) for k, v in p.items()}


def columns(v):
    """The same columns of wider rows on the GPU."""
    lead = v.shape[:2]
    step = v.stride(1) if lead[1] > 1 else v.stride(0)
    wide = torch.zeros(*lead, step, dtype=v.dtype, device="cuda")
    flat = v.reshape(*lead, -1)
    wide[..., 1:1 + flat.shape[-1]] = flat.cuda()
    return wide[..., 1:1 + flat.shape[-1]].view(v.shape) if v.dim() == 3 else wide[..., 1:1 + flat.shape[-1]].unflatten(-1, v.shape[2:])


def ids_of(lengths):
    if lengths is None:
        return {}
    i = torch.repeat_interleave(torch.arange(len(lengths), dtype=torch.int32), torch.tensor(lengths))
    return {"seq_idx": i.cuda(), "nseq": len(lengths)}


def check(case, dtype, lengths=None, softplus=True, bwd=True):
    p, s0, dy, df = case
    g = on_gpu(p)
    c = lambda t: None if t is None else t.cuda()
    kw = dict(D=g["D"], z=g["z"], dt_bias=g["dt_bias"], dt_softplus=softplus, initial_states=c(s0), **ids_of(lengths))
    ins = (g["x"], g["dt"], g["A"], g["B"], g["C"])
    y, fin = ssd.selective_scan_fwd(*ins, **kw)
    gr = ssd.selective_scan_bwd(*ins, dy.cuda(), dfinal_states=c(df), **kw) if bwd else None
    torch.cuda.synchronize()
    ref = dict(p, softplus=softplus, init=s0, lengths=lengths)
    yr, fr = sel.scan_forward(**ref)
    near(y, yr, dtype)
    near(fin, fr)
    if not bwd:
        return
    r = sel.scan_backward(**ref, dy=dy, dfinal=df)
    sz = r["sizes"]
    near(gr["dx"], r["dx"], dtype)
    near(gr["ddt"], r["ddt"], dtype, sz["ddt"])
    near(gr["dB"], r["dB"], dtype, sz["dB"])
    near(gr["dC"], r["dC"], dtype, sz["dC"])
    near(gr["dA"], r["dA"], size=sz["dA"])
    near(gr["dinitial_states"], r["dinitial_states"])
    if p["D"] is not None:
        near(gr["dD"], r["dD"], size=sz["dD"])
    else:
        assert gr["dD"] is None
    if p["dt_bias"] is not None:
        near(gr["ddt_bias"], r["ddt_bias"], size=sz["ddt_bias"])
    if p["z"] is not None:
        near(gr["dz"], r["dz"], dtype)
    else:
        assert gr["dz"] is None


# every number of lanes a channel is held by (1, 2, 4, 8, 16), full and not
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 13, 16, 17, 32, 40, 64])
def test_state_widths(dtype, N):
    check(draw(N, 2, 75, 37, N, dtype=dtype), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200])
def test_lengths(dtype, T):
    check(draw(T, 3, T, 70, 16, dtype=dtype), dtype)


@pytest.mark.parametrize("dim,G", [(1, 1), (3, 3), (63, 1), (64, 1), (65, 1), (130, 2), (256, 4), (195, 3), (257, 1)])
def test_channels_and_groups(dim, G):
    check(draw(dim, 2, 70, dim, 16, G), "fp32")
    check(draw(dim, 1, 40, dim, 6, G, "bf16"), "bf16")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_long_rows_are_cut(dtype):
    """Few channels and many tokens: the forward in chunks too."""
    check(draw(1, 1, 1111, 40, 16, dtype=dtype), dtype)
    check(draw(2, 2, 520, 20, 32, dtype=dtype), dtype)


PACKED = [[1], [5, 1, 64, 65, 3], [0, 3, 0, 0, 70, 1, 0], [128, 1, 1, 1, 128], [63, 130, 2], [1] * 40, [300, 2, 0, 17]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", PACKED)
def test_packed(dtype, lengths):
    check(draw(len(lengths), 1, sum(lengths), 70, 16, 2, dtype, lengths), dtype, lengths)
    check(draw(len(lengths), 1, sum(lengths), 33, 5, 1, dtype, lengths, init=False), dtype, lengths)


def test_packed_long_rows_are_cut():
    lengths = [700, 3, 0, 600]
    check(draw(5, 1, sum(lengths), 24, 16, 1, "fp32", lengths), "fp32", lengths)


@pytest.mark.parametrize("which", ["gate", "skip", "bias", "init", "softplus"])
def test_without(which):
    check(draw(7, 2, 90, 50, 16, **{which: False}), "fp32", softplus=which != "softplus")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_columns_of_wider_rows(dtype):
    check(draw(8, 2, 77, 45, 10, 3, dtype, wide=True), dtype)
    p, s0, dy, df = draw(8, 2, 77, 45, 10, 3, dtype, wide=True)
    g = on_gpu(p)
    assert not g["x"].is_contiguous() and not g["B"].is_contiguous()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,dim,G", [(16, 70, 2), (1, 5, 1), (64, 33, 3), (7, 300, 1)])
def test_steps_are_the_scan(dtype, N, dim, G):
    b, T = 3, 9
    p, s0, _, _ = draw(9, b, T, dim, N, G, dtype)
    g = on_gpu(p)
    state = s0.cuda()
    ys = []
    for t in range(T):
        at = lambda n: g[n][:, t]
        ys.append(ssd.selective_scan_step(at("x"), at("dt"), g["A"], at("B"), at("C"), state, D=g["D"], z=at("z"), dt_bias=g["dt_bias"]))
    torch.cuda.synchronize()
    yr, fr = sel.scan_forward(**p, init=s0)
    near(torch.stack(ys, 1), yr, dtype)
    near(state, fr)


def test_extreme_steps():
    """Steps that decay everything (Delta A of -1e4), and none at all (softplus of -1e4 is 0)."""
    p, s0, dy, df = draw(10, 1, 40, 20, 16)
    p["dt"][:, 5:9] = 1e4
    p["dt"][:, 20:24] = -1e4
    p["A"] = p["A"].clamp(max=-0.5)
    # x B of a step of 1e4 is 1e4 times the others', so those are measured against it, as in the reference
    check((p, s0, dy, df), "fp32")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_not_finite_stays_in_its_channel_and_behind(dtype):
    p, s0, dy, _ = draw(11, 2, 100, 70, 16, dtype=dtype)
    g = on_gpu(p)
    run = lambda x: ssd.selective_scan_fwd(x, g["dt"], g["A"], g["B"], g["C"], D=g["D"], z=g["z"], dt_bias=g["dt_bias"])
    y, f = run(g["x"])
    bad = g["x"].clone()
    bad[1, 50, 3] = float("nan")
    yb, fb = run(bad)
    keep = torch.ones(2, 100, 70, dtype=torch.bool, device="cuda")
    keep[1, 50:, 3] = False
    assert torch.equal(y[keep], yb[keep]) and torch.isnan(yb[1, 50:, 3]).all()
    k2 = torch.ones(2, 70, dtype=torch.bool, device="cuda")
    k2[1, 3] = False
    assert torch.equal(f[k2], fb[k2]) and torch.isnan(fb[1, 3]).all()


def test_packed_segments_do_not_meet():
    """A segment that is all NaN leaves the others' outputs and gradients as they are, bit for bit, and nothing but
    the sums over tokens changes."""
    lengths = [50, 70, 20]
    p, s0, dy, df = draw(12, 1, 140, 40, 16, lengths=lengths)
    g, ids = on_gpu(p), ids_of(lengths)
    def run(x):
        kw = dict(D=g["D"], z=g["z"], dt_bias=g["dt_bias"], initial_states=s0.cuda(), **ids)
        y, f = ssd.selective_scan_fwd(x, g["dt"], g["A"], g["B"], g["C"], **kw)
        return y, f, ssd.selective_scan_bwd(x, g["dt"], g["A"], g["B"], g["C"], dy.cuda(), dfinal_states=df.cuda(), **kw)
    y, f, gr = run(g["x"])
    bad = g["x"].clone()
    bad[:, 50:120] = float("nan")
    yb, fb, gb = run(bad)
    out = [slice(0, 50), slice(120, 140)]
    for at in out:
        assert torch.equal(y[:, at], yb[:, at])
        assert all(torch.equal(gr[n][:, at], gb[n][:, at]) for n in ("dx", "ddt", "dz", "dB", "dC"))
    assert torch.equal(f[[0, 2]], fb[[0, 2]]) and torch.equal(gr["dinitial_states"][[0, 2]], gb["dinitial_states"][[0, 2]])


def test_no_tokens():
    p, s0, dy, df = draw(13, 2, 0, 10, 4)
    check((p, s0, dy, df), "fp32")
    lengths = [0, 0, 0]
    p, s0, dy, df = draw(13, 1, 0, 10, 4, lengths=lengths)
    check((p, s0, dy, df), "fp32", lengths)


def test_ids_out_of_range_and_order_touch_nothing_else():
    """Streams that break the precondition: whatever comes out, nothing outside the outputs is written."""
    T, dim, N, nseq = 150, 20, 16, 4
    p, s0, dy, df = draw(14, 1, T, dim, N, lengths=[T // 2, T // 2, 0, 0])
    g = on_gpu(p)
    for ids in (torch.full((T,), 9), torch.full((T,), -3), torch.arange(T).flip(0), torch.randint(-5, 9, (T,), generator=torch.Generator().manual_seed(0))):
        pad = 4096
        def guarded(*shape):
            n = int(np.prod(shape))
            buf = torch.full((n + 2 * pad,), 7.0, device="cuda")
            return buf, buf[pad:pad + n].view(shape)
        yb, y = guarded(1, T, dim)
        fb, f = guarded(nseq, dim, N)
        kw = dict(D=g["D"], z=g["z"], dt_bias=g["dt_bias"], initial_states=s0.cuda(), seq_idx=ids.int().cuda(), nseq=nseq)
        ssd.selective_scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], y=y, final_states=f, **kw)
        bufs, grads = [], {}
        for n, shape in dict(dx=(1, T, dim), ddt=(1, T, dim), dz=(1, T, dim), dA=(dim, N), dB=(1, T, 1, N), dC=(1, T, 1, N), dD=(dim,),
                             ddt_bias=(dim,), dinitial_states=(nseq, dim, N)).items():
            b, grads[n] = guarded(*shape)
            bufs.append(b)
        ssd.selective_scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], dy.cuda(), dfinal_states=df.cuda(), grads=grads, **kw)
        torch.cuda.synchronize()
        for b in [yb, fb, *bufs]:
            assert (b[:pad] == 7).all() and (b[-pad:] == 7).all()


def test_captured_other_streams_and_repeatable():
    p, s0, dy, df = draw(15, 1, 700, 40, 16, dtype="bf16")
    g, s0, dy, df = on_gpu(p), s0.cuda(), dy.cuda(), df.cuda()
    def both(stream=None):
        kw = dict(D=g["D"], z=g["z"], dt_bias=g["dt_bias"], initial_states=s0, stream=stream)
        y, f = ssd.selective_scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw)
        gr = ssd.selective_scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], dy, dfinal_states=df, **kw)
        return [y, f] + [gr[k] for k in sorted(gr)]
    want = [t.clone() for t in both()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        both()


def test_given_buffers():
    p, s0, dy, df = draw(16, 1, 1000, 24, 16)
    g = on_gpu(p)
    ins = (g["x"], g["dt"], g["A"], g["B"], g["C"])
    n = ssd.selective_scan_fwd_workspace_bytes(*ins)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    y0 = torch.empty_like(g["x"])
    y, f = ssd.selective_scan_fwd(*ins, y=y0, workspace=ws, want_final=False)
    assert y is y0 and f is None
    y2, _ = ssd.selective_scan_fwd(*ins)
    ws = torch.empty(ssd.selective_scan_bwd_workspace_bytes(*ins), dtype=torch.uint8, device="cuda")
    gr = ssd.selective_scan_bwd(*ins, dy.cuda(), workspace=ws, want_dinit=False)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and gr["dinitial_states"] is None and gr["dD"] is None
    with pytest.raises(ssd.SSDError):
        ssd.selective_scan_fwd(*ins, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_past_2_to_the_32_bytes():
    """x of 4.7 GB: the last tokens of a long row against the same tokens as a row of their own."""
    T, dim, N = 70000, 16800, 4
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(1, T, dim, device="cuda", generator=gen)
    dt = x.flip(1).contiguous().mul_(0.1)
    B, C = (torch.randn(1, T, 1, N, device="cuda", generator=gen) for _ in range(2))
    A = -torch.rand(dim, N, device="cuda", generator=gen) - 0.5
    y, f = ssd.selective_scan_fwd(x, dt, A, B, C)
    cut = T - 300
    _, mid = ssd.selective_scan_fwd(*(t[:, :cut].contiguous() if t.dim() > 2 else t for t in (x, dt, A, B, C)))
    y2, f2 = ssd.selective_scan_fwd(*(t[:, cut:].contiguous() if t.dim() > 2 else t for t in (x, dt, A, B, C)), initial_states=mid)
    torch.cuda.synchronize()
    err = (y[:, cut:] - y2).double().norm() / y2.double().norm()
    assert err <= 2 * BAR and (f - f2).double().norm() <= 2 * BAR * f2.double().norm()
