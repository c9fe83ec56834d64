"""GPU parity of the causal convolution with a carried window (ssd_causal_conv_fwd, _bwd, _step) against fp64.

Bars, counted before the first run: K products and sums in fp32, SiLU from the hardware's exponential and
reciprocal (1 ulp each): about 1e-6 (bar 1e-5); sums over tokens against their terms' sizes, 1e-5; bf16 outputs
are rounded once, 2^-8.  Windows hold inputs and come out exactly.
"""
import numpy as np
import pytest
import torch

from oracle import selective as sel
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

EL = {"fp32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"fp32": 0.0, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def near(got, ref, dtype=None, size=None):
    got = sel.f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    bar = (ROUND[dtype] if dtype else 0.0) * np.linalg.norm(ref) + 1e-5 * np.linalg.norm(ref if size is None else size) + 1e-30
    assert np.linalg.norm(got - ref) <= bar, (np.linalg.norm(got - ref), bar)


def draw(seed, b, T, dim, K, dtype, lengths=None, init=True):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    rows = b if lengths is None else len(lengths)
    el = EL[dtype]
    return (t(b, T, dim).to(el), t(dim, K), t(dim), t(rows, K - 1, dim).to(el) if init else None, t(b, T, dim).to(el),
            t(rows, K - 1, dim).to(el) if init else None)


def ids_of(lengths):
    if lengths is None:
        return {}
    i = torch.repeat_interleave(torch.arange(len(lengths), dtype=torch.int32), torch.tensor(lengths))
    return {"seq_idx": i.cuda(), "nseq": len(lengths)}


def check(case, dtype, lengths=None, silu=True, bias=True, x_on_gpu=None):
    x, w, b, win, dy, dwin = case
    b = b if bias else None
    c = lambda t: None if t is None else t.cuda()
    xg = c(x) if x_on_gpu is None else x_on_gpu
    kw = dict(bias=c(b), silu=silu, initial_window=c(win), **ids_of(lengths))
    y, fin = ssd.causal_conv_fwd(xg, c(w), **kw)
    g = ssd.causal_conv_bwd(xg, c(w), c(dy), dfinal_window=c(dwin), **kw)
    torch.cuda.synchronize()
    yr, fr = sel.conv_forward(x, w, b, silu, win, lengths)
    near(y, yr, dtype)
    assert np.array_equal(sel.f64(fin), fr)
    r = sel.conv_backward(x, w, dy, b, silu, win, dwin, lengths)
    near(g["dx"], r["dx"], dtype)
    near(g["dweight"], r["dweight"], size=r["sizes"]["dweight"])
    near(g["dinitial_window"], r["dinitial_window"], dtype)
    if bias:
        near(g["dbias"], r["dbias"], size=r["sizes"]["dbias"])
    else:
        assert g["dbias"] is None


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dim", [1, 7, 64, 100, 264, 771])
def test_widths(dtype, K, dim):
    check(draw(dim + K, 2, 37, dim, K, dtype), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 15, 16, 17, 18, 31, 33, 64, 65, 67, 130, 500])
def test_lengths(dtype, T):
    check(draw(T, 3, T, 40, 4, dtype), dtype)


def test_long_strips():
    """Threads enough for strips of 64 tokens in the backward."""
    check(draw(1, 4, 1030, 512, 4, "bf16"), "bf16")


PACKED = [[1], [1, 1, 1, 2, 3, 4], [0, 5, 0, 0, 40, 1, 0], [16, 16, 1, 15, 17], [3, 130, 2], [1] * 40, [14, 2, 2, 2, 60]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("lengths", PACKED)
def test_packed(dtype, K, lengths):
    check(draw(len(lengths), 1, sum(lengths), 24, K, dtype, lengths), dtype, lengths)
    check(draw(len(lengths), 1, sum(lengths), 5, K, dtype, lengths, init=False), dtype, lengths, silu=False)


@pytest.mark.parametrize("silu,bias,init", [(False, True, True), (True, False, True), (True, True, False), (False, False, False)])
def test_without(silu, bias, init):
    check(draw(3, 2, 50, 33, 4, "fp32", init=init), "fp32", silu=silu, bias=bias)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dim,wide,first", [(64, 128, 0), (64, 131, 0), (64, 128, 3), (40, 96, 8)])
def test_columns_of_wider_rows(dtype, dim, wide, first):
    case = draw(4, 2, 45, dim, 4, dtype)
    rows = torch.full((2, 45, wide), float("nan"), dtype=EL[dtype], device="cuda")
    rows[..., first:first + dim] = case[0].cuda()
    check(case, dtype, x_on_gpu=rows[..., first:first + dim])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,dim", [(1, 16), (2, 33), (3, 64), (4, 520), (4, 5)])
def test_steps_are_the_convolution(dtype, K, dim):
    x, w, b, win, _, _ = draw(5, 3, 7, dim, K, dtype)
    window, ys = win.cuda(), []
    xg = x.cuda()
    for t in range(7):
        ys.append(ssd.causal_conv_step(xg[:, t], window, w.cuda(), bias=b.cuda()))
    torch.cuda.synchronize()
    yr, fr = sel.conv_forward(x, w, b, True, win)
    near(torch.stack(ys, 1), yr, dtype)
    assert np.array_equal(sel.f64(window), fr)


def test_large_values_and_not_finite():
    """SiLU and its slope where the exponential overflows; a NaN reaches the K tokens that see it, in its channel."""
    x, w, b, _, dy, _ = draw(6, 1, 30, 8, 4, "fp32", init=False)
    check((x * 1e4, w, b, None, dy, None), "fp32")
    xg = x.cuda()
    y, _ = ssd.causal_conv_fwd(xg, w.cuda(), bias=b.cuda())
    bad = xg.clone()
    bad[0, 10, 2] = float("nan")
    yb, _ = ssd.causal_conv_fwd(bad, w.cuda(), bias=b.cuda())
    torch.cuda.synchronize()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[0, 10:14, 2] = False
    assert torch.equal(y[keep], yb[keep]) and torch.isnan(yb[~keep]).all()


def test_segments_do_not_meet():
    lengths = [9, 20, 11]
    x, w, b, win, dy, dwin = (t.cuda() for t in draw(7, 1, 40, 16, 4, "bf16", lengths))
    ids = ids_of(lengths)
    def run(x):
        y, f = ssd.causal_conv_fwd(x, w, bias=b, initial_window=win, **ids)
        return y, f, ssd.causal_conv_bwd(x, w, dy, bias=b, initial_window=win, dfinal_window=dwin, **ids)
    y, f, g = run(x)
    bad = x.clone()
    bad[:, 9:29] = float("inf")
    yb, fb, gb = run(bad)
    torch.cuda.synchronize()
    for at in (slice(0, 9), slice(29, 40)):
        assert torch.equal(y[:, at], yb[:, at]) and torch.equal(g["dx"][:, at], gb["dx"][:, at])
    assert torch.equal(f[[0, 2]], fb[[0, 2]]) and torch.equal(g["dinitial_window"][[0, 2]], gb["dinitial_window"][[0, 2]])


def test_no_tokens():
    check(draw(8, 2, 0, 10, 4, "bf16"), "bf16")
    check(draw(8, 1, 0, 10, 3, "fp32", [0, 0]), "fp32", [0, 0])


def test_ids_out_of_range_and_order_touch_nothing_else():
    T, dim, nseq, pad = 90, 16, 3, 4096
    x, w, b, win, dy, dwin = (t.cuda() for t in draw(9, 1, T, dim, 4, "fp32", [30, 30, 30]))
    for ids in (torch.full((T,), 9), torch.full((T,), -3), torch.arange(T).flip(0), torch.randint(-5, 9, (T,), generator=torch.Generator().manual_seed(0))):
        bufs = []
        def guarded(shape):
            n = int(np.prod(shape))
            buf = torch.full((n + 2 * pad,), 7.0, device="cuda")
            bufs.append(buf)
            return buf[pad:pad + n].view(shape)
        kw = dict(bias=b, initial_window=win, seq_idx=ids.int().cuda(), nseq=nseq)
        ssd.causal_conv_fwd(x, w, y=guarded(x.shape), final_window=guarded(win.shape), **kw)
        ssd.causal_conv_bwd(x, w, dy, dfinal_window=dwin, grads={"dx": guarded(x.shape), "dweight": guarded(w.shape), "dbias": guarded(b.shape),
                                                                "dinitial_window": guarded(win.shape)}, **kw)
        torch.cuda.synchronize()
        assert all((t[:pad] == 7).all() and (t[-pad:] == 7).all() for t in bufs)


def test_captured_and_on_another_stream():
    x, w, b, win, dy, dwin = (t.cuda() for t in draw(10, 2, 200, 96, 4, "bf16"))
    def both(stream=None):
        y, f = ssd.causal_conv_fwd(x, w, bias=b, initial_window=win, stream=stream)
        g = ssd.causal_conv_bwd(x, w, dy, bias=b, initial_window=win, dfinal_window=dwin, stream=stream)
        return [y, f] + [g[k] for k in sorted(g)]
    want = [t.clone() for t in both()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), i
        both()
