"""GPU parity of layer norm (ssd_layer_norm_fwd, ssd_layer_norm_bwd) against fp64.

Bars, counted before the first run: everything is computed in fp32 from exact inputs, a
row's sums have at most 65536 terms in partial sums of at most a few hundred, so y, mean
and rstd are good to about 1e-6 (bar 1e-5; the mean against the row's spread, since a
mean may vanish), dweight and dbias likewise against the sum of their terms' sizes.
bf16 outputs are rounded once: 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import delta
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

EL = {"fp32": torch.float32, "bf16": torch.bfloat16}
OUT = {"fp32": 1e-5, "bf16": 2.0 ** -8}


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


def draw(seed, rows, dim, dtype, offset=1.0):
    rng = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    x = t(rng.standard_normal((rows, dim)) * (0.5 + rng.uniform(0, 2, (rows, 1))) + offset * rng.standard_normal((rows, 1)))
    return x.to(EL[dtype]), t(rng.standard_normal((rows, dim))).to(EL[dtype]), t(1 + 0.1 * rng.standard_normal(dim)), t(rng.standard_normal(dim))


def check(x, dy, w, b, dtype, eps=1e-5):
    c = lambda t: None if t is None else t.cuda()
    y, mean, rstd = ssd.layer_norm_fwd(c(x), c(w), c(b), eps=eps)
    gr = ssd.layer_norm_bwd(c(x), c(dy), mean, rstd, c(w), want_params=True)
    torch.cuda.synchronize()
    yr, mr, rr = delta.layer_norm(x, w, b, eps)
    assert rel(f64(y), yr) <= OUT[dtype]
    spread = np.sqrt((f64(x) ** 2).mean(-1))
    assert (np.abs(f64(mean) - mr) <= 1e-5 * spread).all()
    assert rel(f64(rstd), rr) <= 1e-5
    dx, dw, db = delta.layer_norm_backward(x, dy, mean, rstd, w)
    # dx subtracts two averages from dy: of one or two values nothing is left, so the bar
    # stands against what is subtracted from
    ww = f64(dy) * (1 if w is None else f64(w))
    size = np.linalg.norm(ww * f64(rstd)[..., None])
    assert np.linalg.norm(f64(gr["dx"]) - dx) <= OUT[dtype] * np.linalg.norm(dx) + 1e-5 * size
    xhat = (f64(x) - f64(mean)[..., None]) * f64(rstd)[..., None]
    assert np.linalg.norm(f64(gr["dweight"]) - dw) <= 1e-5 * np.linalg.norm(np.abs(f64(dy) * xhat).sum(0))
    assert np.linalg.norm(f64(gr["dbias"]) - db) <= 1e-5 * np.linalg.norm(np.abs(f64(dy)).sum(0))


# every way a row is held: 16, 64 and 256 lanes with 16-byte vectors and with single
# elements, each number of vectors per lane, and rows longer than the registers
DIMS = [1, 2, 7, 16, 31, 33, 64, 100, 128, 255, 256, 300, 320, 512, 520, 1000, 1024, 1531, 2047, 2049, 2560, 4096, 5120,
        8192, 8200, 16384, 16392, 20001]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dim", DIMS)
def test_widths(dtype, dim):
    check(*draw(dim, 37, dim, dtype), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 64), (1, 2560), (3, 4096), (511, 128), (513, 96), (2050, 40), (5000, 16),
                                      (1500, 2560), (700, 21), (1030, 8200)])
def test_rows(dtype, rows, dim):
    check(*draw(rows + dim, rows, dim, dtype), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("which", ["none", "weight", "bias"])
def test_without_parameters(dtype, which):
    x, dy, w, b = draw(3, 40, 320, dtype)
    check(x, dy, w if which == "weight" else None, b if which == "bias" else None, dtype)


def test_far_off_centre_and_constant_rows():
    """The squares are taken around the mean: a row at 1000 with spread 1 keeps its
    variance (one pass over x^2 would lose 6 digits), a constant row gives the bias."""
    x, dy, w, b = draw(4, 20, 1000, "fp32", offset=1000.0)
    y, _, _ = ssd.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    torch.cuda.synchronize()
    # x itself is held to 2^-24 * 3000 = 2e-4 of the spread, exactly; the mean to a few of
    # those steps, which moves y by as much
    assert rel(f64(y), delta.layer_norm(x, w, b)[0]) <= 2e-3
    c = torch.full((3, 300), 2.5, device="cuda")
    y, mean, rstd = ssd.layer_norm_fwd(c, None, b[:300].cuda(), eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), b[:300].expand(3, 300)) and (mean == 2.5).all()
    assert rel(f64(rstd), np.full(3, 1e-5 ** -0.5)) <= 1e-5


@pytest.mark.parametrize("dim", [2560, 1531, 20001])
def test_nan_stays_in_its_row_and_in_place(dim):
    x, dy, w, b = (t.cuda() for t in draw(5, 30, dim, "bf16"))
    y, mean, rstd = ssd.layer_norm_fwd(x, w, b)
    gr = ssd.layer_norm_bwd(x, dy, mean, rstd, w)
    bad = x.clone()
    bad[7, dim // 2] = float("nan")
    yb, mb, rb = ssd.layer_norm_fwd(bad, w, b)
    keep = torch.arange(30, device="cuda") != 7
    assert torch.equal(y[keep], yb[keep]) and torch.isnan(yb[7]).all()
    # y over x, dx over dy
    x2, dy2 = x.clone(), dy.clone()
    y2, _, _ = ssd.layer_norm_fwd(x2, w, b, y=x2)
    g2 = ssd.layer_norm_bwd(x, dy2, mean, rstd, w, grads={"dx": dy2})
    torch.cuda.synchronize()
    assert y2.data_ptr() == x2.data_ptr() and torch.equal(x2, y)
    assert g2["dx"].data_ptr() == dy2.data_ptr()
    assert all(torch.equal(gr[n], g2[n]) for n in ("dx", "dweight", "dbias"))


def test_leading_axes_stats_and_no_rows():
    x, dy, w, b = (t.cuda() for t in draw(6, 24, 96, "fp32"))
    y, mean, rstd = ssd.layer_norm_fwd(x, w, b)
    y3, m3, r3 = ssd.layer_norm_fwd(x.view(2, 3, 4, 96), w, b)
    assert y3.shape == (2, 3, 4, 96) and m3.shape == (2, 3, 4)
    assert torch.equal(y3.view(24, 96), y) and torch.equal(m3.view(24), mean) and torch.equal(r3.view(24), rstd)
    y4, m4, r4 = ssd.layer_norm_fwd(x, w, b, want_stats=False)
    assert torch.equal(y4, y) and m4 is None and r4 is None
    e = x[:0]
    ye, me, re_ = ssd.layer_norm_fwd(e, w, b)
    g = ssd.layer_norm_bwd(e, dy[:0], me, re_, w, grads={"dweight": torch.ones(96, device="cuda")})
    torch.cuda.synchronize()
    assert ye.shape == (0, 96) and not g["dweight"].any() and not g["dbias"].any()


def test_captured_and_on_another_stream():
    x, dy, w, b = (t.cuda() for t in draw(7, 600, 320, "bf16"))

    def both(stream=None):
        y, m, r = ssd.layer_norm_fwd(x, w, b, stream=stream)
        g = ssd.layer_norm_bwd(x, dy, m, r, w, stream=stream)
        return [y, m, r, g["dx"], g["dweight"], g["dbias"]]

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


def test_the_block_norm_conv_and_rule_together():
    """One block's front end as a model runs it, forward and one token of decode: layer
    norm, a projection, the convolution, the gated delta rule."""
    H, P, N, G, T, D = 4, 64, 64, 2, 150, 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)
    el = torch.bfloat16
    x = rnd(1, T, D).to(el)
    w, b = 1 + 0.1 * rnd(D), 0.1 * rnd(D)
    proj = (rnd(D, H * P + 2 * G * N) / D ** 0.5).to(el)
    taps, bias = 0.4 * rnd(H * P + 2 * G * N, 4), 0.1 * rnd(H * P + 2 * G * N)
    g, beta = (-0.2 * torch.rand(1, T, H, device="cuda", generator=gen)).to(el), torch.rand(1, T, H, device="cuda", generator=gen).to(el)
    n, _, _ = ssd.layer_norm_fwd(x, w, b)
    v, k, q = ssd.conv1d_silu((n.view(T, D) @ proj).view(1, T, -1), taps, H, P, G, N, bias=bias)
    unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(el)
    q, k = unit(q), unit(k)
    y, fin = ssd.gdr_fwd(q, k, v, g, beta, scale=N ** -0.5)
    state = torch.zeros_like(fin)
    ys = [ssd.gdr_step(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(), g[:, t].contiguous(),
                       beta[:, t].contiguous(), state, scale=N ** -0.5) for t in range(T)]
    torch.cuda.synchronize()
    yr, fr = delta.gdr_forward(q, k, v, g, beta, N ** -0.5)
    assert rel(f64(n), delta.layer_norm(x, w, b)[0]) <= 2.0 ** -8
    assert rel(f64(y), yr) <= 2e-2 and rel(f64(torch.stack(ys, 1)), yr) <= 2.0 ** -8
    assert rel(f64(fin), fr) <= 1e-4 and rel(f64(state), fr) <= 1e-4
