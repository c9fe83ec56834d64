"""GPU parity of RMS norm with the residual's addition (ssd_rms_norm_fwd, ssd_rms_norm_bwd) against fp64.

Bars, counted before the first run: sums of at most 65536 squares in fp32 in parts of a few hundred, then a handful of
roundings: about 1e-6 (bar 1e-5; dweight against its terms' sizes).  bf16 outputs are rounded once, 2^-8.  The
stream's values are the sum rounded to its type, exactly.  In 8 bits every value is within half a step of its
neighbourhood, 2^-4 of itself, or 2^-10 below the smallest normal number of 2^-6 (steps of 2^-9), up to the same 1e-5 of
the largest, 448.
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


def draw(seed, rows, dim, dtype, res):
    rng = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    n = lambda: rng.standard_normal((rows, dim)) * (0.3 + rng.uniform(0, 2, (rows, 1)))
    x, dy = t(n()).to(EL[dtype]), t(rng.standard_normal((rows, dim))).to(EL[dtype])
    r = None if res is None else t(3 * n()).to(EL[res])
    dr = None if res is None else t(rng.standard_normal((rows, dim))).to(EL[res])
    return x, r, t(1 + 0.2 * rng.standard_normal(dim)), dy, dr


def check(case, dtype, res, weight=True, eps=1e-5):
    x, r, w, dy, dr = case
    w = w if weight else None
    c = lambda t: None if t is None else t.cuda()
    y, ro, rstd = ssd.rms_norm_fwd(c(x), c(w), residual=c(r), eps=eps)
    q, scales, ro2 = ssd.rms_norm_quant(c(x), c(w), residual=c(r), eps=eps)
    torch.cuda.synchronize()
    stream = x if r is None else (x.float() + r.float()).to(r.dtype)
    if r is None:
        assert ro is None and ro2 is None
    else:
        assert torch.equal(ro.cpu(), stream) and torch.equal(ro2.cpu(), stream)
    yr, rr = sel.rms_norm(stream, w, eps)
    near(y, yr, dtype)
    near(rstd, rr)
    sr, qr = sel.to_8bit(yr)
    near(scales, sr)
    q = sel.f64(q)
    assert (np.abs(q - qr) <= np.maximum(2.0 ** -4 * np.abs(qr), 2.0 ** -10) + 448e-5).all()
    stream = stream.cuda()
    g = ssd.rms_norm_bwd(stream, c(dy), rstd, c(w), dresidual=c(dr), want_dweight=True)
    torch.cuda.synchronize()
    gr, dw, size = sel.rms_norm_backward(stream, dy, rstd, w, dr)
    # two terms that may cancel: the bar stands against the first
    ww = sel.f64(dy) * (1 if w is None else sel.f64(w))
    terms = np.abs(ww * sel.f64(rstd)[..., None])
    near(g["dx"], gr, dtype, terms + np.abs(gr))
    near(g["dweight"], dw, size=size)
    if dr is None:
        assert g["dresidual"] is None
    elif dr.dtype == dy.dtype:
        assert g["dresidual"] is g["dx"]
    else:
        near(g["dresidual"], gr, res, terms + np.abs(gr))


# every form that holds a row, in both directions, whole vectors and single elements, and the long ones
DIMS = [1, 2, 7, 8, 16, 100, 128, 129, 136, 255, 512, 520, 1000, 1024, 1032, 1531, 1536, 2048, 2050, 2560, 2568, 4096, 4104, 6144, 6150, 8192,
        8200, 16384, 16392, 20001]


@pytest.mark.parametrize("dtype,res", [("bf16", "fp32"), ("fp32", None), ("bf16", "bf16")])
@pytest.mark.parametrize("dim", DIMS)
def test_widths(dtype, res, dim):
    check(draw(dim, 21, dim, dtype, res), dtype, res)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("res", [None, "fp32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 64), (1, 2560), (513, 96), (2050, 40), (5000, 16), (700, 21), (1030, 2560), (530, 8200)])
def test_rows(dtype, res, rows, dim):
    check(draw(rows + dim, rows, dim, dtype, res), dtype, res)


@pytest.mark.parametrize("dim", [320, 321])
def test_without_weight(dim):
    check(draw(3, 40, dim, "bf16", "fp32"), "bf16", "fp32", weight=False)


def test_zero_rows_tiny_and_large():
    """Rows of zeros (scales of 2^-126, all zero), of the type's small and large values."""
    x, _, w, dy, _ = draw(4, 6, 300, "fp32", None)
    x[0] = 0
    x[1] = 1e-30 * x[1]
    x[2] = 1e15 * x[2]
    x[3, :128] = 0
    check((x, None, w, dy, None), "fp32", None)
    q, s, _ = ssd.rms_norm_quant(x.cuda(), w.cuda())
    torch.cuda.synchronize()
    assert (s[0] == 2.0 ** -126).all() and (q[0].float() == 0).all() and s[3, 0] == 2.0 ** -126


def test_not_finite_stays_in_its_row():
    x, r, w, dy, dr = (t.cuda() for t in draw(5, 30, 1531, "bf16", "fp32"))
    bad = x.clone()
    bad[7, 100] = float("nan")
    bad[9, 5] = float("inf")
    keep = [i for i in range(30) if i not in (7, 9)]
    y, ro, rs = ssd.rms_norm_fwd(x, w, residual=r)
    yb, rob, rsb = ssd.rms_norm_fwd(bad, w, residual=r)
    q, s, _ = ssd.rms_norm_quant(x, w, residual=r)
    qb, sb, _ = ssd.rms_norm_quant(bad, w, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(y[keep], yb[keep]) and torch.equal(rs[keep], rsb[keep]) and torch.isnan(yb[7]).all()
    assert torch.equal(q[keep].float(), qb[keep].float()) and torch.equal(s[keep], sb[keep])


@pytest.mark.parametrize("dim", [2560, 1531, 20001])
def test_in_place(dim):
    x, r, w, dy, dr = (t.cuda() for t in draw(6, 30, dim, "bf16", "bf16"))
    y, ro, rs = ssd.rms_norm_fwd(x, w, residual=r)
    g = ssd.rms_norm_bwd(ro, dy, rs, w, dresidual=dr)
    x2, r2 = x.clone(), r.clone()
    y2, ro2, _ = ssd.rms_norm_fwd(x2, w, residual=r2, y=x2, residual_out=r2)
    x3 = x.clone()
    q, s, _ = ssd.rms_norm_quant(x, w, residual=r)
    q3, s3, ro3 = ssd.rms_norm_quant(x3, w, residual=r, residual_out=x3)
    dy2, dr2 = dy.clone(), dr.clone()
    g2 = ssd.rms_norm_bwd(ro, dy2, rs, w, dresidual=dr2, grads={"dx": dy2, "dresidual": dr2})
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(r2, ro) and torch.equal(x3, ro) and torch.equal(q.float(), q3.float()) and torch.equal(s, s3)
    assert torch.equal(g2["dx"], g["dx"]) and g2["dx"].data_ptr() == dy2.data_ptr() and torch.equal(g2["dweight"], g["dweight"])
    assert torch.equal(dr2, g["dx"])


def test_leading_axes_and_no_rows():
    x, r, w, dy, dr = (t.cuda() for t in draw(7, 24, 200, "fp32", "fp32"))
    y, ro, rs = ssd.rms_norm_fwd(x, w, residual=r)
    q, s, _ = ssd.rms_norm_quant(x.view(2, 3, 4, 200), w, residual=r.view(2, 3, 4, 200))
    y3, _, rs3 = ssd.rms_norm_fwd(x.view(2, 3, 4, 200), w, residual=r.view(2, 3, 4, 200))
    assert q.shape == (2, 3, 4, 200) and s.shape == (2, 3, 4, 2) and rs3.shape == (2, 3, 4) and torch.equal(y3.view(24, 200), y)
    e = ssd.rms_norm_fwd(x[:0], w, residual=r[:0])
    g = ssd.rms_norm_bwd(e[1], dy[:0], e[2], w, grads={"dweight": torch.ones(200, device="cuda")})
    torch.cuda.synchronize()
    assert e[0].shape == (0, 200) and not g["dweight"].any()


def test_captured_and_on_another_stream():
    x, r, w, dy, dr = (t.cuda() for t in draw(8, 600, 320, "bf16", "fp32"))

    def both(stream=None):
        y, ro, rs = ssd.rms_norm_fwd(x, w, residual=r, stream=stream)
        q, s, _ = ssd.rms_norm_quant(x, w, residual=r, stream=stream)
        g = ssd.rms_norm_bwd(ro, dy, rs, w, dresidual=dr, stream=stream)
        return [y, ro, rs, q.view(torch.uint8), s, g["dx"], g["dresidual"], g["dweight"]]

    want = [t.clone() for t in both()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = both(st.cuda_stream)
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
