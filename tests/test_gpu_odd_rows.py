"""RMS norm and the 8-bit product with rows that are not whole vectors, in every form a row takes and at every
remainder of its length, in buffers with something behind them.

Bars: fp32 sums and one rounding of each output: 1e-6 in norm for fp32, half a step (2^-8) beside it for bf16;
8-bit values half a step (2^-4 of themselves, or of the smallest normal value, 2^-10 in units of the scale) beside
1e-5; the product's bf16 outputs 2^-8 and 5e-5 of their terms.
"""
import numpy as np
import pytest
import torch

from oracle import selective as sel
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

EL = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": 1e-6, "bf16": 2.0 ** -8 + 1e-6}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def behind(shape, dtype):
    """A tensor and the buffer that goes on behind it."""
    n, size = int(np.prod(shape)), torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n * size + 256,), 0x41, dtype=torch.uint8, device="cuda")
    return buf[n * size:], buf[:n * size].view(dtype).view(shape)


def near(got, ref, bar, size=None):
    got = sel.f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    assert np.linalg.norm(got - ref) <= bar * np.linalg.norm(ref if size is None else size) + 1e-30


@pytest.mark.parametrize("dtype,res", [("bf16", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("dim", [*range(1, 17), 121, 127, 129, 135, 513, 1021, 1030, 2047, 4099, 8187, 8191, 8193, 16383, 16385, 20001])
def test_norm(dtype, res, dim):
    rows = 5
    gen = torch.Generator().manual_seed(dim)
    t = lambda *s: torch.randn(*s, generator=gen)
    x, r, w, dy, dr = t(rows, dim).to(EL[dtype]), t(rows, dim).to(EL[res]), t(dim), t(rows, dim).to(EL[dtype]), t(rows, dim).to(EL[res])
    c = lambda v: v.cuda()
    (b0, y), (b1, ro), (b2, rstd) = behind((rows, dim), EL[dtype]), behind((rows, dim), EL[res]), behind((rows,), torch.float32)
    ssd.rms_norm_fwd(c(x), c(w), residual=c(r), y=y, residual_out=ro, rstd=rstd)
    (b3, q), (b4, s) = behind((rows, dim), F8), behind((rows, -(-dim // 128)), torch.float32)
    ssd.rms_norm_quant(c(x), c(w), residual=c(r), q=q, scales=s)
    (b5, dx), (b6, dres), (b7, dw) = behind((rows, dim), EL[dtype]), behind((rows, dim), EL[res]), behind((dim,), torch.float32)
    grads = dict(dx=dx, dweight=dw)
    if dtype != res:
        grads["dresidual"] = dres
    ssd.rms_norm_bwd(ro, c(dy), rstd, c(w), dresidual=c(dr), grads=grads)
    torch.cuda.synchronize()
    for b in (b0, b1, b2, b3, b4, b5, b6, b7):
        assert (b == 0x41).all()
    stream = (x.float() + r.float()).to(EL[res])
    assert torch.equal(ro.cpu(), stream)
    yr, rr = sel.rms_norm(stream, w)
    near(y, yr, HALF[dtype])
    near(rstd, rr, 1e-6)
    scales, units = sel.to_8bit(yr)
    near(s, scales, 1e-5)
    err = np.abs(sel.f64(q) - units)
    assert (err <= np.maximum(np.abs(units) * 2.0 ** -4, 2.0 ** -10) + 1e-5 * 448).all()
    d, dwr, size = sel.rms_norm_backward(stream, dy, rr, w, dr)
    near(dx, d, HALF[dtype])
    if dtype != res:
        near(dres, d, HALF[res])
    near(dw, dwr, 1e-6 * 4, size)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("m,n,k", [*((4090, 4096 + i, 48) for i in (1, 2, 3, 4, 5, 6, 7)), (1700, 1811, 144), (1700, 1812, 144), (1601, 1794, 144),
                                   (9, 61, 272), (33, 66, 2064), (64, 1029, 272)])
def test_product(dtype, bias, m, n, k):
    gen = torch.Generator().manual_seed(n)
    t = lambda *s: torch.randn(*s, generator=gen)
    a, w, kb = t(m, k).to(F8), t(n, k).to(F8), -(-k // 128)
    sa, sw, b = torch.rand(m, kb, generator=gen) + 0.5, torch.rand(-(-n // 128), kb, generator=gen) + 0.5, t(n) if bias else None
    rest, out = behind((m, n), EL[dtype])
    ssd.matmul_fp8(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), bias=None if b is None else b.cuda(), out_dtype=EL[dtype], out=out)
    torch.cuda.synchronize()
    assert (rest == 0x41).all()
    ref, size = sel.matmul_fp8(a, sa, w, sw, b)
    near(out, ref, HALF[dtype])
    if dtype == "bf16":
        assert (np.abs(sel.f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 5e-5 * size + 1e-6 * np.abs(ref).max()).all()
