"""GPU parity of the 8-bit block-scaled product (ssd_matmul_fp8) against fp64.

Bars, counted before the first run.  fp32 outputs: products of two e4m3 numbers have 8 bits and are exact in fp32; a
block's sum and the sum over blocks are in fp32, off by up to a few times 2^-24 of their terms' sizes a step, at
random: every value is within 1e-5 of its terms' sizes for the 10000s of terms here.  bf16 outputs are rounded once, 2^-8 of
themselves, and their products are added to 13 bits below the largest: with normal numbers, the largest about 4
times the mean, a product is off by at most 4 * 2^-13 of the mean, at random, a sum of 128 by 4 * 2^-13 / sqrt(3 * 128) = 2.5e-5
of its terms' sizes at one sigma if every product lost its whole step, in norm over a row or a column a fraction
of that: 1e-5.
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


def draw(seed, m, n, k):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)
    kb, nb = -(-k // 128), -(-n // 128)
    f8 = lambda t: (t * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    return f8(rnd(m, k)), torch.exp(rnd(m, kb)), f8(rnd(n, k)), torch.exp(rnd(nb, kb)), rnd(n)


def check(case, dtype="fp32", bias=False):
    a, sa, w, sw, b = case
    b = b if bias else None
    out = ssd.matmul_fp8(a, sa, w, sw, bias=b, out_dtype=EL[dtype])
    torch.cuda.synchronize()
    ref, size = sel.matmul_fp8(a, sa, w, sw, b)
    got = sel.f64(out)
    assert got.shape == ref.shape and np.isfinite(got).all()
    err = np.abs(got - ref)
    if dtype == "fp32":
        assert (err <= 1e-5 * size + 1e-6 * np.abs(ref)).all(), (err / size).max()
        return
    for axis in (0, 1):
        n = lambda v: np.linalg.norm(v, axis=axis)
        assert (n(err) <= 1e-5 * n(size) + ROUND[dtype] * n(ref)).all(), (n(err) / n(ref)).max()


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 100])
@pytest.mark.parametrize("n,k", [(128, 128), (200, 400), (1531, 1040), (2560, 2560), (8200, 3840)])
def test_few_rows(m, n, k):
    check(draw(m + n, m, n, k), "bf16" if m % 2 else "fp32")


@pytest.mark.parametrize("n", [1, 2, 3, 5, 127, 128, 129, 130])
@pytest.mark.parametrize("k", [16, 112, 128, 144, 272])
def test_odd_columns_and_short_inner(n, k):
    check(draw(n + k, 20, n, k), "fp32", True)
    check(draw(n + k, 70, n, k), "bf16", True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(2048, 2048, 256), (2000, 2049, 400), (1999, 1999, 16), (4096, 4096, 128), (4100, 3999, 272), (4095, 4097, 1040), (4000, 4104, 272),
                                   (2050, 2056, 128), (4608, 4608, 384), (20000, 300, 512)])
def test_tiles(dtype, m, n, k):
    check(draw(m, m, n, k), dtype, True)


def test_long_inner():
    check(draw(1, 3, 130, 20000), "fp32")
    check(draw(2, 300, 300, 20000), "fp32")
    check(draw(3, 1600, 1600, 10256), "fp32")


def test_zeros_and_largest_values():
    """All 448 with equal signs, 128 long: the largest a block's sum can be; zero rows and zero scales."""
    a, sa, w, sw, b = draw(4, 40, 140, 256)
    a = torch.full_like(a, 448.0)
    w = torch.full_like(w, -448.0)
    a[3] = 0
    sa[5] = 0
    check((a, sa, w, sw, b), "fp32")


def test_not_finite_stays_in_its_row_or_column():
    a, sa, w, sw, b = draw(5, 300, 300, 400)
    for m in (300, 20):
        aa = a[:m].contiguous()
        good = ssd.matmul_fp8(aa, sa[:m].contiguous(), w, sw)
        bad_a, bad_w = aa.clone(), w.clone()
        bad_a.view(torch.uint8)[7, 399] = 0x7f   # NaN
        bad_w.view(torch.uint8)[11, 0] = 0xff
        got = ssd.matmul_fp8(bad_a, sa[:m].contiguous(), bad_w, sw)
        torch.cuda.synchronize()
        keep = torch.ones_like(good, dtype=torch.bool)
        keep[7] = False
        keep[:, 11] = False
        assert torch.equal(good[keep], got[keep]) and torch.isnan(got[~keep]).all()


def test_rows_do_not_depend_on_their_company():
    """A row's values do not change with other rows in the same form of the product."""
    a, sa, w, sw, _ = draw(6, 64, 512, 1024)
    whole = ssd.matmul_fp8(a, sa, w, sw)
    part = ssd.matmul_fp8(a[5:6].contiguous(), sa[5:6].contiguous(), w, sw)
    torch.cuda.synchronize()
    near = (whole[5].float() - part[0].float()).abs() <= 2.0 ** -7 * whole[5].float().abs() + 1e-3
    assert near.all()


def test_leading_axes_and_nothing():
    a, sa, w, sw, b = draw(7, 24, 96, 256)
    out = ssd.matmul_fp8(a.view(2, 3, 4, 256), sa.view(2, 3, 4, 2), w, sw)
    assert out.shape == (2, 3, 4, 96) and torch.equal(out.view(24, 96), ssd.matmul_fp8(a, sa, w, sw))
    assert ssd.matmul_fp8(a[:0], sa[:0], w, sw).shape == (0, 96)
    assert ssd.matmul_fp8(a, sa, w[:0], sw[:0]).shape == (24, 0)


def test_the_norm_s_output():
    """What rms_norm_quant leaves, through the product: the product of what it stands for."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(70, 1000, device="cuda", generator=gen).bfloat16()
    _, _, w, sw, _ = draw(8, 1, 300, 1000 // 16 * 16)
    x = x[:, :992].contiguous()
    q, s, _ = ssd.rms_norm_quant(x)
    check((q, s, w, sw, None), "bf16")


def test_captured_on_another_stream_and_repeatable():
    few, many = draw(9, 40, 1000, 2048), draw(10, 2048, 2048, 512)

    def both(stream=None):
        return [ssd.matmul_fp8(*c[:4], bias=c[4], stream=stream) for c in (few, many)]

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


def test_past_2_to_the_32_bytes():
    """An output of 4.9 GB: its last rows."""
    a, sa, w, sw, b = draw(11, 300000, 8200, 32)
    out = ssd.matmul_fp8(a, sa, w, sw)
    tail = ssd.matmul_fp8(a[-2048:].contiguous(), sa[-2048:].contiguous(), w, sw)
    torch.cuda.synchronize()
    assert torch.equal(out[-2048:], tail)
