"""The 8-bit product where a few products of a block of 128 are far larger than the rest: a channel that
stands out of the activations, two such channels that cancel, and small products of one sign beside them.

Bars, counted before the first run.  Products of two e4m3 numbers are exact in fp32 and every sum is held in fp32: a sum
of 128 of them is off by at most 127 * 2^-24 = 7.6e-6 of its terms' sizes whatever their order, the blocks' scaling and
sums (fewer than 20) by 21 * 2^-24 = 1.3e-6 more: every value is within 1e-5 of its terms' sizes.  A bf16 output is rounded
once more: half a step, 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import selective as sel
from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def draw(kind, m, n, k):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)
    kb, nb = -(-k // 128), -(-n // 128)
    a, w = rnd(m, k), 60 * rnd(n, k)
    big = torch.arange(k, device="cuda") % 128
    if kind == "channel":      # one channel of a block 100 times the others, whose values are what that leaves of 448
        a = torch.where(big == 5, 448 * torch.sign(a), 1.5 * a)
    else:                      # two channels that cancel: what is left is the others' sum
        a = torch.where(big == 0, 448.0, torch.where(big == 9, -448.0, 0.25 * a))
        w = torch.where(big == 9, w.roll(9, 1), w)
        if kind == "cancel_one_sign":   # of products just under 2^-13 of the two
            a, w = torch.where((big == 0) | (big == 9), a, 0.25), torch.where((big == 0) | (big == 9), 448.0, 80.0 + 0 * w)
    f8 = lambda t: t.clamp(-448, 448).to(torch.float8_e4m3fn)
    return f8(a), torch.exp(0.3 * rnd(m, kb)), f8(w), torch.exp(0.3 * rnd(nb, kb))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["channel", "cancel", "cancel_one_sign"])
@pytest.mark.parametrize("m,n,k", [(1, 200, 128), (16, 640, 1024), (20, 300, 400), (64, 2560, 2560), (300, 129, 1040), (2048, 2048, 512),
                                   (1999, 2047, 272), (4096, 4096, 384)])
def test_small_products_beside_large_ones(kind, dtype, m, n, k):
    case = draw(kind, m, n, k)
    out = ssd.matmul_fp8(*case, out_dtype=dtype)
    torch.cuda.synchronize()
    ref, size = sel.matmul_fp8(*case)
    err = np.abs(sel.f64(out) - ref)
    assert (err <= 1e-5 * size + ROUND[dtype] * np.abs(ref)).all(), ((err - ROUND[dtype] * np.abs(ref)) / size).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(50, 640, 2560), (1200, 1100, 400)])   # few rows, tiles
def test_a_row_does_not_change_with_the_others(dtype, m, n, k):
    """Same sizes, so the same form of the product: other rows' contents, NaN among them, change no bit of a row."""
    a, sa, w, sw = draw("channel", m, n, k)
    want = ssd.matmul_fp8(a, sa, w, sw, out_dtype=dtype)
    keep = [0, 17, m - 1]
    other, so = draw("cancel", m, n, k)[:2]
    other.view(torch.uint8)[5] = 0x7f
    other.view(torch.uint8)[keep] = a.view(torch.uint8)[keep]
    so[keep] = sa[keep]
    got = ssd.matmul_fp8(other, so, w, sw, out_dtype=dtype)
    torch.cuda.synchronize()
    assert torch.equal(got[keep], want[keep]) and not torch.equal(got[1], want[1]) and torch.isnan(got[5]).all()
