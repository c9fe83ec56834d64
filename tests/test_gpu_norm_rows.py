"""Layer norm over more rows than one launch takes (2^21): the rows around the boundary and
the last ones are what a call on them alone gives, bit for bit (a row's arithmetic does not
depend on the others)."""
import pytest
import torch

from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


# rows held by 16 lanes, by single elements, and longer than the registers
@pytest.mark.parametrize("dim", [8, 3, 2049])
def test_more_rows_than_a_launch(dim):
    rows = (1 << 21) + 24
    gen = torch.Generator(device="cuda")
    gen.manual_seed(dim)
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty_like(x)
    for i in range(0, rows, 1 << 19):
        x[i:i + (1 << 19)].normal_(generator=gen)
        dy[i:i + (1 << 19)].normal_(generator=gen)
    w = torch.randn(dim, device="cuda", generator=gen)
    y, mean, rstd = ssd.layer_norm_fwd(x, w, w)
    dx = ssd.layer_norm_bwd(x, dy, mean, rstd, w, want_params=False)["dx"]
    for lo, hi in ((0, 40), ((1 << 21) - 40, (1 << 21) + 8), (rows - 16, rows)):
        cut = lambda t: t[lo:hi].clone()
        y1, m1, r1 = ssd.layer_norm_fwd(cut(x), w, w)
        d1 = ssd.layer_norm_bwd(cut(x), cut(dy), m1, r1, w, want_params=False)["dx"]
        torch.cuda.synchronize()
        for a, b in ((y, y1), (mean, m1), (rstd, r1), (dx, d1)):
            assert torch.equal(a[lo:hi], b), (dim, lo)
