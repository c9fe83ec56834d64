"""Sizes of the selective scan that a direction's own launches take: a forward past what its gradients can have, single
tokens out of long rows.  Bars: fp32 sums in another order, 1e-5; bf16 outputs rounded once on either side, 2 * 2^-8."""
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


def near(got, want, bar):
    return (got.float() - want.float()).norm() <= bar * want.float().norm()


def test_forward_of_many_groups():
    b, T, dim, N = 513, 1024, 256, 16   # 2^29 / 4 keys and more
    x = torch.randn(b, T, dim, device="cuda", dtype=torch.bfloat16)
    B, C = (torch.randn(b, T, dim, N, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    A = -torch.rand(dim, N, device="cuda") - 0.1
    y, fin = ssd.selective_scan_fwd(x, x, A, B, C)
    with pytest.raises(ssd.SSDError):
        ssd.selective_scan_bwd(x, x, A, B, C, x)
    for r in (0, b - 1):
        y1, fin1 = ssd.selective_scan_fwd(*(t[r:r + 1] if t is not A else A for t in (x, x, A, B, C)))
        torch.cuda.synchronize()
        assert near(fin[r], fin1[0], 1e-5) and near(y[r], y1[0], 2 * 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_single_tokens_of_long_rows(dtype):
    b, T, dim, N = 3, 3001, 2000, 16   # 6 M elements from row to row
    x, z, dt = (torch.randn(b, T, dim, device="cuda").to(dtype) for _ in range(3))
    B, C = (torch.randn(b, T, 90, N, device="cuda").to(dtype) for _ in range(2))   # 4.3 M
    A, D = -torch.rand(dim, N, device="cuda"), torch.randn(dim, device="cuda")
    state = torch.randn(b, dim, N, device="cuda")
    other = state.clone()
    for t in (0, T - 1):
        part = [v[:, t] for v in (x, dt, B[:, :, :1], C[:, :, 3:4], z)]
        got = ssd.selective_scan_step(part[0], part[1], A, part[2], part[3], state, D=D, z=part[4])
        part = [v.contiguous() for v in part]
        want = ssd.selective_scan_step(part[0], part[1], A, part[2], part[3], other, D=D, z=part[4])
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, other)
