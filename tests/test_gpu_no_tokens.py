"""The SSD without any tokens (seqlen 0)."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_gradients_of_rows_without_tokens(dtype):
    """The final state is the initial state: its gradient passes straight through."""
    b, H, P, N, G = 2, 4, 32, 48, 2
    z = lambda *s, dt=dtype: torch.zeros(s, dtype=dt, device="cuda")
    args = (z(b, 0, H, P), z(b, 0, H), -torch.ones(H, device="cuda"), z(b, 0, G, N), z(b, 0, G, N), 64)
    dfin = torch.randn(b, H, P, N, device="cuda")
    y = z(b, 0, H, P)
    gr = ssd.bwd(*args, y, y.clone(), D=torch.ones(H, device="cuda"), dfinal_states=dfin)
    torch.cuda.synchronize()
    assert bool((gr["dinitial_states"] == dfin).all())
    assert bool((gr["dA"] == 0).all()) and bool((gr["dD"] == 0).all()) and gr["dx"].numel() == 0
