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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_an_empty_packed_stream(dtype):
    """Every segment's final state is zero (none of its tokens received the initial state), and
    so is the gradient of the initial state."""
    nseq, H, P, N, G = 3, 2, 32, 48, 1
    z = lambda *s, dt=dtype: torch.zeros(s, dtype=dt, device="cuda")
    args = (z(1, 0, H, P), z(1, 0, H), -torch.ones(H, device="cuda"), z(1, 0, G, N), z(1, 0, G, N), 64)
    kw = dict(initial_states=torch.randn(1, H, P, N, device="cuda"), seq_idx=z(0, dt=torch.int32), nseq=nseq)
    fin = torch.full((nseq, H, P, N), 7.0, device="cuda")
    y, f = ssd.fwd(*args, **kw, final_states=fin)
    gr = ssd.bwd(*args, y, y.clone(), **kw, dfinal_states=torch.randn(nseq, H, P, N, device="cuda"))
    torch.cuda.synchronize()
    assert f is fin and y.numel() == 0
    assert bool((fin == 0).all())
    assert bool((gr["dinitial_states"] == 0).all())
