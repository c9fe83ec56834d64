"""A packed stream of the gated delta rule without any tokens: every segment's final state
is its initial state, and the gradient passes straight through, for all segments."""
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
@pytest.mark.parametrize("init", [True, False], ids=["carried", "fresh"])
def test_every_segment_keeps_its_state(dtype, init):
    nseq, H, P, N, G = 3, 2, 32, 48, 1
    z = lambda *s, dt=dtype: torch.zeros(s, dtype=dt, device="cuda")
    x = dict(q=z(1, 0, G, N), k=z(1, 0, G, N), v=z(1, 0, H, P), g=z(1, 0, H), beta=z(1, 0, H), seq_idx=z(0, dt=torch.int32),
             nseq=nseq, initial_states=torch.randn(nseq, H, P, N, device="cuda") if init else None)
    want = x["initial_states"] if init else z(nseq, H, P, N, dt=torch.float32)
    fin, dinit = (torch.full((nseq, H, P, N), 7.0, device="cuda") for _ in range(2))
    dfin = torch.randn(nseq, H, P, N, device="cuda")
    y, f = ssd.gdr_fwd(**x, final_states=fin)
    gr = ssd.gdr_bwd(**x, dy=y.clone(), dfinal_states=dfin, grads={"dinitial_states": dinit})
    torch.cuda.synchronize()
    assert f is fin
    assert bool((fin == want).all())
    assert bool((gr["dinitial_states"] == dfin).all())
