"""RMS norm of rows of a length that is no multiple of 8 at any element: slices of taller tensors give the same bits as
copies of them."""
import pytest
import torch

from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dim", [1, 9, 127, 513, 2561, 8193, 16385])
@pytest.mark.parametrize("dtype,res", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16)])
def test_slices(dtype, res, dim):
    rows, rnd = 6, lambda t: torch.randn(7, dim, device="cuda").to(t)
    x, r, dy, dr, w = rnd(dtype), rnd(res), rnd(dtype), rnd(res), torch.randn(dim, device="cuda")
    outs = lambda: {n: torch.full((rows + 2, dim), 1.0, device="cuda").to(t) for n, t in
                    (("y", dtype), ("residual_out", res), ("q", F8), ("dx", dtype), ("dresidual", res))}

    def run(cut, o):
        a, b, d, e = cut(x), cut(r), cut(dy), cut(dr)
        at = {n: (t[1:-1] if cut is slice_ else t[1:-1].clone()) for n, t in o.items()}
        _, _, rstd = ssd.rms_norm_fwd(a, w, residual=b, y=at["y"], residual_out=at["residual_out"])
        q, s, _ = ssd.rms_norm_quant(a, w, residual=b, q=at["q"])
        grads = {"dx": at["dx"], **({"dresidual": at["dresidual"]} if dtype != res else {})}
        g = ssd.rms_norm_bwd(at["residual_out"], d, rstd, w, dresidual=e, grads=grads)
        plain = ssd.rms_norm_fwd(a, w)[0]
        return [at["y"], at["residual_out"], rstd, q.view(torch.uint8), s, g["dx"], g["dresidual"], g["dweight"], plain]

    slice_, copy = lambda t: t[1:], lambda t: t[1:].clone()
    o = outs()
    got, want = run(slice_, o), run(copy, outs())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t[[0, -1]].float() == 1).all() for t in o.values())   # the rows around


def test_in_place_at_an_element():
    x = torch.randn(9, 301, device="cuda").bfloat16()
    want = ssd.rms_norm_fwd(x[1:].clone())[0]
    ssd.rms_norm_fwd(x[1:], y=x[1:])
    torch.cuda.synchronize()
    assert torch.equal(x[1:], want)
