"""A block's training step with the new operators in a row: layer norm, a projection to q, k
and v, the gated delta rule, and back through all of them, in one graph replayed.  Each
operator's gradients are held to the fp64 formulas on what the operator was given."""
import numpy as np
import pytest
import torch

from oracle import delta
from ssd_chunked_scan_amd import ssd
from test_gpu_gdr import DV, TOL, f64, rel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 63, 200])
def test_a_training_step(dtype, T):
    b, H, P, N, G, D = 2, 6, 32, 48, 2, 160
    el = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)
    x, w, bias = rnd(b, T, D).to(el), 1 + 0.1 * rnd(D), 0.1 * rnd(D)
    # (k and q of about unit length: rows of the projection of length 1 / sqrt(N))
    cols = H * P + 2 * G * N
    proj = (rnd(D, cols) / D ** 0.5 * torch.cat([torch.ones(H * P, device="cuda"),
                                                 torch.full((2 * G * N,), N ** -0.5, device="cuda")])).to(el)
    back = proj.t().contiguous()
    g = (-0.2 * torch.rand(b, T, H, device="cuda", generator=gen)).to(el)
    beta = torch.rand(b, T, H, device="cuda", generator=gen).to(el)
    dy, dfin = rnd(b, T, H, P).to(el), 0.3 * rnd(b, H, P, N)

    def step():
        n, mean, rstd = ssd.layer_norm_fwd(x, w, bias)
        u = (n.view(b * T, D) @ proj).view(b, T, cols)
        v = u[..., :H * P].reshape(b, T, H, P).contiguous()
        k, q = (u[..., H * P + i * G * N:H * P + (i + 1) * G * N].reshape(b, T, G, N).contiguous() for i in range(2))
        y, fin = ssd.gdr_fwd(q, k, v, g, beta, scale=N ** -0.5)
        gr = ssd.gdr_bwd(q, k, v, g, beta, dy, scale=N ** -0.5, dfinal_states=dfin)
        du = torch.cat([gr["dv"].view(b, T, -1), gr["dk"].view(b, T, -1), gr["dq"].view(b, T, -1)], -1)
        dn = (du.view(b * T, cols) @ back).view(b, T, D)
        gn = ssd.layer_norm_bwd(x, dn, mean, rstd, w)
        return [q, k, v, y, fin, *(gr[m] for m in ("dq", "dk", "dv", "dg", "dbeta")), dn, mean, rstd, gn["dx"], gn["dweight"],
                gn["dbias"]]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    q, k, v, y, fin, dq, dk, dv, dg, dbeta, dn, mean, rstd, dx, dw, db = want
    c = lambda t: t.cpu()
    yr, fr = delta.gdr_forward(c(q), c(k), c(v), c(g), c(beta), N ** -0.5)
    r = delta.gdr_backward(c(q), c(k), c(v), c(g), c(beta), c(dy), N ** -0.5, dfinal_states=c(dfin))
    assert rel(f64(y), yr) <= TOL[dtype] and rel(f64(fin), fr) <= 1e-4
    for got, name in ((dq, "dq"), (dk, "dk"), (dbeta, "dbeta")):
        assert rel(f64(got), r[name]) <= TOL[dtype], name
    assert rel(f64(dv), r["dv"]) <= DV[dtype]
    # (fresh states: dg of a sequence of one token is 0)
    assert rel(f64(dg), r["dg"]) <= TOL[dtype] if T > 1 else not dg.any()
    rx, rw, rb = delta.layer_norm_backward(c(x), c(dn), c(mean), c(rstd), c(w))
    xhat = (f64(x) - f64(mean)[..., None]) * f64(rstd)[..., None]
    terms = np.linalg.norm(np.abs(f64(dn) * xhat).sum((0, 1))), np.linalg.norm(np.abs(f64(dn)).sum((0, 1)))
    assert rel(f64(dx), rx) <= (2.0 ** -8 if dtype == "bf16" else 1e-5)
    assert np.linalg.norm(f64(dw) - rw) <= 1e-5 * terms[0] and np.linalg.norm(f64(db) - rb) <= 1e-5 * terms[1]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(out, want)), i
        step()
