"""Values that are not finite in the selective scan's gradients: dB and dC of a token are not finite where the formula's
are not, and stay what they are everywhere else; so do the other channels' gradients.

Bars as in the scan's other tests: fp32 throughout, 1e-5 of the terms' sizes in norm.
"""
import numpy as np
import pytest
import torch

from oracle import selective as sel
from ssd_chunked_scan_amd import ssd

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("what", ["dy", "x", "dy_nan"])
@pytest.mark.parametrize("T,dim,N,G,t0", [(45, 9, 16, 1, 21), (45, 70, 16, 2, 44), (150, 40, 4, 1, 70), (150, 33, 7, 1, 9), (100, 20, 13, 2, 0), (100, 40, 30, 1, 64),
                                          (70, 18, 50, 1, 37), (64, 16, 64, 2, 63)])
def test_only_what_depends_on_it(T, dim, N, G, t0, what, gate):
    rng = np.random.default_rng(T + dim + N)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    x, dt, dy, z, B, C = t(1, T, dim), 0.5 * t(1, T, dim), t(1, T, dim), t(1, T, dim) if gate else None, t(1, T, G, N), t(1, T, G, N)
    A, D, bias = -torch.exp(0.5 * t(dim, N)), t(dim), t(dim) - 2
    d0 = dim // 2
    (x if what == "x" else dy)[0, t0, d0] = float("nan" if what == "dy_nan" else "inf")
    ref = sel.scan_backward(x, dt, A, B, C, dy, D=D, z=z, dt_bias=bias)
    c = lambda v: None if v is None else v.cuda()
    g = ssd.selective_scan_bwd(c(x), c(dt), c(A), c(B), c(C), c(dy), D=c(D), z=c(z), dt_bias=c(bias))
    torch.cuda.synchronize()
    for name in ("dB", "dC"):
        got, want, size = sel.f64(g[name]), ref[name], ref["sizes"][name]
        good = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), good), (name, np.argwhere(np.isfinite(got) != good)[:5])
        assert np.linalg.norm(got[good] - want[good]) <= 1e-5 * np.linalg.norm(size[good])
    others = np.arange(dim) != d0
    for name in ("dx", "ddt", "dA", "dD", "ddt_bias") + (("dz",) if gate else ()):
        got, want = sel.f64(g[name]), ref[name]
        got, want = (got[others], want[others]) if name in ("dA", "dD", "ddt_bias") else (got[..., others], want[..., others])
        size = {"dx": want, "dz": want}.get(name)
        size = ref["sizes"][name][others] if name in ("dA", "dD", "ddt_bias") else ref["sizes"][name][..., others] if size is None else size
        assert np.isfinite(got).all() and np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(size), name
