"""The gated delta rule at sizes that change how it stores and addresses: triangles past
256 MiB, which the preparing kernel writes past the caches (other kernels than the smaller
tests run), and a backward whose tensors pass 2^32 bytes.

Bars: bf16 as in test_gpu_gdr_rounding.py, fp32 and states as in test_gpu_gdr.py."""
import numpy as np
import pytest
import torch

from oracle import delta
from ssd_chunked_scan_amd import ssd
from test_gpu_gdr import STATE, TOL, draw, f64, gpu, worst_states, worst_tokens
from test_gpu_gdr_rounding import GRADS, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def group(x, dy, dfin, j):
    """Group j of a problem and its heads, as a problem of its own."""
    n = x["v"].shape[2] // x["k"].shape[2]
    hs = slice(j * n, (j + 1) * n)
    y = dict(x, q=x["q"][:, :, j:j + 1], k=x["k"][:, :, j:j + 1], initial_states=x["initial_states"][:, hs])
    return y | {m: x[m][:, :, hs] for m in ("v", "g", "beta")}, dy[:, :, hs], dfin[:, hs], hs


# chunks * heads of 24 KiB of triangles (forward) and 36 KiB (backward): past 256 MiB.  With
# 196 heads a workgroup takes 64 columns, with 48 heads 16.
SIZES = {"wide": (3901, 196, 49), "narrow": (15500, 48, 24)}


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("size", SIZES)
def test_triangles_past_the_caches(size, N, dtype):
    T, H, G = SIZES[size]
    P = 16
    assert (T + 63) // 64 * H * 24 * 1024 > 256 << 20
    x, dy, dfin = draw(N + H, 1, T, H, P, N, G, dtype)
    g = gpu(x)
    y, fin = ssd.gdr_fwd(**g)
    got = ssd.gdr_bwd(**g, dy=dy.cuda(), dfinal_states=dfin.cuda())
    torch.cuda.synchronize()
    off = lambda a, b, p: worst(a, b, p) if dtype == "bf16" else worst_tokens(a, b, p) / TOL[dtype]
    for j in (0, G - 1):
        p, d, df, hs = group(x, dy, dfin, j)
        yr, fr = delta.gdr_forward(**p)
        ref = delta.gdr_backward(**p, dy=d, dfinal_states=df)
        e = {"y": off(f64(y[:, :, hs]), yr, p), "final_states": worst_states(f64(fin[:, hs]), fr) / STATE,
             "dinitial_states": worst_states(f64(got["dinitial_states"][:, hs]), ref["dinitial_states"]) / STATE}
        for n in GRADS:
            cols = slice(j, j + 1) if n in ("dq", "dk") else hs
            e[n] = off(f64(got[n][:, :, cols]), ref[n], p)
        print(f"[gdr large] {size} N={N} {dtype} group {j} " + " ".join(f"{n}={v:.3f}" for n, v in e.items()), flush=True)
        assert max(e.values()) <= 1, e


def test_backward_offsets_past_32_bits():
    """v, dy, dv and the workspace pass 2^32 bytes.  The stream's two halves, which meet at a
    chunk boundary, by themselves give the same bits: the second from the first's final
    state, the first from the second's gradient of it."""
    T, H, P, N = 1 << 16, 32, 1040, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    el = torch.bfloat16

    def values():
        t = torch.empty(1, T, H, P, dtype=el, device="cuda")
        for i in range(0, T, 1 << 13):
            t[:, i:i + (1 << 13)] = torch.randn(1, 1 << 13, H, P, device="cuda", generator=gen).to(el)
        return t

    k = torch.nn.functional.normalize(torch.randn(1, T, H, N, device="cuda", generator=gen), dim=-1).to(el)
    q, v, dy = k.flip(1).contiguous(), values(), values()
    g = (-0.1 * torch.rand(1, T, H, device="cuda", generator=gen)).to(el)
    beta = torch.rand(1, T, H, device="cuda", generator=gen).to(el)
    assert v.numel() * 2 > 1 << 32
    got = ssd.gdr_bwd(q, k, v, g, beta, dy)
    half = T // 2
    part = lambda lo, hi: [t[:, lo:hi].contiguous() for t in (q, k, v, g, beta, dy)]
    first, second = part(0, half), part(half, T)
    _, s1 = ssd.gdr_fwd(*first[:5])
    g2 = ssd.gdr_bwd(*second, initial_states=s1)
    g1 = ssd.gdr_bwd(*first, dfinal_states=g2["dinitial_states"])
    torch.cuda.synchronize()
    for n in GRADS:
        assert torch.equal(got[n][:, half:].contiguous(), g2[n]) and torch.equal(got[n][:, :half].contiguous(), g1[n]), n
    assert torch.equal(got["dinitial_states"], g1["dinitial_states"])
