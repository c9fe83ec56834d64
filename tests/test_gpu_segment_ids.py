"""Packed streams whose ids are the largest and smallest 32-bit numbers: whatever comes out, nothing outside the
outputs and the workspace is written, and the calls end."""
import numpy as np
import pytest
import torch

from ssd_chunked_scan_amd import ssd

pytestmark = pytest.mark.gpu

LEAST, MOST = -2 ** 31, 2 ** 31 - 1
PAD = 4096


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


class Guarded:
    """Tensors with `PAD` elements in front and behind that have to stay as they are."""

    def __init__(self):
        self.bufs = []

    def __call__(self, *shape, dtype=torch.float32):
        n = int(np.prod(shape))
        self.bufs.append(torch.full((n + 2 * PAD,), 7, device="cuda", dtype=dtype))
        return self.bufs[-1][PAD:PAD + n].view(shape)

    def whole(self):
        torch.cuda.synchronize()
        return all((b[:PAD] == 7).all() and (b[-PAD:] == 7).all() for b in self.bufs)


def streams(T, nseq):
    half = torch.arange(T) * nseq // (2 * T)
    some = torch.tensor([LEAST, -1, 0, nseq - 1, nseq, MOST])
    return {"largest": torch.full((T,), MOST), "smallest": torch.full((T,), LEAST), "pads": torch.where(torch.arange(T) < T - 2, half, MOST),
            "one pad": torch.where(torch.arange(T) < T - 1, half, MOST), "from least": torch.where(torch.arange(T) < 5, LEAST, half),
            "falls": torch.where(torch.arange(T) < T // 2, MOST, half), "any": some[torch.randint(0, 6, (T,), generator=torch.Generator().manual_seed(0))]}


KINDS = list(streams(8, 2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,dim,nseq", [(150, 20, 4), (1, 3, 1), (1030, 8, 2)])
def test_scan(kind, T, dim, nseq):
    N, rnd = 16, lambda *s: torch.randn(s, device="cuda")
    x, dt, z, dy, B, C = rnd(1, T, dim), rnd(1, T, dim), rnd(1, T, dim), rnd(1, T, dim), rnd(1, T, 1, N), rnd(1, T, 1, N)
    A, s0 = -torch.rand(dim, N, device="cuda"), rnd(nseq, dim, N)
    ids = streams(T, nseq)[kind].int().cuda()
    kw = dict(D=rnd(dim), z=z, dt_bias=rnd(dim), initial_states=s0, seq_idx=ids, nseq=nseq)
    out = Guarded()
    byte = dict(dtype=torch.uint8)
    ssd.selective_scan_fwd(x, dt, A, B, C, y=out(1, T, dim), final_states=out(nseq, dim, N),
                           workspace=out(ssd.selective_scan_fwd_workspace_bytes(x, dt, A, B, C, seq_idx=ids, nseq=nseq), **byte), **kw)
    assert out.whole()
    shapes = dict(dx=(1, T, dim), ddt=(1, T, dim), dz=(1, T, dim), dA=(dim, N), dB=(1, T, 1, N), dC=(1, T, 1, N), dD=(dim,), ddt_bias=(dim,),
                  dinitial_states=(nseq, dim, N))
    ssd.selective_scan_bwd(x, dt, A, B, C, dy, dfinal_states=rnd(nseq, dim, N), grads={n: out(*s) for n, s in shapes.items()},
                           workspace=out(ssd.selective_scan_bwd_workspace_bytes(x, dt, A, B, C, seq_idx=ids, nseq=nseq), **byte), **kw)
    assert out.whole()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,dim,K,nseq", [(90, 16, 4, 3), (1, 3, 2, 1), (700, 7, 3, 5)])
def test_conv(kind, T, dim, K, nseq):
    rnd = lambda *s: torch.randn(s, device="cuda")
    x, dy, w, b, win = rnd(1, T, dim), rnd(1, T, dim), rnd(dim, K), rnd(dim), rnd(nseq, K - 1, dim)
    kw = dict(bias=b, initial_window=win, seq_idx=streams(T, nseq)[kind].int().cuda(), nseq=nseq)
    out = Guarded()
    ssd.causal_conv_fwd(x, w, y=out(1, T, dim), final_window=out(nseq, K - 1, dim), **kw)
    assert out.whole()
    grads = dict(dx=out(1, T, dim), dweight=out(dim, K), dbias=out(dim), dinitial_window=out(nseq, K - 1, dim))
    ssd.causal_conv_bwd(x, w, dy, dfinal_window=rnd(nseq, K - 1, dim), grads=grads, **kw)
    assert out.whole()


@pytest.mark.parametrize("dim", [3, 18])
def test_conv_with_many_segments_without_tokens(dim):
    """Their windows, and the gradients of those, pass through; the others are what they are by themselves."""
    nseq, K, at = 3000, 4, torch.tensor([7, 8, 8, 8, 8, 1500, 1500, 2998])
    rnd = lambda *s: torch.randn(s, device="cuda")
    x, dy, w, win, dwin = rnd(1, len(at), dim), rnd(1, len(at), dim), rnd(dim, K), rnd(nseq, K - 1, dim), rnd(nseq, K - 1, dim)
    y, fin = ssd.causal_conv_fwd(x, w, initial_window=win, seq_idx=at.int().cuda(), nseq=nseq)
    g = ssd.causal_conv_bwd(x, w, dy, initial_window=win, dfinal_window=dwin, seq_idx=at.int().cuda(), nseq=nseq)
    used = at.unique()
    few = torch.searchsorted(used, at).int().cuda()
    part = dict(initial_window=win[used].contiguous(), seq_idx=few, nseq=len(used))
    y1, fin1 = ssd.causal_conv_fwd(x, w, **part)
    g1 = ssd.causal_conv_bwd(x, w, dy, dfinal_window=dwin[used].contiguous(), **part)
    torch.cuda.synchronize()
    none = torch.ones(nseq, dtype=torch.bool)
    none[used] = False
    assert torch.equal(fin[none], win[none]) and torch.equal(g["dinitial_window"][none], dwin[none])
    assert torch.equal(fin[used], fin1) and torch.equal(g["dinitial_window"][used], g1["dinitial_window"])
    assert torch.equal(y, y1) and all(torch.equal(g[k], g1[k]) for k in ("dx", "dweight"))
    zeros, _ = ssd.causal_conv_fwd(x, w, seq_idx=at.int().cuda(), nseq=nseq, final_window=fin)
    assert torch.equal(fin[none], torch.zeros_like(fin[none]))


@pytest.mark.parametrize("nseq,at", [(3000, [7, 8, 8, 8, 8, 1500, 1500, 2998]), (1100, [0, 1, 9, 10, 27, 1099]), (5000, [4999]), (700, [0, 0, 3]),
                                     (2000, sorted([5, 5, 900, 1999] * 300))])
def test_scan_with_many_segments_without_tokens(nseq, at):
    """Their states, and the gradients of those, pass through; the others are what they are by themselves."""
    dim, N, at = 6, 5, torch.tensor(at)
    T, rnd = len(at), lambda *s: torch.randn(s, device="cuda")
    x, dt, dy, B, C = rnd(1, T, dim), rnd(1, T, dim), rnd(1, T, dim), rnd(1, T, 1, N), rnd(1, T, 1, N)
    A, s0, ds = -torch.rand(dim, N, device="cuda"), rnd(nseq, dim, N), rnd(nseq, dim, N)
    used = at.unique()
    few = torch.searchsorted(used, at).int().cuda()

    def both(states, dstates, ids, n):
        y, fin = ssd.selective_scan_fwd(x, dt, A, B, C, initial_states=states, seq_idx=ids, nseq=n)
        return y, fin, ssd.selective_scan_bwd(x, dt, A, B, C, dy, initial_states=states, dfinal_states=dstates, seq_idx=ids, nseq=n)

    y, fin, g = both(s0, ds, at.int().cuda(), nseq)
    y1, fin1, g1 = both(s0[used].contiguous(), ds[used].contiguous(), few, len(used))
    torch.cuda.synchronize()
    none = torch.ones(nseq, dtype=torch.bool)
    none[used] = False
    assert torch.equal(fin[none], s0[none]) and torch.equal(g["dinitial_states"][none], ds[none])
    near = lambda a, b: (a - b).norm() <= 1e-5 * b.norm()   # more segments, other chunks: sums in another order, 1e-6 or less
    assert near(y, y1) and near(fin[used], fin1) and near(g["dinitial_states"][used], g1["dinitial_states"])
    assert all(near(g[k], g1[k]) for k in ("dx", "ddt", "dA", "dB", "dC"))


def test_scan_without_tokens_hands_on_many_states():
    nseq, dim, N = 5000, 3, 4
    e = lambda *s: torch.empty(s, device="cuda")
    s0 = torch.randn(nseq, dim, N, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    _, fin = ssd.selective_scan_fwd(e(1, 0, dim), e(1, 0, dim), -torch.ones(dim, N, device="cuda"), e(1, 0, 1, N), e(1, 0, 1, N), initial_states=s0,
                                    seq_idx=ids, nseq=nseq)
    torch.cuda.synchronize()
    assert torch.equal(fin, s0)
