"""The gated delta rule where many chains run at once: workgroups that own 64 columns of a
chain, heads shared out over workgroups and added up again, long packed streams, calls
beside each other.  Inputs, measures and bars are test_gpu_gdr.py's."""
import numpy as np
import pytest
import torch

from oracle import delta
from ssd_chunked_scan_amd import ssd
from test_gpu_gdr import DV, STATE, TOL, check_fwd, draw, f64, gpu, spans, worst_states, worst_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def worst_slices(got, ref, x):
    """max over (row or segment, head or group) of the relative error over its tokens, a
    slice of fewer than 64 tokens held to the mean square per token of all such slices
    where that is larger.  A one-token gradient is one dot product: dg = e^g <D, S> sums
    P N terms d s, each off by 2^-8 of |d s| for the roundings of d and s, so its error is
    2^-8 (sum d^2 s^2)^(1/2) in norm, however far the sum itself cancels.  Short segments
    and their heads are drawn alike, and the mean square of such sums is the mean of
    sum d^2 s^2, products of different terms averaging to nothing.  (The whole tensor's
    average would be the wrong measure beside long segments: with carried states of 0.3 and
    dfinal_states of 0.3, D and S of a one-token segment are about 0.3 in every element, so
    dg is about 0.09 (P N)^(1/2), 5 at P = 48 and N = 64, against 0.2 for a token far from
    both ends.  Nor is one segment's average over its heads, where these are one or two.)"""
    norm = lambda a: np.linalg.norm(a, axis=(0,) if a.ndim == 2 else (0, 2))
    sl = [(hi - lo, norm(ref[r, lo:hi]), norm(got[r, lo:hi] - ref[r, lo:hi])) for r, lo, hi in spans(x)]
    short = [(t, n) for t, n, _ in sl if t < 64]
    rms = np.sqrt(sum((n ** 2).sum() for _, n in short) / max(1, sum(t * n.size for t, n in short)))
    return max((e / np.maximum(np.maximum(n, rms * np.sqrt(t) if t < 64 else 0), 1e-30)).max() for t, n, e in sl)


def check_bwd(x, dy, dfin, dtype, label=""):
    got = ssd.gdr_bwd(**gpu(x), dy=dy.cuda(), dfinal_states=None if dfin is None else dfin.cuda())
    torch.cuda.synchronize()
    ref = delta.gdr_backward(**x, dy=dy, dfinal_states=dfin)
    e = {n: worst_slices(f64(got[n]), ref[n], x) for n in ("dq", "dk", "dv", "dbeta", "dg")}
    e["dinit"] = worst_states(f64(got["dinitial_states"]), ref["dinitial_states"])
    print(f"[gdr bwd] {label} " + " ".join(f"{k}={v:.2e}" for k, v in e.items()), flush=True)
    for n, v in e.items():
        assert np.isfinite(f64(got[n if n != "dinit" else "dinitial_states"])).all(), n
        assert v <= (STATE if n == "dinit" else DV[dtype] if n == "dv" else TOL[dtype]), (n, v)


# more chains and column tiles than CUs, each state width, column tiles that are full, cut
# and padded, whole and cut last chunks, one and many heads of a group
SHAPES = [(3, 130, 96, 16, 48, 4), (2, 129, 130, 80, 64, 13), (5, 64, 64, 64, 128, 1), (4, 200, 72, 32, 112, 3),
          (1, 130, 264, 16, 256, 8), (2, 70, 66, 144, 208, 2), (300, 3, 1, 16, 16, 1)]
IDS = lambda s: "b%d_T%d_H%d_P%d_N%d_G%d" % s


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_many_chains(dtype, shape):
    b, T, H, P, N, G = shape
    x, dy, dfin = draw(sum(shape), b, T, H, P, N, G, dtype)
    check_fwd(x, dtype, str(shape))
    check_bwd(x, dy, dfin, dtype, str(shape))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [64, 128, 256])
def test_many_packed_chains(dtype, N):
    x, dy, dfin = draw(N, 1, 0, 60, 48, N, 3, dtype, lengths=[130, 0, 1, 64, 200])
    check_fwd(x, dtype, f"packed N={N}")
    check_bwd(x, dy, dfin, dtype, f"packed N={N}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_more_sequences_than_threads(dtype):
    lengths = np.random.default_rng(3).integers(0, 4, 1500).tolist()
    x, dy, dfin = draw(19, 1, 0, 2, 16, 16, 1, dtype, lengths=lengths)
    check_fwd(x, dtype, "1500 sequences")
    check_bwd(x, dy, dfin, dtype, "1500 sequences")


def test_a_long_packed_stream_is_its_sequences():
    """Each sequence by itself runs the same products in the same order: the same bits."""
    lengths = [60001, 3, 100000, 4097, 0, 64, 90000]
    x, dy, dfin = draw(20, 1, 0, 2, 16, 32, 1, "bf16", lengths=lengths)
    g, d, df = gpu(x), dy.cuda(), dfin.cuda()
    y, f = ssd.gdr_fwd(**g)
    gr = ssd.gdr_bwd(**g, dy=d, dfinal_states=df)
    lo = 0
    for i, n in enumerate(lengths):
        if n:
            one = {m: g[m][:, lo:lo + n].contiguous() for m in ("q", "k", "v", "g", "beta")}
            one |= dict(initial_states=g["initial_states"][i:i + 1].contiguous(), scale=x["scale"])
            y1, f1 = ssd.gdr_fwd(**one)
            assert torch.equal(y[:, lo:lo + n], y1) and torch.equal(f[i:i + 1], f1), i
            g1 = ssd.gdr_bwd(**one, dy=d[:, lo:lo + n].contiguous(), dfinal_states=df[i:i + 1].contiguous())
            for m in ("dv", "dg", "dbeta"):
                assert torch.equal(gr[m][:, lo:lo + n], g1[m]), (i, m)
            assert torch.equal(gr["dinitial_states"][i:i + 1], g1["dinitial_states"]), i
        else:
            assert torch.equal(f[i], g["initial_states"][i]) and torch.equal(gr["dinitial_states"][i], df[i])
        lo += n


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H", [4, 160], ids=["few", "many"])
def test_a_column_tile_s_results_do_not_depend_on_its_neighbours(dtype, H):
    """Head 0 of a problem, alone and among H heads of its group: y, the state and dv are
    held to the same reference."""
    x, dy, dfin = draw(21, 1, 150, H, 64, 64, 1, dtype)
    g = gpu(x)
    y, f = ssd.gdr_fwd(**g)
    gr = ssd.gdr_bwd(**g, dy=dy.cuda(), dfinal_states=dfin.cuda())
    one = {m: x[m] if m in "qk" else x[m][:, :, :1].contiguous() for m in ("q", "k", "v", "g", "beta")}
    one |= dict(initial_states=x["initial_states"][:, :1].contiguous(), scale=x["scale"], seq_idx=None, nseq=None)
    yr, fr = delta.gdr_forward(**one)
    ref = delta.gdr_backward(**one, dy=dy[:, :, :1], dfinal_states=dfin[:, :1])
    torch.cuda.synchronize()
    assert worst_tokens(f64(y)[:, :, :1], yr, one) <= TOL[dtype]
    assert worst_states(f64(f)[:, :1], fr) <= 1e-4
    assert worst_tokens(f64(gr["dg"])[:, :, :1], ref["dg"], one) <= TOL[dtype]
    assert worst_tokens(f64(gr["dv"])[:, :, :1], ref["dv"], one) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cuts", [[37], [0], [63, 64, 65], [99]], ids=str)
def test_gradients_of_gates_that_reset_the_state(dtype, cuts):
    """g = -inf drops the state, and dg of such a token is 0: in the kernels a difference of
    fp32 sums of up to 64 x 64 terms, held to 1e-4 of dg's norm (2^-24 of each term; all
    errors of one sign would be 2.4e-4 of the terms' mean size)."""
    x, dy, dfin = draw(22, 1, 100, 2, 32, 64, 1, dtype)
    x["g"][:, cuts] = -float("inf")
    check_bwd(x, dy, dfin, dtype, f"reset at {cuts}")
    dg = ssd.gdr_bwd(**gpu(x), dy=dy.cuda(), dfinal_states=dfin.cuda())["dg"]
    torch.cuda.synchronize()
    assert dg[:, cuts].float().norm() <= 1e-4 * dg.float().norm()


def test_two_streams_at_once():
    """Two problems in flight beside each other, workspaces of their own."""
    probs = [draw(23 + i, 4, 600, 16, 64, 64, 2, "bf16") for i in range(2)]
    gs = [(gpu(x), dy.cuda()) for x, dy, _ in probs]
    want = [(ssd.gdr_fwd(**g)[0], ssd.gdr_bwd(**g, dy=d)) for g, d in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    got = [[], []]
    for _ in range(3):
        for i, (g, d) in enumerate(gs):
            with torch.cuda.stream(streams[i]):
                got[i].append((ssd.gdr_fwd(**g)[0], ssd.gdr_bwd(**g, dy=d)))
    torch.cuda.synchronize()
    for i in range(2):
        for y, gr in got[i]:
            assert torch.equal(y, want[i][0]) and all(torch.equal(gr[n], want[i][1][n]) for n in gr)


def test_nothing_is_written_outside_the_outputs():
    """Outputs with room before and behind them: the room keeps its bytes."""
    x, dy, dfin = draw(25, 1, 0, 3, 16, 48, 1, "bf16", lengths=[70, 0, 33])
    g = gpu(x)

    def inside(t):
        """A tensor like t in a larger buffer, and the buffer."""
        n, pad = t.numel() * t.element_size(), 4096
        buf = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf[pad:pad + n].view(t.dtype).view(t.shape), buf

    y0, f0 = ssd.gdr_fwd(**g)
    (y, by), (f, bf) = inside(y0), inside(f0)
    ws, bw = inside(torch.empty(ssd.gdr_fwd_workspace_bytes(*(g[n] for n in ("q", "k", "v", "g", "beta")), g["seq_idx"], 3),
                                dtype=torch.uint8))
    ssd.gdr_fwd(**g, y=y, final_states=f, workspace=ws)
    want = ssd.gdr_bwd(**g, dy=dy.cuda(), dfinal_states=dfin.cuda())
    outs = {n: inside(t) for n, t in want.items()}
    wsb, bwb = inside(torch.empty(ssd.gdr_bwd_workspace_bytes(*(g[n] for n in ("q", "k", "v", "g", "beta")), g["seq_idx"], 3),
                                  dtype=torch.uint8))
    ssd.gdr_bwd(**g, dy=dy.cuda(), dfinal_states=dfin.cuda(), grads={n: t for n, (t, _) in outs.items()}, workspace=wsb)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(f, f0)
    assert all(torch.equal(outs[n][0], want[n]) for n in want)
    for buf in (by, bf, bw, bwb, *(b for _, b in outs.values())):
        assert (buf[:4096] == 0xA5).all() and (buf[-4096:] == 0xA5).all()
