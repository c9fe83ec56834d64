"""bf16 problems of the gated delta rule are as exact as one rounding of their outputs,
with random keys and with keys that resemble each other.

With similar keys, beta near 1 and weak decay, what a token adds to y is mostly taken
back by the next one: sums of terms several times as large as y cancel.  An operand
rounded once to 8 bits then shows in y as several roundings of y itself.

The bar, per (batch row, head): an output computed as ref + d and rounded to the nearest
is off by at most |bf16(ref) - ref| + 2 |d| in every element (the nearest number to
ref + d is at most as far from it as bf16(ref) is).  The first part is known from the
reference.  d: every operand of a product is exact or the sum of two bf16 numbers, off
by 2^-16 of itself at most, and a product drops that of the two small parts, 2^-16: three
such errors, which add in norm, of terms up to 5 times the sum: 5 * 3 * 2^-16 < 2^-12.
"""
import numpy as np
import pytest
import torch

from oracle import delta
from ssd_chunked_scan_amd import ssd
from test_gpu_gdr import f64, gpu, spans

pytestmark = pytest.mark.gpu

EXACT = 2.0 ** -12   # |d| / |ref|


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()
    torch.cuda.set_device(0)


def alike(seed, b, T, H, P, N, G, cos, beta, gate, init, lengths=None):
    """bf16 inputs whose keys and queries have cosines of about `cos` with each other."""
    rng = np.random.default_rng(seed)
    nseq = None
    if lengths is not None:
        b, T, nseq = 1, sum(lengths), len(lengths)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)
    axis = unit(rng.standard_normal((b, 1, G, N)))
    key = lambda: t(unit(cos ** 0.5 * axis + (1 - cos) ** 0.5 * unit(rng.standard_normal((b, T, G, N))))).bfloat16()
    n = nseq or b
    x = dict(q=key(), k=key(), v=t(rng.standard_normal((b, T, H, P))).bfloat16(),
             g=t(np.full((b, T, H), gate) if gate is not None else -0.3 * rng.uniform(0, 1, (b, T, H))).bfloat16(),
             beta=t(np.full((b, T, H), beta) if beta is not None else rng.uniform(0, 1, (b, T, H))).bfloat16(),
             initial_states=t(0.3 * rng.standard_normal((n, H, P, N))) if init else None,
             seq_idx=None if lengths is None else torch.from_numpy(np.repeat(np.arange(nseq), lengths).astype(np.int32)),
             nseq=nseq, scale=N ** -0.5)
    dy = t(rng.standard_normal((b, T, H, P))).bfloat16()
    dfin = t(0.3 * rng.standard_normal((n, H, P, N))) if init else None
    return x, dy, dfin


def worst(got, ref, x):
    """max over (row or segment, head) of |got - ref| over its bar."""
    once = f64(torch.from_numpy(ref).bfloat16()) - ref
    axes = (0,) if ref.ndim == 3 else (0, 2)
    norm = lambda a, s: np.sqrt((a[s[0], s[1]:s[2]] ** 2).sum(axes))
    return max((norm(got - ref, s) / (norm(once, s) + 2 * EXACT * norm(ref, s))).max() for s in spans(x))


KEYS = {"random": dict(cos=0.0, beta=None, gate=None, init=True), "alike": dict(cos=0.9, beta=1.0, gate=-0.01, init=True),
        "alike_no_decay": dict(cos=0.9, beta=1.0, gate=0.0, init=False), "alike_gated": dict(cos=0.9, beta=None, gate=-0.01, init=True)}
# every state width, chains of 16 columns per workgroup and (the last three) of 64
SHAPES = [(1, 200, 4, 64, 64, 2), (2, 130, 2, 48, 128, 1), (1, 257, 2, 64, 256, 1), (2, 130, 104, 64, 64, 4),
          (2, 130, 100, 64, 128, 2), (2, 70, 100, 32, 256, 1)]
IDS = lambda s: "b%d_T%d_H%d_P%d_N%d_G%d" % s


@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_y_is_off_by_one_rounding(shape, keys):
    x, _, _ = alike(sum(shape), *shape, **KEYS[keys])
    y, _ = ssd.gdr_fwd(**gpu(x))
    torch.cuda.synchronize()
    e = worst(f64(y), delta.gdr_forward(**x)[0], x)
    print(f"[gdr rounding] y {keys} {shape} {e:.3f}", flush=True)
    assert e <= 1


GRADS = ("dq", "dk", "dv", "dbeta", "dg")


def worst_gradients(got, ref, x):
    e = {n: worst(f64(got[n]), ref[n], x) for n in GRADS}
    e["dinitial_states"] = max(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-30)
                               for a, b in zip(f64(got["dinitial_states"]), ref["dinitial_states"])) / 1e-4
    return e


@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gradients_are_off_by_one_rounding(shape, keys):
    """(dinitial_states, fp32: the bar of test_gpu_gdr.py.)"""
    x, dy, dfin = alike(sum(shape) + 1, *shape, **KEYS[keys])
    got = ssd.gdr_bwd(**gpu(x), dy=dy.cuda(), dfinal_states=None if dfin is None else dfin.cuda())
    torch.cuda.synchronize()
    e = worst_gradients(got, delta.gdr_backward(**x, dy=dy, dfinal_states=dfin), x)
    print(f"[gdr rounding] {keys} {shape} " + " ".join(f"{n}={v:.3f}" for n, v in e.items()), flush=True)
    assert max(e.values()) <= 1, e
