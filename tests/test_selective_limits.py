"""Which sizes and alignments the newer operators' entry points take: each direction of the selective scan by its own launches, single
tokens by their own strides, rows of the norm by their length (host only: what is taken ends at a missing pointer, an overlap or in the workspace's size)."""
import ctypes
import os

import pytest

from ssd_chunked_scan_amd import ssd

OK, NULLP, SHAPE = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        pytest.skip("libssd.so not built")
    return ssd.load_library()


def workspaces(lib, **kw):
    a = ssd.SelectiveScanArgs(**{**dict(batch=1, seqlen=100, dim=64, dstate=16, ngroups=1, dtype=1, dt_softplus=1), **kw})
    n = ctypes.c_size_t()
    return tuple(getattr(lib, f"ssd_selective_scan_{d}_workspace_size")(ctypes.addressof(a), ctypes.addressof(n)) for d in ("fwd", "bwd"))


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(batch=1 << 14, seqlen=1 << 12, dim=1 << 9), OK, OK), (dict(batch=1 << 14, seqlen=1 << 12, dim=1 << 11), OK, SHAPE),
    (dict(batch=1 << 11, seqlen=1 << 12, dim=1 << 11, dstate=32), OK, OK), (dict(batch=1 << 12, seqlen=1 << 12, dim=1 << 12, dstate=32), OK, SHAPE),
    (dict(batch=1 << 10, seqlen=1 << 12, dim=1 << 10, dstate=64), OK, OK), (dict(batch=1 << 10, seqlen=1 << 12, dim=1 << 12, dstate=64), OK, SHAPE),
    # the keys' gradients
    (dict(batch=1 << 9, seqlen=1 << 10, dim=256, ngroups=256), OK, SHAPE), (dict(batch=1 << 9, seqlen=1 << 9, dim=256, ngroups=256), OK, OK),
    (dict(batch=1 << 10, seqlen=1 << 20, dim=1 << 10), OK, SHAPE), (dict(batch=1 << 10, seqlen=1 << 20, dim=1 << 11), SHAPE, SHAPE),
    (dict(batch=1 << 20, seqlen=1, dim=1 << 13), SHAPE, SHAPE),   # the states
])
def test_each_direction_s_own_limits(lib, kw, fwd, bwd):
    assert workspaces(lib, **kw) == (fwd, bwd)


@pytest.mark.parametrize("name", ["x", "dt", "z", "B", "C"])
def test_single_tokens_of_long_rows(lib, name):
    """One token of every row of a [b,T,D] tensor: its stride is T * D."""
    def ask(stride):
        a = ssd.SelectiveScanStepArgs(batch=2, dim=64, dstate=16, ngroups=1, dtype=1, dt_softplus=1, **{name + "_stride": stride})
        return lib.ssd_selective_scan_step(ctypes.addressof(a), None)
    assert ask(1 << 22) == ask((1 << 22) + 64) == ask(1 << 36) == NULLP
    assert ask((1 << 36) + 1) == ask(15 if name in "BC" else 63) == ask(-1) == SHAPE


def test_norm_s_alignment(lib):
    """Rows of whole runs of 8 start at 16 bytes, others at an element; weights at 16 bytes."""
    at = {n: (i + 1) << 34 for i, n in enumerate(("x", "residual", "weight", "residual_out", "y", "q", "scales", "rstd"))}

    def ask(dim, **kw):
        a = ssd.RmsNormArgs(rows=100, dim=dim, dtype=1, residual_dtype=0, eps=1e-5, reserved=0, **{**at, **kw})
        a.residual_out = a.y   # past the alignment checks it ends here
        return lib.ssd_rms_norm_fwd(ctypes.addressof(a), None)
    MISAL, ALIAS = 8, 9
    for name, size in (("x", 2), ("residual", 4), ("q", 1)):
        assert ask(321, **{name: at[name] + size}) == ALIAS and ask(320, **{name: at[name] + size}) == MISAL
    assert ask(321, x=at["x"] + 1) == ask(321, residual=at["residual"] + 2) == ask(321, weight=at["weight"] + 4) == MISAL
