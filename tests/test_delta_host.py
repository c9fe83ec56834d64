"""Host-only checks of the gated delta rule's and layer norm's entry points: invalid
arguments give the documented status before any HIP call, and the binding refuses
what the library would misread (CPU, no GPU work)."""
import ctypes
import os

import pytest
import torch

from ssd_chunked_scan_amd import ssd

OK, NULLP, SHAPE, DTYPE, CHUNK, GROUPS, SEQ, WS, MISAL, ALIAS = range(10)
BASE = 0x10000000   # fake aligned addresses, 16 GiB apart: validation never reads them


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        pytest.skip("libssd.so not built")
    return ssd.load_library()


def fill(a, names, kw):
    for i, n in enumerate(names):
        setattr(a, n, kw.pop(n, BASE + (i << 34)))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


GDR_IN = ["q", "k", "v", "g", "beta", "initial_states"]


def gdr(**kw):
    d = dict(batch=1, seqlen=256, nheads=4, headdim=64, dstate=64, ngroups=2, dtype=1, scale=1.0)
    d.update({k: kw.pop(k) for k in list(kw) if k in d})
    a = ssd.GdrArgs(**d)
    kw.setdefault("workspace_bytes", 1 << 33)
    return fill(a, GDR_IN + ["y", "final_states", "workspace"], kw)


GDR_OUT = ["dy", "dfinal_states", "dq", "dk", "dv", "dg", "dbeta", "dinitial_states", "workspace"]


def gdr_bwd(**kw):
    kw.setdefault("workspace_bytes", 1 << 33)
    a = ssd.GdrBwdArgs()
    for i, n in enumerate(GDR_OUT):
        kw.setdefault(n, BASE + ((20 + i) << 34))
    return fill(a, GDR_OUT, kw)


SHARED = [
    (dict(dtype=7), DTYPE), (dict(nheads=6, ngroups=4), GROUPS), (dict(headdim=24), SHAPE), (dict(dstate=40), SHAPE),
    (dict(dstate=272), SHAPE), (dict(headdim=4112), SHAPE), (dict(batch=0), SHAPE), (dict(seqlen=-1), SHAPE),
    (dict(seqlen=1 << 31), SHAPE), (dict(nheads=0), SHAPE), (dict(ngroups=0), SHAPE),
    (dict(batch=2, seq_idx=0x7000000000, nseq=3), SEQ), (dict(seq_idx=0x7000000000, nseq=0), SEQ),
    (dict(q=0), NULLP), (dict(beta=0), NULLP), (dict(k=BASE + 8), MISAL), (dict(initial_states=BASE + 4), MISAL), (dict(beta=BASE + (4 << 34) + 1), MISAL),
    (dict(seq_idx=0x7000000004, nseq=2), MISAL),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(y=0), NULLP), (dict(workspace=0), NULLP), (dict(workspace_bytes=1000), WS),
    (dict(y=BASE + (2 << 34)), ALIAS),            # y over v
    (dict(final_states=BASE + (5 << 34)), ALIAS),  # final over initial states
    (dict(workspace=BASE), ALIAS),
])
def test_gdr_fwd_refuses(lib, kw, code):
    a = gdr(**kw)
    assert lib.ssd_gdr_fwd(ctypes.addressof(a), None) == code


@pytest.mark.parametrize("kw,code", SHARED)
def test_gdr_bwd_refuses_the_forward_s_arguments(lib, kw, code):
    a, g = gdr(**kw), gdr_bwd()
    assert lib.ssd_gdr_bwd(ctypes.addressof(a), ctypes.addressof(g), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), NULLP), (dict(dq=0), NULLP), (dict(dbeta=0), NULLP), (dict(workspace=0), NULLP),
    (dict(dv=BASE + (30 << 34) + 2), MISAL), (dict(workspace_bytes=1 << 16), WS),
    (dict(dv=BASE + (20 << 34)), ALIAS),   # dv over dy
    (dict(dk=BASE + (22 << 34)), ALIAS),   # dk over dq
    (dict(dq=BASE), ALIAS),                # dq over q
])
def test_gdr_bwd_refuses(lib, kw, code):
    a, g = gdr(), gdr_bwd(**kw)
    assert lib.ssd_gdr_bwd(ctypes.addressof(a), ctypes.addressof(g), None) == code


def test_gdr_workspaces(lib):
    n = ctypes.c_size_t()
    sizes = {}
    for fn in ("fwd", "bwd"):
        f = getattr(lib, f"ssd_gdr_{fn}_workspace_size")
        assert f(ctypes.addressof(gdr()), ctypes.addressof(n)) == OK
        sizes[fn] = n.value
        assert f(ctypes.addressof(gdr(dstate=40)), ctypes.addressof(n)) == SHAPE
        assert f(None, ctypes.addressof(n)) == NULLP
        assert f(ctypes.addressof(gdr()), None) == NULLP
        # packed: every one of 5 segments may add a chunk
        assert f(ctypes.addressof(gdr(seq_idx=0x7000000000, nseq=5)), ctypes.addressof(n)) == OK
        assert n.value > sizes[fn]
    assert sizes["bwd"] > sizes["fwd"] > 0
    assert lib.ssd_gdr_fwd(None, None) == NULLP
    assert lib.ssd_gdr_bwd(ctypes.addressof(gdr()), None, None) == NULLP


def step(**kw):
    d = dict(batch=2, nheads=4, headdim=64, dstate=64, ngroups=2, dtype=1, scale=1.0)
    d.update({k: kw.pop(k) for k in list(kw) if k in d})
    return fill(ssd.GdrStepArgs(**d), ["q", "k", "v", "g", "beta", "state", "y"], kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(nheads=3), GROUPS), (dict(headdim=8), SHAPE), (dict(dstate=512), SHAPE),
    (dict(batch=0), SHAPE), (dict(g=0), NULLP), (dict(state=0), NULLP), (dict(v=BASE + 6), MISAL),
    (dict(y=BASE + (2 << 34)), ALIAS), (dict(state=BASE), ALIAS), (dict(y=BASE + (5 << 34)), ALIAS),
])
def test_gdr_step_refuses(lib, kw, code):
    assert lib.ssd_gdr_step(ctypes.addressof(step(**kw)), None) == code


def test_null_args(lib):
    for f in (lib.ssd_gdr_step, lib.ssd_layer_norm_fwd, lib.ssd_layer_norm_bwd):
        assert f(None, None) == NULLP


def norm(**kw):
    d = dict(rows=10, dim=320, dtype=1, eps=1e-5)
    d.update({k: kw.pop(k) for k in list(kw) if k in d})
    return fill(ssd.NormArgs(**d), ["x", "weight", "bias", "y", "mean", "rstd"], kw)


def norm_bwd(**kw):
    d = dict(rows=10, dim=320, dtype=1, reserved=0)
    d.update({k: kw.pop(k) for k in list(kw) if k in d})
    kw.setdefault("workspace_bytes", 1 << 30)
    return fill(ssd.NormBwdArgs(**d), ["x", "dy", "mean", "rstd", "weight", "dx", "dweight", "dbias", "workspace"], kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(dim=0), SHAPE), (dict(dim=65537), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 30, dim=4096), SHAPE), (dict(x=0), NULLP), (dict(y=0), NULLP),
    (dict(weight=BASE + 4), MISAL), (dict(y=BASE + 16), ALIAS), (dict(mean=BASE + (1 << 34)), ALIAS),
    (dict(rstd=BASE + (4 << 34)), ALIAS),
])
def test_norm_fwd_refuses(lib, kw, code):
    assert lib.ssd_layer_norm_fwd(ctypes.addressof(norm(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(dim=0), SHAPE), (dict(dy=0), NULLP), (dict(mean=0), NULLP), (dict(dx=0), NULLP),
    (dict(workspace=0), NULLP), (dict(workspace_bytes=100), WS), (dict(dx=BASE + (5 << 34) + 8), MISAL),
    (dict(dx=BASE), ALIAS), (dict(dx=BASE + (1 << 34) + 64), ALIAS), (dict(dbias=BASE + (6 << 34)), ALIAS),
    (dict(workspace=BASE + (4 << 34)), ALIAS),
])
def test_norm_bwd_refuses(lib, kw, code):
    assert lib.ssd_layer_norm_bwd(ctypes.addressof(norm_bwd(**kw)), None) == code


def test_norm_workspace(lib):
    n = ctypes.c_size_t()
    f = lib.ssd_layer_norm_bwd_workspace_size
    assert f(ctypes.addressof(norm_bwd()), ctypes.addressof(n)) == OK
    assert n.value >= 2 * 320 * 4
    assert f(ctypes.addressof(norm_bwd(rows=0)), ctypes.addressof(n)) == OK and n.value == 0
    assert f(ctypes.addressof(norm_bwd(dim=70000)), ctypes.addressof(n)) == SHAPE


def test_the_binding_refuses_host_tensors_types_and_shapes():
    z = lambda *s: torch.zeros(s)
    with pytest.raises(ValueError, match="GPU"):
        ssd.gdr_fwd(z(1, 8, 1, 16), z(1, 8, 1, 16), z(1, 8, 2, 16), z(1, 8, 2), z(1, 8, 2))
    with pytest.raises(ValueError, match="v must be"):
        ssd.gdr_fwd(z(1, 8, 1, 16), z(1, 8, 1, 16), z(1, 8, 2), z(1, 8, 2), z(1, 8, 2))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssd.gdr_fwd(*(t.half() for t in (z(1, 8, 1, 16), z(1, 8, 1, 16), z(1, 8, 2, 16), z(1, 8, 2), z(1, 8, 2))))
    with pytest.raises(ValueError, match="GPU"):
        ssd.gdr_bwd(z(1, 8, 1, 16), z(1, 8, 1, 16), z(1, 8, 2, 16), z(1, 8, 2), z(1, 8, 2), z(1, 8, 2, 16))
    with pytest.raises(ValueError, match="q must be"):
        ssd.gdr_step(z(1, 1, 16, 1), z(1, 1, 16), z(1, 2, 16), z(1, 2), z(1, 2), z(1, 2, 16, 16))
    with pytest.raises(ValueError, match="GPU"):
        ssd.gdr_step(z(1, 1, 16), z(1, 1, 16), z(1, 2, 16), z(1, 2), z(1, 2), z(1, 2, 16, 16))
    with pytest.raises(ValueError, match="GPU"):
        ssd.layer_norm_fwd(z(4, 8))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssd.layer_norm_fwd(z(4, 8).double())
    with pytest.raises(ValueError, match="GPU"):
        ssd.layer_norm_bwd(z(4, 8), z(4, 8), z(4), z(4))


def test_packed_arguments_match_the_structures():
    """The binding packs its arguments into bytes: same size, same place of every field."""
    import struct
    for packer, mirror in ((ssd._GDR, ssd.GdrArgs), (ssd._GDR_BWD, ssd.GdrBwdArgs), (ssd._GDR_STEP, ssd.GdrStepArgs),
                           (ssd._NORM, ssd.NormArgs), (ssd._NORM_BWD, ssd.NormBwdArgs)):
        assert packer.size == ctypes.sizeof(mirror)
        n = len(mirror._fields_)
        vals = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(mirror._fields_)]
        a = mirror.from_buffer_copy(packer.pack(*vals))
        assert [getattr(a, f) for f, _ in mirror._fields_] == vals and n == len(struct.unpack(packer.format, bytes(a)))
