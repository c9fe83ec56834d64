"""Host-only checks of the selective scan's, the convolution's, RMS norm's and the 8-bit product's entry points:
invalid arguments give the documented status before any HIP call, and the binding refuses what the library would
misread (CPU, no GPU work)."""
import ctypes
import os

import pytest
import torch

from ssd_chunked_scan_amd import ssd

OK, NULLP, SHAPE, DTYPE, CHUNK, GROUPS, SEQ, WS, MISAL, ALIAS = range(10)
BASE = 0x10000000   # fake aligned addresses, 16 GiB apart: validation never reads them
IDS = 0x7000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        pytest.skip("libssd.so not built")
    return ssd.load_library()


def made(cls, sizes, names, kw, first=0):
    """`cls` with these sizes, fake addresses for `names`, and what `kw` says instead."""
    a = cls(**{k: kw.pop(k, v) for k, v in sizes.items()})
    for i, n in enumerate(names):
        setattr(a, n, kw.pop(n, BASE + ((first + i) << 34)))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


SCAN = ["x", "dt", "A", "B", "C", "D", "dt_bias", "z", "initial_states", "y", "final_states", "workspace"]
SCAN_OUT = ["dy", "dfinal_states", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dz", "dinitial_states", "workspace"]


def scan(**kw):
    kw.setdefault("workspace_bytes", 1 << 34)
    return made(ssd.SelectiveScanArgs, dict(batch=1, seqlen=2000, dim=128, dstate=16, ngroups=2, dtype=1, dt_softplus=1), SCAN, kw)


def scan_bwd(**kw):
    kw.setdefault("workspace_bytes", 1 << 34)
    return made(ssd.SelectiveScanBwdArgs, {}, SCAN_OUT, kw, 20)


def at(name, off=0, names=SCAN, first=0):
    return BASE + ((first + names.index(name)) << 34) + off


SCAN_SHARED = [
    (dict(dtype=5), DTYPE), (dict(ngroups=3), GROUPS), (dict(batch=0), SHAPE), (dict(seqlen=-1), SHAPE), (dict(dim=0), SHAPE),
    (dict(dim=(1 << 20) + 2), SHAPE), (dict(dstate=0), SHAPE), (dict(dstate=65), SHAPE), (dict(ngroups=0), SHAPE),
    (dict(batch=1 << 16, seqlen=1 << 15), SHAPE), (dict(seqlen=1 << 31), SHAPE), (dict(seqlen=1 << 30, dim=1 << 20), SHAPE),
    (dict(x_stride=127), SHAPE), (dict(z_stride=-1), SHAPE), (dict(B_stride=31), SHAPE), (dict(C_stride=(1 << 22) + 1), SHAPE),
    (dict(batch=2, seq_idx=IDS, nseq=2), SEQ), (dict(seq_idx=IDS, nseq=0), SEQ), (dict(seq_idx=IDS, nseq=2, seqlen=(1 << 28) + 1, dim=2), SHAPE),
    (dict(x=0), NULLP), (dict(dt=0), NULLP), (dict(A=0), NULLP), (dict(B=0), NULLP), (dict(C=0), NULLP),
    (dict(x=at("x", 1)), MISAL), (dict(A=at("A", 2)), MISAL), (dict(dt_bias=at("dt_bias", 2)), MISAL), (dict(seq_idx=IDS + 2, nseq=2), MISAL),
    (dict(z=at("z", 1)), MISAL), (dict(initial_states=at("initial_states", 1)), MISAL),
]


@pytest.mark.parametrize("kw,code", SCAN_SHARED + [
    (dict(y=0), NULLP), (dict(y=at("y", 1)), MISAL), (dict(workspace=0), NULLP), (dict(workspace_bytes=1000), WS), (dict(workspace=at("workspace", 8)), MISAL),
    (dict(y=at("x")), ALIAS), (dict(y=at("z", 512000 - 2)), ALIAS), (dict(final_states=at("initial_states")), ALIAS), (dict(workspace=at("y")), ALIAS),
    (dict(x_stride=1024, y=at("x", 2 * 1024 * 1999 + 254)), ALIAS),
])
def test_scan_fwd_refuses(lib, kw, code):
    assert lib.ssd_selective_scan_fwd(ctypes.addressof(scan(**kw)), None) == code


@pytest.mark.parametrize("kw,code", SCAN_SHARED)
def test_scan_bwd_refuses_the_forward_s_arguments(lib, kw, code):
    assert lib.ssd_selective_scan_bwd(ctypes.addressof(scan(**kw)), ctypes.addressof(scan_bwd()), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), NULLP), (dict(dx=0), NULLP), (dict(ddt=0), NULLP), (dict(dA=0), NULLP), (dict(dB=0), NULLP), (dict(dC=0), NULLP),
    (dict(dz=0), NULLP), (dict(workspace=0), NULLP), (dict(workspace_bytes=1 << 16), WS), (dict(dx=at("dx", 1, SCAN_OUT, 20)), MISAL),
    (dict(dA=at("dA", 2, SCAN_OUT, 20)), MISAL), (dict(workspace=at("workspace", 4, SCAN_OUT, 20)), MISAL),
    (dict(dx=at("dy", 0, SCAN_OUT, 20)), ALIAS), (dict(dC=at("dB", 0, SCAN_OUT, 20)), ALIAS), (dict(dz=at("z")), ALIAS),
    (dict(dinitial_states=at("dfinal_states", 0, SCAN_OUT, 20)), ALIAS),
])
def test_scan_bwd_refuses(lib, kw, code):
    assert lib.ssd_selective_scan_bwd(ctypes.addressof(scan()), ctypes.addressof(scan_bwd(**kw)), None) == code


def test_scan_workspaces_and_nulls(lib):
    n = ctypes.c_size_t()
    p = ctypes.addressof(n)
    for d in ("fwd", "bwd"):
        f = getattr(lib, f"ssd_selective_scan_{d}_workspace_size")
        assert f(ctypes.addressof(scan()), p) == OK and n.value > 0
        assert f(ctypes.addressof(scan(dstate=99)), p) == SHAPE
        assert f(ctypes.addressof(scan()), None) == NULLP and f(None, p) == NULLP
        for T in (0, 1):   # nothing to divide by
            for kw in ({}, dict(seq_idx=IDS, nseq=3)):
                assert f(ctypes.addressof(scan(seqlen=T, **kw)), p) == OK
    assert lib.ssd_selective_scan_fwd(None, None) == NULLP and lib.ssd_selective_scan_step(None, None) == NULLP
    assert lib.ssd_selective_scan_bwd(ctypes.addressof(scan()), None, None) == NULLP
    # rows enough to fill the card take no chunks and no workspace
    assert lib.ssd_selective_scan_fwd_workspace_size(ctypes.addressof(scan(batch=64, dim=4096)), p) == OK and n.value == 0


STEP = ["x", "dt", "A", "B", "C", "D", "dt_bias", "z", "state", "y"]


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(ngroups=3), GROUPS), (dict(batch=0), SHAPE), (dict(batch=1 << 30), SHAPE), (dict(dstate=70), SHAPE),
    (dict(x_stride=5), SHAPE), (dict(x=0), NULLP), (dict(A=0), NULLP), (dict(state=0), NULLP), (dict(y=0), NULLP),
    (dict(B=at("B", 1, STEP)), MISAL), (dict(state=at("state", 2, STEP)), MISAL), (dict(y=at("x", 0, STEP)), ALIAS),
    (dict(state=at("A", 0, STEP)), ALIAS), (dict(y=at("state", 0, STEP)), ALIAS),
])
def test_scan_step_refuses(lib, kw, code):
    a = made(ssd.SelectiveScanStepArgs, dict(batch=2, dim=128, dstate=16, ngroups=2, dtype=1, dt_softplus=1), STEP, kw)
    assert lib.ssd_selective_scan_step(ctypes.addressof(a), None) == code


CONV = ["x", "weight", "bias", "initial_window", "y", "final_window"]
CONV_OUT = ["dy", "dfinal_window", "dx", "dweight", "dbias", "dinitial_window", "workspace"]


def conv(**kw):
    return made(ssd.CausalConvArgs, dict(batch=1, seqlen=200, dim=64, width=4, dtype=1, silu=1), CONV, kw)


def conv_bwd(**kw):
    kw.setdefault("workspace_bytes", 1 << 30)
    return made(ssd.CausalConvBwdArgs, {}, CONV_OUT, kw, 20)


CONV_SHARED = [
    (dict(dtype=3), DTYPE), (dict(width=0), SHAPE), (dict(width=5), SHAPE), (dict(dim=0), SHAPE), (dict(dim=(1 << 22) + 1), SHAPE),
    (dict(batch=0), SHAPE), (dict(seqlen=-1), SHAPE), (dict(x_stride=63), SHAPE), (dict(x_stride=1 << 31), SHAPE),
    (dict(batch=1 << 16, seqlen=1 << 15), SHAPE), (dict(seqlen=1 << 30, dim=1 << 22), SHAPE), (dict(batch=2, seq_idx=IDS, nseq=2), SEQ),
    (dict(seq_idx=IDS, nseq=0), SEQ), (dict(seq_idx=IDS, nseq=1 << 30, dim=1 << 22), SHAPE), (dict(x=0), NULLP), (dict(weight=0), NULLP),
    (dict(x=at("x", 1, CONV)), MISAL), (dict(weight=at("weight", 2, CONV)), MISAL), (dict(bias=at("bias", 1, CONV)), MISAL),
    (dict(initial_window=at("initial_window", 1, CONV)), MISAL), (dict(seq_idx=IDS + 1, nseq=2), MISAL),
]


@pytest.mark.parametrize("kw,code", CONV_SHARED + [
    (dict(y=0), NULLP), (dict(y=at("y", 1, CONV)), MISAL), (dict(y=at("x", 0, CONV)), ALIAS), (dict(final_window=at("initial_window", 0, CONV)), ALIAS),
    (dict(final_window=at("y", 100, CONV)), ALIAS),
])
def test_conv_fwd_refuses(lib, kw, code):
    assert lib.ssd_causal_conv_fwd(ctypes.addressof(conv(**kw)), None) == code


@pytest.mark.parametrize("kw,code", CONV_SHARED)
def test_conv_bwd_refuses_the_forward_s_arguments(lib, kw, code):
    assert lib.ssd_causal_conv_bwd(ctypes.addressof(conv(**kw)), ctypes.addressof(conv_bwd()), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), NULLP), (dict(dx=0), NULLP), (dict(dweight=0), NULLP), (dict(workspace=0), NULLP), (dict(workspace_bytes=64), WS),
    (dict(dx=at("dx", 1, CONV_OUT, 20)), MISAL), (dict(dx=at("dy", 0, CONV_OUT, 20)), ALIAS), (dict(dweight=at("weight", 0, CONV)), ALIAS),
    (dict(workspace=at("dx", 0, CONV_OUT, 20)), ALIAS),
])
def test_conv_bwd_refuses(lib, kw, code):
    assert lib.ssd_causal_conv_bwd(ctypes.addressof(conv()), ctypes.addressof(conv_bwd(**kw)), None) == code


def test_conv_workspace_and_nulls(lib):
    n = ctypes.c_size_t()
    p = ctypes.addressof(n)
    assert lib.ssd_causal_conv_bwd_workspace_size(ctypes.addressof(conv()), p) == OK and n.value > 0
    assert lib.ssd_causal_conv_bwd_workspace_size(ctypes.addressof(conv(seqlen=0)), p) == OK and n.value == 0
    assert lib.ssd_causal_conv_bwd_workspace_size(None, p) == NULLP
    assert lib.ssd_causal_conv_bwd_workspace_size(ctypes.addressof(conv()), None) == NULLP
    assert lib.ssd_causal_conv_bwd(ctypes.addressof(conv()), None, None) == NULLP
    assert lib.ssd_causal_conv_fwd(None, None) == NULLP and lib.ssd_causal_conv_step(None, None) == NULLP


CSTEP = ["x", "weight", "bias", "window", "y"]


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(width=5), SHAPE), (dict(batch=0), SHAPE), (dict(batch=1 << 33), SHAPE), (dict(x_stride=3), SHAPE),
    (dict(x=0), NULLP), (dict(window=0), NULLP), (dict(y=0), NULLP), (dict(window=at("window", 1, CSTEP)), MISAL),
    (dict(y=at("x", 0, CSTEP)), ALIAS), (dict(window=at("x", 0, CSTEP)), ALIAS),
])
def test_conv_step_refuses(lib, kw, code):
    a = made(ssd.CausalConvStepArgs, dict(batch=2, dim=64, width=4, dtype=1, silu=1), CSTEP, kw)
    assert lib.ssd_causal_conv_step(ctypes.addressof(a), None) == code


RMS = ["x", "residual", "weight", "residual_out", "y", "q", "scales", "rstd"]
RMS_BWD = ["r", "dy", "dresidual_out", "rstd", "weight", "dx", "dresidual", "dweight", "workspace"]


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), DTYPE), (dict(residual_dtype=9), DTYPE), (dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dim=65537), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 30, dim=2048), SHAPE), (dict(x=0), NULLP), (dict(y=0, q=0), NULLP), (dict(residual_out=0), NULLP),
    (dict(residual=0), NULLP), (dict(scales=0), NULLP), (dict(x=at("x", 8, RMS)), MISAL), (dict(weight=at("weight", 4, RMS)), MISAL),
    (dict(q=at("q", 8, RMS)), MISAL), (dict(scales=at("scales", 2, RMS)), MISAL), (dict(rstd=at("rstd", 1, RMS)), MISAL),
    (dict(y=at("residual", 0, RMS)), ALIAS), (dict(residual_out=at("residual", 16, RMS)), ALIAS), (dict(q=at("x", 0, RMS)), ALIAS),
    (dict(y=at("residual_out", 0, RMS)), ALIAS), (dict(residual_out=at("x", 0, RMS)), ALIAS),   # of another type
    (dict(scales=at("weight", 0, RMS)), ALIAS),
])
def test_rms_fwd_refuses(lib, kw, code):
    a = made(ssd.RmsNormArgs, dict(rows=100, dim=320, dtype=1, residual_dtype=0, eps=1e-5, reserved=0), RMS, kw)
    assert lib.ssd_rms_norm_fwd(ctypes.addressof(a), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), DTYPE), (dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(r=0), NULLP), (dict(dy=0), NULLP), (dict(rstd=0), NULLP),
    (dict(dx=0), NULLP), (dict(workspace=0), NULLP), (dict(workspace_bytes=100), WS), (dict(dy=at("dy", 4, RMS_BWD)), MISAL),
    (dict(dweight=at("dweight", 4, RMS_BWD)), MISAL), (dict(dx=at("r", 0, RMS_BWD)), ALIAS), (dict(dx=at("dy", 16, RMS_BWD)), ALIAS),
    (dict(dresidual=at("dx", 0, RMS_BWD)), ALIAS), (dict(dresidual=at("r", 0, RMS_BWD)), ALIAS), (dict(dweight=at("weight", 0, RMS_BWD)), ALIAS),
])
def test_rms_bwd_refuses(lib, kw, code):
    kw.setdefault("workspace_bytes", 1 << 30)
    a = made(ssd.RmsNormBwdArgs, dict(rows=100, dim=320, dtype=1, residual_dtype=0), RMS_BWD, kw)
    assert lib.ssd_rms_norm_bwd(ctypes.addressof(a), None) == code


def test_rms_workspace_and_nulls(lib):
    n = ctypes.c_size_t()
    a = made(ssd.RmsNormBwdArgs, dict(rows=100, dim=320, dtype=1, residual_dtype=0), RMS_BWD, {})
    assert lib.ssd_rms_norm_bwd_workspace_size(ctypes.addressof(a), ctypes.addressof(n)) == OK and n.value > 0
    a.rows = 0
    assert lib.ssd_rms_norm_bwd_workspace_size(ctypes.addressof(a), ctypes.addressof(n)) == OK and n.value == 0
    assert lib.ssd_rms_norm_fwd(None, None) == NULLP and lib.ssd_rms_norm_bwd(None, None) == NULLP


MM = ["a", "a_scales", "w", "w_scales", "bias", "out", "workspace"]


def mm(**kw):
    kw.setdefault("workspace_bytes", 1 << 33)
    return made(ssd.MatmulFp8Args, dict(m=20, n=300, k=1024, dtype=1, reserved=0), MM, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(m=-1), SHAPE), (dict(n=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=24), SHAPE), (dict(k=(1 << 22) + 16), SHAPE),
    (dict(m=1 << 31), SHAPE), (dict(m=1 << 21, n=1 << 21), SHAPE), (dict(a=0), NULLP), (dict(a_scales=0), NULLP), (dict(w=0), NULLP),
    (dict(w_scales=0), NULLP), (dict(out=0), NULLP), (dict(workspace=0), NULLP), (dict(workspace_bytes=8), WS), (dict(a=at("a", 8, MM)), MISAL),
    (dict(out=at("out", 4, MM)), MISAL), (dict(bias=at("bias", 2, MM)), MISAL), (dict(out=at("a", 0, MM)), ALIAS), (dict(workspace=at("out", 0, MM)), ALIAS),
])
def test_product_refuses(lib, kw, code):
    assert lib.ssd_matmul_fp8(ctypes.addressof(mm(**kw)), None) == code


def test_product_workspace_and_nothing_to_do(lib):
    n = ctypes.c_size_t()
    p = ctypes.addressof(n)
    assert lib.ssd_matmul_fp8_workspace_size(ctypes.addressof(mm()), p) == OK and n.value > 0
    for kw in (dict(m=0), dict(n=0), dict(m=0, n=0)):   # no tiles to divide by
        assert lib.ssd_matmul_fp8_workspace_size(ctypes.addressof(mm(**kw)), p) == OK and n.value == 0
        assert lib.ssd_matmul_fp8(ctypes.addressof(mm(**kw)), None) == OK
    assert lib.ssd_matmul_fp8(None, None) == NULLP and lib.ssd_matmul_fp8_workspace_size(ctypes.addressof(mm()), None) == NULLP


@pytest.mark.parametrize("packed,cls", [
    (ssd._SCAN, ssd.SelectiveScanArgs), (ssd._SCAN_BWD, ssd.SelectiveScanBwdArgs), (ssd._SCAN_STEP, ssd.SelectiveScanStepArgs),
    (ssd._CCONV, ssd.CausalConvArgs), (ssd._CCONV_BWD, ssd.CausalConvBwdArgs), (ssd._CCONV_STEP, ssd.CausalConvStepArgs),
    (ssd._RMS, ssd.RmsNormArgs), (ssd._RMS_BWD, ssd.RmsNormBwdArgs), (ssd._MM, ssd.MatmulFp8Args)])
def test_packed_bytes_match_the_structures(packed, cls):
    assert packed.size == ctypes.sizeof(cls)


def test_token_strides():
    """What may be columns of wider rows, and what is refused (CPU tensors: only the layout is looked at)."""
    dev = torch.device("cpu")
    ask = lambda t, lead, shape=None: ssd._token_stride(t, "t", t.dtype, t.shape if shape is None else shape, dev, lead)
    w = torch.zeros(2, 5, 40)
    assert ask(w, 2) == 0 and ask(w[..., 3:20], 2) == 40 and ask(w[:, 0, 3:20], 1) == 200 and ask(w[:1, :1, 3:20], 2) == 0
    assert ask(w[:, :1, 4:8], 2) == 200 and ask(w[..., 4:28].unflatten(-1, (3, 8)), 2) == 40
    for bad in (w[:, :3, :7], w[..., ::2], w.transpose(0, 1), w[..., :24].unflatten(-1, (3, 8)).transpose(2, 3), w[:, :1].expand(2, 5, 40)):
        with pytest.raises(ValueError):
            ask(bad, 2)
    with pytest.raises(TypeError):
        ssd._token_stride(w, "t", torch.bfloat16, w.shape, dev, 2)
    with pytest.raises(ValueError):
        ask(w, 2, (2, 5, 41))


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    k = torch.zeros(1, 4, 1, 16)
    A = torch.zeros(8, 16)
    with pytest.raises(ValueError):
        ssd.selective_scan_fwd(x, x, A, k, k)
    with pytest.raises(ValueError):
        ssd.causal_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        ssd.rms_norm_fwd(x)
    with pytest.raises(TypeError):
        ssd.matmul_fp8(x, x, x, x)
