"""Sizes past what the gated delta rule's entry points address are refused, before any
GPU work and for the workspace queries too (CPU)."""
import ctypes
import os

import pytest

from ssd_chunked_scan_amd import ssd
from test_delta_host import NULLP, OK, SHAPE, gdr, gdr_bwd, step


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        pytest.skip("libssd.so not built")
    return ssd.load_library()


PAST = [dict(nheads=1 << 17, headdim=64, ngroups=1),                    # H P = 2^23
        dict(nheads=1 << 17, headdim=16, dstate=64, ngroups=1 << 17),   # G N = 2^23
        dict(seqlen=(1 << 28) + 1, seq_idx=0x7000000000, nseq=3),
        dict(batch=1 << 30, nheads=4),                                  # chains of a grid
        dict(batch=1 << 20, seqlen=1 << 20)]                            # chunks


@pytest.mark.parametrize("kw", PAST, ids=str)
def test_past_the_limits(lib, kw):
    n = ctypes.c_size_t(7)
    a = gdr(**dict(kw))
    for f in (lib.ssd_gdr_fwd_workspace_size, lib.ssd_gdr_bwd_workspace_size):
        assert f(ctypes.addressof(a), ctypes.addressof(n)) == SHAPE
    assert lib.ssd_gdr_fwd(ctypes.addressof(a), None) == SHAPE
    assert lib.ssd_gdr_bwd(ctypes.addressof(a), ctypes.addressof(gdr_bwd()), None) == SHAPE


@pytest.mark.parametrize("kw", [dict(nheads=1 << 16, headdim=64, ngroups=1), dict(nheads=1 << 16, headdim=16, ngroups=1 << 16),
                                dict(seqlen=1 << 28, seq_idx=0x7000000000, nseq=3, ngroups=1), dict(nheads=1, ngroups=1, headdim=4096)],
                         ids=str)
def test_at_the_limits(lib, kw):
    n = ctypes.c_size_t()
    a = gdr(**dict(kw))
    for f in (lib.ssd_gdr_fwd_workspace_size, lib.ssd_gdr_bwd_workspace_size):
        assert f(ctypes.addressof(a), ctypes.addressof(n)) == OK and n.value > 0


def test_chunks_and_groups_past_the_gradient_kernel_s_grid(lib):
    n = ctypes.c_size_t()
    a = gdr(seqlen=1 << 28, seq_idx=0x7000000000, nseq=3, ngroups=2)
    assert lib.ssd_gdr_fwd_workspace_size(ctypes.addressof(a), ctypes.addressof(n)) == OK
    assert lib.ssd_gdr_bwd_workspace_size(ctypes.addressof(a), ctypes.addressof(n)) == SHAPE
    assert lib.ssd_gdr_bwd(ctypes.addressof(a), ctypes.addressof(gdr_bwd()), None) == SHAPE


def test_step_rows_past_a_grid(lib):
    assert lib.ssd_gdr_step(ctypes.addressof(step(batch=1 << 22, nheads=4)), None) == SHAPE
    # just below: the next check answers
    assert lib.ssd_gdr_step(ctypes.addressof(step(batch=(1 << 22) - 1, nheads=4, g=0)), None) == NULLP
