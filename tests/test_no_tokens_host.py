"""Workspace queries for a problem without tokens (seqlen 0) answer, for whole rows and for
packed streams (host code, CPU)."""
import ctypes
import os

import pytest

from ssd_chunked_scan_amd import ssd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        pytest.skip("libssd.so not built")
    return ssd.load_library()


@pytest.mark.parametrize("dtype", [ssd.DTYPE_F32, ssd.DTYPE_BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("nseq", [0, 3], ids=["rows", "packed"])
@pytest.mark.parametrize("heads", [(2, 1), (8, 8)], ids=["shared", "single"])
def test_workspace_queries(lib, dtype, nseq, heads):
    n = ctypes.c_size_t(7)
    a = ssd.FwdArgs(batch=1, seqlen=0, nheads=heads[0], headdim=32, dstate=48, ngroups=heads[1], chunk=64, dtype=dtype,
                    seq_idx=0x7000000000 if nseq else None, nseq=nseq)
    for query in (lib.ssd_fwd_workspace_size, lib.ssd_bwd_workspace_size):
        assert query(ctypes.byref(a), ctypes.byref(n)) == 0
    g = ssd.GdrArgs(batch=1, seqlen=0, nheads=heads[0], headdim=32, dstate=48, ngroups=heads[1], dtype=dtype,
                    seq_idx=0x7000000000 if nseq else None, nseq=nseq)
    for query in (lib.ssd_gdr_fwd_workspace_size, lib.ssd_gdr_bwd_workspace_size):
        assert query(ctypes.addressof(g), ctypes.addressof(n)) == 0
