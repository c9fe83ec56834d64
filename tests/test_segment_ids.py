"""The index arithmetic that packed streams' ids go through (``csrc/segment_ids.hpp``), compiled for the host with traps
on signed overflow: whatever 32-bit ids a stream holds, every index stays in range, and non-decreasing ids in
[0, nseq) give every segment its first token."""
import shutil
import subprocess

import numpy as np
import pytest

from conftest import ROOT

LEAST, MOST = -2 ** 31, 2 ** 31 - 1
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "segment_ids.hpp"
// stdin: T nseq ids...; stdout: the starts as the device fills them (-7: never written), then every segment's first token by a
// search, or "out" if an index leaves [0, nseq].
int main()
{
    int T, nseq;
    while (scanf("%d %d", &T, &nseq) == 2) {
        std::vector<int> id(T), start(nseq + 1, -7);
        for (int &v : id) if (scanf("%d", &v) != 1) return 1;
        bool out = false;
        auto put = [&](int i, int t) { if (i < 0 || i > nseq) out = true; else start[i] = t; };
        for (int t = 0; t < T; ++t) {
            const ssd::Segments here = ssd::segments_through(t ? id[t - 1] : -1, id[t], nseq);
            if ((long long)here.to - here.from > nseq) out = true;
            else for (int i = here.from; i < here.to; ++i) put(i, t);
            if (t == T - 1) for (int i = here.to; i <= nseq; ++i) put(i, T);
        }
        std::vector<int> first;
        for (int q = 0; q < nseq; ++q) first.push_back(ssd::first_from(id.data(), T, q));
        if (out) printf("out\n");
        else { for (int v : start) printf("%d ", v); for (int v : first) printf("%d ", v); printf("\n"); }
    }
}
"""


@pytest.fixture(scope="module")
def starts(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("ids")
    (at / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", f"{ROOT}/ssd_chunked_scan_amd/csrc", str(at / "p.cpp"), "-o", str(at / "p")], check=True)

    def run(streams):
        text = "\n".join(" ".join(map(str, [len(ids), nseq, *ids])) for ids, nseq in streams)
        res = subprocess.run([str(at / "p")], input=text, capture_output=True, text=True)
        assert res.returncode == 0, res.returncode   # a trap is a signal
        return [l if l == "out" else [int(v) for v in l.split()] for l in res.stdout.splitlines()]
    return run


def test_any_ids_stay_in_range(starts):
    rng = np.random.default_rng(0)
    edge = [LEAST, LEAST + 1, -2, -1, 0, 1, 2, 3, 4, 5, MOST - 1, MOST]
    streams = [([a, b, c], n) for a in edge for b in edge for c in edge for n in (1, 4)]
    streams += [([MOST], 1), ([LEAST], 3), ([0, 1, MOST, MOST], 2), ([0, 0, 2, MOST, MOST, 1], 3)]
    streams += [([int(v) for v in rng.choice(edge, 40)], 4) for _ in range(200)]
    got = starts(streams)
    assert len(got) == len(streams)
    for (ids, nseq), s in zip(streams, got):
        assert s != "out" and all(v == -7 or 0 <= v <= len(ids) for v in s), (ids, nseq, s)
        assert len(s) == 2 * nseq + 1 and -7 not in s[nseq + 1:]


def test_valid_streams(starts):
    rng = np.random.default_rng(1)
    streams = [(sorted(int(v) for v in rng.integers(0, n, T)), n) for T in (1, 2, 7, 40) for n in (1, 2, 5, 60) for _ in range(5)]
    for (ids, nseq), s in zip(streams, starts(streams)):
        assert s == [int(np.searchsorted(ids, i)) for i in [*range(nseq + 1), *range(nseq)]]

