"""Host replay of which rows the verification of drafts looks at (no GPU): the mapping that
the kernels use, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_decode_matmul_b200", "csrc")
SOURCE = """
#include "verify_jobs.h"
extern "C" int jobs(int n, int base, int* out) {
  for (int i = 0; i < wq::verify::jobs_of(n); ++i) {
    const wq::verify::Job j = wq::verify::job_of(i, n, base);
    out[3 * i] = j.row; out[3 * i + 1] = j.token_row; out[3 * i + 2] = j.is_draft;
  }
  return wq::verify::jobs_of(n);
}
"""


@pytest.fixture(scope="module")
def jobs(tmp_path_factory):
    d = tmp_path_factory.mktemp("jobs")
    (d / "jobs.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "jobs.cpp"), "-o",
                    str(d / "jobs.so")], check=True)
    lib = ctypes.CDLL(str(d / "jobs.so"))

    def of(n, base):
        out = (ctypes.c_int * (6 * n + 3))()
        count = lib.jobs(n, base, out)
        return [tuple(out[3 * i:3 * i + 3]) for i in range(count)]
    return of


@pytest.mark.parametrize("drafts", [0, 1, 5, 31, 32, 33, 64, 70])
def test_rows_that_are_looked_at(jobs, drafts):
    """Every target row and every draft row but a sequence's first, 32 drafts at a time as long
    as all are accepted; the token in question is the one that a target row judges, or its own."""
    target, draft, base = [], [], 0
    while True:
        n = min(drafts - base, 32)
        for row, token_row, is_draft in jobs(n, base):
            assert base <= row <= base + n
            assert token_row == (row if is_draft else row + 1)
            (draft if is_draft else target).append(row)
        if base + n == drafts:
            break
        base += 32
    assert sorted(set(target)) == list(range(drafts + 1))
    assert sorted(draft) == list(range(1, drafts + 1))
