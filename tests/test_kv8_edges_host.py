"""What the 8-bit K/V cache operators do at their edges, without a GPU: functions of csrc/kv8_map.h, compiled here."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(tmp_path, main):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "edges.cpp", tmp_path / "edges"
    src.write_text(main)
    subprocess.check_call([cc, "-std=c++17", "-O1", "-fsanitize=undefined,address", "-I",
                           os.path.join(ROOT, "quantized_decode_gb300", "csrc"), str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def test_how_a_row_ends(tmp_path):
    """A row that saw nothing is 0 with an lse of -infinity; one whose waits ran out is NaN, so that a caller without an err
    word can tell the two apart."""
    _run(tmp_path, r"""
#include <stdio.h>
#include "kv8_map.h"
using namespace qd;
#define CHECK(c) do { if (!(c)) { printf("failed: %s\n", #c); return 1; } } while (0)
int main() {
    CHECK(kv8_row_factor(true, 0.f) == 0.f && kv8_row_log2(true, 0.f, 3.f) == -INFINITY);
    CHECK(kv8_row_factor(true, 4.f) == 0.25f && kv8_row_log2(true, 4.f, 3.f) == 5.f);
    const float sums[3] = {0.f, 4.f, NAN};
    for (float sum : sums) CHECK(isnan(kv8_row_factor(false, sum)) && isnan(kv8_row_log2(false, sum, 3.f)));
    CHECK(isnan(kv8_row_factor(true, NAN)) && isnan(kv8_row_log2(true, NAN, 3.f)));
    printf("ok\n");
    return 0;
}
""")
