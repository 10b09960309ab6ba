"""What a launch keeps of its device's answers, without a GPU: a small host program asks a fake device."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = r"""
#include "resident.h"
#include <cstdio>
#define CHECK(x) if (!(x)) { std::printf("%s\n", #x); return 1; }
static sgq::Resident kept;
int main() {
    int asked = 0, answer = 0;
    auto ask = [&] { ++asked; return answer; };
    CHECK(kept.on(0, ask) == 0 && kept.on(0, ask) == 0 && asked == 2);   // a failure is not kept
    answer = -1;
    CHECK(kept.on(0, ask) == 0 && asked == 3);
    answer = 5;
    CHECK(kept.on(0, ask) == 5 && asked == 4);
    answer = 7;
    CHECK(kept.on(0, ask) == 5 && asked == 4);                           // an answer is,
    CHECK(kept.on(1, ask) == 7 && asked == 5);                           // for its own device
    CHECK(kept.on(63, ask) == 7 && kept.on(0, ask) == 5 && asked == 6);
    CHECK(kept.on(64, ask) == 0 && kept.on(-1, ask) == 0 && asked == 6);
    return 0;
}
"""


def test_answers_are_kept_by_device_and_failures_are_not(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    (tmp_path / "t.cpp").write_text(CODE)
    csrc = os.path.join(ROOT, "fp8_block_scaled_sgq_gb300", "csrc")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", csrc, "-o", str(tmp_path / "t"), str(tmp_path / "t.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_narrow_norms_keep_theirs_so():
    with open(os.path.join(ROOT, "fp8_block_scaled_sgq_gb300", "csrc", "norm.cu")) as f:
        text = f.read()
    at = text.index("cudaOccupancyMaxActiveBlocksPerMultiprocessor")
    assert "resident.on(dev" in text[at - 200:at] and "static const int" not in text
