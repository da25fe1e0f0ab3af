"""The channels that the gated recurrence's blocks take, on the host: every channel belongs to one
block, so a final state written over the initial one is never read by another block."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "gscan_groups.h"
int main() {
    for (int64_t C = 1; C <= 300; ++C)
        for (int64_t g = 0; g < ssm::g_groups(C); ++g)
            for (int64_t i = 0; i < 32; ++i)
                std::printf("%d %d %d\n", (int)C, (int)g, (int)ssm::g_pair(ssm::g_channels(C, g), i));
}
"""


def test_each_channel_in_one_group(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "groups.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "groups"
    subprocess.run([cxx, "-std=c++17", "-I", os.path.join(ROOT, "ssm_sequence_models_amd", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    owner = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        C, g, c0 = map(int, line.split())
        for c in (c0, c0 + 1) if C > 1 else (c0,):
            assert 0 <= c < C
            assert owner.setdefault((C, c), g) == g, f"{C} channels: {c} in two groups"
    assert len(owner) == sum(range(1, 301))
