"""Settings of kernels belong to a device: they are made once for each device
of the process, by whichever thread comes first."""
import os
import re
import shutil
import subprocess

import pytest

from sampling_gnn_mini_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "sg_once.h"

int main() {
    // once for each device, in any order
    static sgi::OncePerDevice flags;
    int calls[66] = {0};
    const int order[] = {0, 0, 1, 0, 1, 63, 63, 7, 64, 64, -1};
    for (int dev : order)
        if (flags(dev, [&] { ++calls[dev + 1]; return 0; }) != 0) return 1;
    if (calls[1] != 1 || calls[2] != 1 || calls[64] != 1 || calls[8] != 1) return 2;
    if (calls[65] != 2 || calls[0] != 1) return 3;  // not remembered
    // a failure is returned and tried again
    static sgi::OncePerDevice fails;
    int tries = 0;
    if (fails(3, [&] { ++tries; return 5; }) != 5 || fails(3, [&] { ++tries; return 0; }) != 0) return 4;
    if (fails(3, [&] { ++tries; return 5; }) != 0 || tries != 2) return 5;
    // threads: nobody goes on before the setting has been made once
    static sgi::OncePerDevice shared;
    std::atomic<int> made{0}, early{0};
    std::vector<std::thread> all;
    for (int t = 0; t < 8; ++t)
        all.emplace_back([&] {
            for (int dev = 0; dev < 64; ++dev) {
                shared(dev, [&] { made.fetch_or(1); return 0; });
                if (!made.load()) ++early;
            }
        });
    for (auto& t : all) t.join();
    if (early.load()) return 6;
    puts("ok");
    return 0;
}
"""


def test_once_per_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, str(src), "-o", str(exe), "-pthread"], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_no_kernel_setting_is_made_once_a_process():
    # a plain flag or a cached answer would stand for every device
    flag = re.compile(r"static\s+(bool|int)\s+\w+\s*=\s*(false|-1)\s*;")
    for name in build.SOURCES:
        with open(os.path.join(build.CSRC, name)) as f:
            assert not flag.search(f.read()), name
