"""What is worked out once per device (csrc/per_device.h), on the host: devices do not share
it, failures are not kept, threads agree."""
import os
import subprocess

from quantized_routed_expert_moe_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

int main() {
    static moe::PerDevice p;
    int made[40] = {};
    auto get = [&](int d) { return p.get(d, [&] { ++made[d]; return 100 + d; }); };
    // the second device works its own out; both keep it
    if (get(0) != 100 || get(1) != 101 || get(0) != 100 || get(1) != 101 || made[0] != 1 || made[1] != 1) return 1;
    // a failure is tried again
    if (p.get(2, [] { return 0; }) != 0 || get(2) != 102 || made[2] != 1) return 2;
    // past the table: right, and not kept
    if (get(39) != 139 || get(39) != 139 || made[39] != 2) return 3;
    if (p.get(-1, [] { return 7; }) != 7) return 4;
    // threads at the same time
    static moe::PerDevice q[64];
    std::vector<std::thread> t;
    std::atomic<int> wrong{0};
    for (int i = 0; i < 8; ++i)
        t.emplace_back([&] {
            for (int n = 0; n < 64 * 16; ++n)
                if (q[n / 16].get(n % 16, [&] { return n + 1; }) != n + 1) ++wrong;
        });
    for (auto& x : t) x.join();
    return wrong ? 5 : 0;
}
"""


def test_devices_do_not_share(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-pthread", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


def test_the_norm_keeps_its_layouts_per_device():
    """No plain static of the norm holds what a device gave."""
    text = open(os.path.join(build.CSRC, "block_norm.cu")).read()
    statics = [line.strip() for line in text.splitlines() if line.strip().startswith("static ")]
    assert len(statics) == 2 and all(line.startswith("static PerDevice ") for line in statics), statics
