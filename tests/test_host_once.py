"""What the library keeps per device (csrc/once.h), compiled here with the host
compiler: threads whose first calls ask for different shared-memory sizes."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

#include "once.h"

int main()
{
    using namespace std::chrono_literals;
    int bad = 0;
    for (int round = 0; round < 40; ++round) {
        as::RaisedLimit limit;
        std::atomic<int> attribute{0}, calls{0};
        // the small size's setting is slow: unordered, it lands after the large one's
        auto set = [&](int v) {
            ++calls;
            std::this_thread::sleep_for(v < 100 ? 3ms : 1ms);
            attribute = v;
            std::this_thread::sleep_for(1ms);
            return 0;
        };
        std::vector<std::thread> t;
        for (int v : {50, 200, 60, 200, 40}) t.emplace_back([&, v] {
            if (limit.raise(0, v, set) || attribute < v) ++bad;  // a launch with v bytes would fail
        });
        for (auto &x : t) x.join();
        if (attribute != 200 || calls > 4) ++bad;
        const int before = calls;
        if (limit.raise(0, 200, set) || limit.raise(0, 10, set) || calls != before) ++bad;  // nothing to do
        if (limit.raise(1, 30, set) || calls != before + 1) ++bad;                          // another device
        if (limit.raise(2, 30, [](int) { return 7; }) != 7) ++bad;
        if (limit.raise(2, 30, set) || calls != before + 2) ++bad;                          // a failure is not kept
        if (limit.raise(as::KEPT_DEVICES, 30, set) || calls != before + 3) ++bad;
    }
    as::DeviceAnswer answer;
    for (int dev : {0, 1, 0, 1, -1, as::KEPT_DEVICES})
        if (answer.get(dev, [&] { return dev + 5; }) != dev + 5) ++bad;
    if (answer.get(0, [] { return 99; }) != 5 || answer.get(-1, [] { return 99; }) != 99) ++bad;
    printf("%d\n", bad);
    return bad != 0;
}
"""


def test_limits_with_many_threads(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "sparse_linear_b200", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
