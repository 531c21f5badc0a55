"""The remembered shared-memory limits of the kernels (csrc/largest_set.h), compiled for the
host with a setter that stands in for the CUDA call.  No GPU."""
import os
import subprocess

from mxfp4_expert_ffn_moe_b200 import build as moe_build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_expert_ffn_moe_b200", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "largest_set.h"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
    std::atomic<int> applied{0}, calls{0};
    const auto set = [&](int v) { applied = v; ++calls; return true; };
    {   // two threads whose first calls meet: the small size's setter is slow, the large one starts meanwhile
        moe::LargestSet<int> s;
        std::atomic<bool> inside{false};
        bool small = false, large = false;
        std::thread a([&] {
            small = s.ensure(1, 60, false, [&](int v) {
                inside = true;
                std::this_thread::sleep_for(std::chrono::milliseconds(200));
                return set(v);
            });
        });
        std::thread b([&] {
            while (!inside) std::this_thread::yield();
            large = s.ensure(1, 200, false, set);
        });
        a.join();
        b.join();
        CHECK(small && large && applied == 200);
        calls = 0;
        CHECK(s.ensure(1, 200, false, set) && s.ensure(1, 60, false, set) && calls == 0);
    }
    {   // keys are apart; a size that may be gone is set again and never lowered
        moe::LargestSet<int> s;
        CHECK(s.ensure(1, 100, false, set) && applied == 100);
        CHECK(s.ensure(2, 50, false, set) && applied == 50);
        CHECK(s.ensure(1, 70, true, set) && applied == 100);
        CHECK(s.ensure(1, 120, true, set) && applied == 120);
    }
    {   // a setter that fails is reported and not remembered
        moe::LargestSet<int> s;
        CHECK(!s.ensure(1, 100, false, [](int) { return false; }));
        calls = 0;
        CHECK(s.ensure(1, 100, false, set) && calls == 1);
    }
    return 0;
}
"""


def test_a_size_is_never_lowered(tmp_path):
    src = tmp_path / "program.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "program"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout


def test_the_library_sets_its_limits_through_it():
    text = open(os.path.join(CSRC, "moe_api.cu")).read()
    assert text.count("cudaFuncSetAttribute(kernel") == 1 and "LargestSet<" in text


def test_every_header_is_a_dependency_of_the_build():
    deps = {os.path.basename(d) for d in moe_build._deps()}
    assert {f for f in os.listdir(CSRC) if f.endswith((".h", ".cuh", ".cu"))} <= deps
