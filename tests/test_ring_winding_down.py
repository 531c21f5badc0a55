"""The filling warp's last wait (csrc/ring.cuh), compiled for the host against a model of the
barriers: it has to block on exactly the stages whose last fill has not landed.  No GPU."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_expert_ffn_moe_b200", "csrc")

MODEL = r"""
#include <cstdio>
#include "ring.cuh"
// A barrier that has completed `phases` phases: a wait for a parity blocks while the
// running phase has it.
static bool passes(int phases, uint32_t parity) { return (uint32_t)(phases & 1) != parity; }
int main() {
    int checked = 0;
    for (int stages = 1; stages <= 8; ++stages)
        for (int fills = 0; fills <= 5 * stages + 3; ++fills) {
            int stage = 0, filled[8] = {};
            uint32_t phase = 0;
            for (int f = 0; f < fills; ++f) {
                ++filled[stage];
                if (++stage == stages) stage = 0, phase ^= 1u;
            }
            for (int i = 0; i < stages; ++i) {
                const uint32_t parity = moe::last_fill_parity(i, stage, phase);
                // a stage is filled again only once its fill before has landed: one at most is under way
                if (!passes(filled[i], parity)) return std::printf("blocks on landed fill %d of %d\n", i, stages), 1;
                if (filled[i] && passes(filled[i] - 1, parity)) return std::printf("misses fill %d of %d\n", i, stages), 1;
                ++checked;
            }
        }
    return checked > 500 ? 0 : 1;
}
"""


def test_the_last_fill_of_every_stage_is_waited_for(tmp_path):
    src = tmp_path / "model.cpp"
    src.write_text(MODEL)
    exe = tmp_path / "model"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout


def test_every_filling_warp_waits_before_it_leaves():
    # one wait per ring with copies under way: the row kernels' two rings, and the matvec's weights and scales
    count = {name: open(os.path.join(CSRC, name)).read().count("wait_for_fills(") for name in ("pair_rows.cuh", "matvec.cuh")}
    assert count == {"pair_rows.cuh": 2, "matvec.cuh": 2}
