"""What is under way when the CTAs of a TMA ring give up (csrc/ring_end.h), on the CPU: the header that the kernels
use, on modelled barriers.

A producer, or two of a pair, and the tensor cores run by a random schedule and stop at random slices, each by itself, as
after waits that ran out; copies land in any order and at any time. After that no copy may be under way once
land_ring returns, and every barrier that it waits for completes by the copies that there are."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_async_gb300", "csrc")

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "ring_end.h"

static std::mt19937 rng(1);
static uint32_t below(uint32_t n) { return (uint32_t)(rng() % n); }

struct Barrier {                     // one arrival and the announced bytes make a phase
    long long pending = 1, bytes = 0;
    uint32_t phases = 0;
    void settle() { if (pending == 0 && bytes == 0) { pending = 1; ++phases; } }
    void arrive(long long announced) { bytes += announced; --pending; settle(); }
    void complete(long long n) { bytes -= n; settle(); }
    bool done(uint32_t parity) const { return (phases & 1u) != parity; }
};

constexpr long long X = 16, W = 24;  // bytes of a CTA's two copies
struct Copy { uint32_t stage; long long bytes; };

struct Model {
    std::vector<Barrier> full;
    std::vector<Copy> flying;
    int waits_in_vain = 0;
    void land(size_t i)
    {
        full[flying[i].stage].complete(flying[i].bytes);
        flying[i] = flying.back();
        flying.pop_back();
    }
    // what land_ring is given
    void announce(uint32_t stage) { full[stage].arrive(X + W); }
    void excuse(uint32_t stage) { full[stage].complete(X + W); }
    void landed(uint32_t stage, uint32_t parity)
    {
        while (!full[stage].done(parity)) {
            if (flying.empty()) { ++waits_in_vain; return; }
            land(below((uint32_t)flying.size()));
        }
    }
};

int main(int argc, char** argv)
{
    const uint32_t stages = (uint32_t)atoi(argv[1]);
    const bool pair = atoi(argv[2]) != 0;
    long left_before = 0, apart[2] = {0, 0};
    for (int run = 0; run < 20000; ++run) {
        Model m;
        m.full.resize(stages);
        const uint32_t total = below(4 * stages + 2);
        // each stops before this slice of its own, or runs to the end
        const uint32_t stop[3] = {below(total + 2), below(total + 2), below(total + 2)};
        uint32_t issued[2] = {0, 0}, used = 0;
        for (uint32_t step = below(30 * stages); step > 0; --step) {
            const uint32_t who = below(4);
            if (who < (pair ? 2u : 1u)) {
                uint32_t& i = issued[who];
                // a stage is free once the slice before it there has been used
                if (i < total && i < stop[who] && (i < stages || used > i - stages)) {
                    const uint32_t s = i % stages;
                    if (who == 0) m.full[s].arrive((pair ? 2 : 1) * (X + W));
                    m.flying.push_back({s, X});
                    m.flying.push_back({s, W});
                    ++i;
                }
            } else if (who == 2) {
                if (used < total && used < stop[2] && used < issued[0] && m.full[used % stages].done((used / stages) & 1u)) ++used;
            } else if (!m.flying.empty() && below(3) == 0) {
                m.land(below((uint32_t)m.flying.size()));
            }
        }
        if (!pair) issued[1] = issued[0];
        left_before += !m.flying.empty();
        apart[0] += issued[0] > issued[1];
        apart[1] += issued[1] > issued[0];
        fdpp::land_ring(m, issued[0], issued[1], stages);
        if (!m.flying.empty() || m.waits_in_vain) {
            printf("run %d: issued %u %u of %u, used %u: %zu copies under way, %d waits in vain\n", run, issued[0], issued[1], total,
                   used, m.flying.size(), m.waits_in_vain);
            return 1;
        }
        const uint32_t most = issued[0] > issued[1] ? issued[0] : issued[1];
        for (uint32_t i = 0; i < stages; ++i)
            if (m.full[i].phases != most / stages + (i < most % stages)) {
                printf("run %d: a barrier with the wrong number of phases\n", run);
                return 1;
            }
    }
    printf("%ld %ld %ld\n", left_before, apart[0], apart[1]);
    return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("c++")
    assert compiler
    d = tmp_path_factory.mktemp("ring")
    (d / "model.cpp").write_text(MODEL)
    subprocess.run([compiler, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(d / "model.cpp"), "-o", str(d / "model")],
                   check=True)
    return str(d / "model")


@pytest.mark.parametrize("stages", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("pair", [0, 1])
def test_every_copy_lands(model, stages, pair):
    r = subprocess.run([model, str(stages), str(pair)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    left, first_ahead, second_ahead = map(int, r.stdout.split())
    # the schedules have what it is for: copies under way, and producers of a pair that stopped apart
    assert left > 1000
    assert not pair or (first_ahead > 1000 and second_ahead > 1000)


def test_kernels_end_by_it():
    """Both kernels of the 8-bit linear land their ring after the barrier behind which no warp issues."""
    source = open(os.path.join(CSRC, "scaled_gemm.cu")).read()
    for kernel, barrier in (("scaled_rows_kernel(", "__syncthreads();"), ("scaled_tile_kernel(", "if (meet())")):
        body = source.split(kernel, 1)[1].split("__global__", 1)[0]
        end = body.index("land_ring(")
        assert body.rindex("tma_load_2d", 0, end) < body.rindex(barrier, 0, end) < end
        assert "ring_used(" in body and body.count("land_ring(") == 1
