"""How fp8_gemm.cu lays out its launches for few rows, by the arithmetic it uses (csrc/fp8_plan.h).

Blocks of a cluster wait for one another while they hold tensor memory, 512 columns an SM. Two such
kernels on different streams must never meet on an SM that cannot give both their columns: each
could hold what the other's cluster waits for. Shared memory keeps them apart, which is checked here
over every plan that a call can get. (Blocks that are no cluster's wait for nobody and end.)
"""
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "int4_quantized_b200", "csrc")
SM_SHARED = 228 * 1024  # of an SM; 1 KB of it is kept for each block
MOST = 227 * 1024       # of a block

MAIN = r"""
#include "fp8_plan.h"
#include <cstdio>
// per width and number of CTAs: the least and the most shared memory, the least and the most stages
int main() {
    for (int nt : {16, 32, 64})
        for (int split = 1; split <= 8; split *= 2) {
            size_t lo = ~(size_t)0, hi = 0;
            int s_lo = 1 << 30, s_hi = 0, bad = 0;
            for (int64_t E : {1, 2, 64, 1023, 1024})
                for (int kb = 1; kb <= 600; ++kb)
                    for (int64_t tiles = 1; tiles <= 400; ++tiles) {
                        const q4::StreamPlan p = q4::stream_plan(nt, tiles, kb, E, 148);
                        if (p.split != split) continue;
                        lo = p.smem < lo ? p.smem : lo, hi = p.smem > hi ? p.smem : hi;
                        s_lo = p.stages < s_lo ? p.stages : s_lo, s_hi = p.stages > s_hi ? p.stages : s_hi;
                        bad += p.smem < q4::stream_smem(nt, p.stages, split, E);
                        bad += split > 1 && (tiles * split > 148 || kb < 2 * split);
                    }
            if (hi) std::printf("%d %d %zu %zu %d %d %d\n", nt, split, lo, hi, s_lo, s_hi, bad);
        }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(MAIN)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", CSRC, "-o", str(d / "main"), str(d / "main.cpp")])
    out = subprocess.check_output([str(d / "main")], text=True)
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_plans_fit(plans):
    assert {p[:2] for p in plans} >= {(nt, split) for nt in (16, 32, 64) for split in (1, 2, 4, 8)}
    for nt, split, lo, hi, s_lo, s_hi, bad in plans:
        assert bad == 0 and hi <= MOST and 2 <= s_lo and s_hi <= 16


def test_clusters_that_meet_on_an_sm_share_its_tensor_memory(plans):
    least = {nt: min(p[2] for p in plans if p[0] == nt and p[1] > 1) for nt in (16, 32, 64)}
    # the pairs of many rows hold all columns: at least 4 stages of 32 KB and 64 KB of y or 4 of 48 KB
    kinds = [(8 * nt, smem) for nt, smem in least.items()] + [(512, 192 * 1024)]
    for n in range(2, 6):
        for blocks in itertools.combinations_with_replacement(kinds, n):
            if sum(smem + 1024 for _, smem in blocks) <= SM_SHARED:
                assert sum(cols for cols, _ in blocks) <= 512, blocks


SHAPES = r"""
#include "fp8_plan.h"
#include <cstdio>
int main(int argc, char **argv) {  // lines of: grouped E N R
    long g, E, N, R;
    while (std::scanf("%ld %ld %ld %ld", &g, &E, &N, &R) == 4) std::printf("%d\n", (int)q4::wide_shape(g, E, N, R, 148));
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    d = tmp_path_factory.mktemp("shapes")
    (d / "main.cpp").write_text(SHAPES)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", CSRC, "-o", str(d / "main"), str(d / "main.cpp")])

    def ask(cases):
        text = "".join("%d %d %d %d\n" % c for c in cases)
        return list(map(int, subprocess.run([str(d / "main")], input=text, text=True, capture_output=True, check=True).stdout.split()))

    return ask


def test_one_expert_takes_the_tiles_of_a_dense_product(shapes):
    cases = [(N, R) for N in (1, 128, 768, 1408, 4096, 11008, 14336) for R in range(8, 4200, 37)] + [(4096, 511), (4096, 512), (4096, 513)]
    assert shapes([(1, 1, N, R) for N, R in cases]) == shapes([(0, 1, N, R) for N, R in cases])


def test_no_number_of_rows_an_expert_is_special(shapes):
    # one row more or less changes the shape only where a number of rounds changes, so seldom, and not
    # at the same number of rows an expert for most sizes
    sizes = [(E, N) for E in (2, 8, 16, 64, 200) for N in (300, 1408, 2304, 4096, 14336)]
    changes = {}
    for r in (128, 256, 512, 1024, 2048):
        at = shapes([(1, E, N, E * r) for E, N in sizes])
        below = shapes([(1, E, N, E * r - 1) for E, N in sizes])
        changes[r] = sum(a != b for a, b in zip(at, below))
    assert max(changes.values()) <= 2, changes


def test_shapes_of_the_extremes(shapes):
    # single CTAs, pairs and narrow tiles each have sizes of their own, and the largest do not overflow
    assert shapes([(0, 1, 11008, 333), (0, 1, 14336, 8192), (0, 1, 4096, 512)]) == [0, 1, 2]
    assert shapes([(1, 8, 14336, 32), (1, 2, 2304, 4100)]) == [0, 1]
    assert shapes([(0, 1, 1 << 30, 1 << 30), (1, 1024, 1 << 20, 1 << 30)]) == [1, 1]


def test_the_gpu_tests_reach_every_shape(shapes):
    # the sizes of test_gpu_fp8_tiles.py by the kernel they are there for
    single = [(0, 1, 11008, 333), (0, 1, 10001, 333), (0, 1, 12000, 300), (0, 1, 9473, 300), (1, 4, 9472, 35), (1, 4, 9470, 36)]
    pair = [(0, 1, 9472, 1500), (0, 1, 9328, 1411), (0, 1, 9471, 1511), (0, 1, 6152, 2045), (1, 2, 9001, 2003), (1, 2, 2312, 4100),
            (1, 4, 2340, 4204), (1, 3, 2304, 4104), (1, 3, 2305, 4104), (1, 3, 2312, 4104), (1, 3, 2320, 4104)]
    narrow = [(0, 1, 4096, 512), (0, 1, 4104, 200), (0, 1, 2305, 700), (1, 8, 4736, 35)]
    assert shapes(single + pair + narrow) == [0] * len(single) + [1] * len(pair) + [2] * len(narrow)
