"""The launch rules of the block-scaled FP8 product (csrc/fp8_plan.h), compiled
for the host and checked over a sweep of sizes: what the CTAs of the split
kernel take of an SM together.

An SM has 228 KB of shared memory, of which each resident CTA takes 1 KB more
than it asks for, and 512 columns of tensor memory.  tcgen05.alloc waits
without a time limit for columns that are not free, and a cluster's CTAs wait
for one another, so the CTAs that fit an SM by their shared memory must also
fit it by their tensor memory."""

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_communication_compression_gb300",
                    "csrc")

PROGRAM = r"""
#include <cstdio>
#include "fp8_plan.h"
int main()
{
    long long M, N, K;
    int sms;
    std::printf("%u\n", taco::kSplitTmem);
    while (std::scanf("%lld %lld %lld %d", &M, &N, &K, &sms) == 4) {
        const taco::SplitPlan p = taco::split_plan(M, N, K, sms);
        std::printf("%d %d %d %lld %d %d %u\n", taco::use_split(M, N, K, sms), p.bn, p.tiles_m,
                    static_cast<long long>(p.tiles), p.split, p.stages, p.smem);
    }
}
"""

SIZES = [1, 9, 16, 17, 37, 64, 65, 128, 200, 256, 300, 513, 1000, 2048, 2560, 4096, 4864, 5119, 8192, 10240, 16384, 20000,
         65536, 131072]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(at / "plan.cpp"), "-o",
                           str(at / "plan")])
    shapes = [(M, N, K, sms) for M in SIZES for N in SIZES for K in SIZES if K >= 16 for sms in (152, 148, 20)]
    out = subprocess.run([str(at / "plan")], input="\n".join("%d %d %d %d" % s for s in shapes), text=True,
                         stdout=subprocess.PIPE, check=True).stdout.split("\n")
    rows = [tuple(map(int, line.split())) for line in out[1:] if line]
    assert len(rows) == len(shapes)
    return int(out[0]), [(s, r[1:]) for s, r in zip(shapes, rows) if r[0]]


def test_tensor_memory_of_the_ctas_on_an_sm(plans):
    columns, split = plans
    assert len(split) > 1000
    for shape, (bn, tiles_m, tiles, ways, stages, smem) in split:
        resident = 228 * 1024 // (smem + 1024)
        assert 1 <= resident and resident * columns <= 512, shape
        assert 128 + 2 * 8 <= columns  # the accumulator's columns and two sets of scales


def test_shared_memory_holds_the_ring_and_the_partial_sums(plans):
    _, split = plans
    for (M, N, K, sms), (bn, tiles_m, tiles, ways, stages, smem) in split:
        per = 128 * 128 + 128 * bn
        assert bn % 16 == 0 and 16 <= bn <= 128 and (M <= bn or bn == 128)
        assert tiles_m == -(-M // 128) and tiles == tiles_m * -(-N // 128)
        assert 1 <= stages <= 10 and 512 * bn <= stages * per
        assert 1024 + stages * per + 4 * 1024 <= smem <= 232448
        assert 1 <= ways <= 8 and ways <= -(-K // 128)  # every CTA has a block


SUMS_PROGRAM = r"""
#include <cstdio>
#include "fp8_plan.h"
int main()
{
    long long M, N, K;
    int sms;
    while (std::scanf("%lld %lld %lld %d", &M, &N, &K, &sms) == 4) {
        const taco::SplitPlan p = taco::split_plan(M, N, K, sms, false);
        std::printf("%d %d %lld %d %d %u %d %u\n", taco::use_split(M, N, K, sms), p.bn, static_cast<long long>(p.tiles),
                    p.split, p.stages, p.smem, p.sums, taco::kSplitTmem);
    }
}
"""


def test_fp32_results_are_summed_in_pieces(tmp_path):
    # no CTA leaves more than 12 blocks to one sum in tensor memory
    (tmp_path / "plan.cpp").write_text(SUMS_PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "plan.cpp"), "-o",
                           str(tmp_path / "plan")])
    shapes = [(M, N, K, sms) for M in SIZES for N in SIZES for K in SIZES if K >= 16 for sms in (152, 148, 20)]
    out = subprocess.run([str(tmp_path / "plan")], input="\n".join("%d %d %d %d" % s for s in shapes), text=True,
                         stdout=subprocess.PIPE, check=True).stdout.split("\n")
    seen = set()
    for (M, N, K, sms), line in zip(shapes, out):
        use, bn, tiles, ways, stages, smem, sums, tmem = map(int, line.split())
        if not use:
            continue
        seen.add(sums)
        share = -(-(-(-K // 128)) // ways)
        assert sums in (0, 64, 128) and (share <= 12 if sums == 0 else bn <= sums), (M, N, K, sms)
        # what the sums and two sets of scales take, and what an SM has
        columns = 128  # one accumulator of up to 128, two of up to 64
        assert columns + 16 <= tmem and tmem in (256, 512)
        assert 228 * 1024 // (smem + 1024) * tmem <= 512, (M, N, K, sms)
        assert 1024 + stages * (128 * 128 + 128 * bn) + 4 * 1024 <= smem <= 232448 and 512 * bn <= stages * (128 + bn) * 128
        assert 1 <= ways <= 8 and ways <= -(-K // 128)
    assert seen == {0, 64, 128}
