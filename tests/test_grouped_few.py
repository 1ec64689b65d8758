"""The rule by which the 8-bit product streams the weights for few rows, compiled on the CPU from the header that the kernel
takes it from, at counts on either side of it."""
import os
import subprocess

import moe_dispatch_expert_amd as mk

PROGRAM = r"""
#define __host__
#define __device__
#include <cstdio>
#include "grouped_args.h"
int main()
{
    int H, passes, most, N;
    while (std::scanf("%d %d %d %d", &H, &passes, &most, &N) == 4)
        std::printf("%d\n", mk::few_width(H, passes, most, N, 256, mk::inverse_of(256)));
    return 0;
}
"""

# rows of the experts that have any, N, the width of the stream's weight tiles (0: tiles) on 256 workgroups
CASES = [
    # one pass an expert: always the stream, of 16-row tiles where fewer rounds of them follow (or no task at all: 32)
    ([1], 8, 16), ([16], 4096, 16), ([16], 14336, 32), ([1] * 32, 2816, 32), ([16] * 32, 2048, 32), ([1] * 512, 40, 16),
    ([16] * 8, 14336, 32), ([1] * 1024, 1 << 20, 32), ([], 64, 32),
    # a long expert beside short ones: what the busiest workgroup goes through, not the mean of rows an expert
    ([17] + [1] * 31, 2816, 32), ([64] + [1] * 31, 2816, 32), ([256] + [1] * 31, 2816, 0), ([481] + [1] * 31, 2816, 0),
    ([481] + [1] * 31, 1408, 0), ([481] + [1] * 31, 56, 0), ([17] + [1] * 7, 14336, 32), ([128] + [1] * 7, 14336, 0),
    # several passes of many experts
    ([17] * 16 + [2] * 16, 2816, 0), ([17] * 4 + [2] * 28, 2816, 32), ([24] * 8, 14336, 0), ([32] * 16, 1024, 0),
    # few tasks: up to the weight rows of the narrowest tile
    ([17], 4096, 16), ([64], 4096, 16), ([65], 4096, 0), ([512], 72, 0), ([17], 14336, 0), ([17, 1], 4096, 32),
    ([40] * 8, 512, 16), ([80] + [1] * 7, 512, 0),
]


def test_rule_of_the_stream(tmp_path):
    src, exe = tmp_path / "few.cpp", tmp_path / "few"
    src.write_text(PROGRAM)
    csrc = os.path.join(os.path.dirname(mk.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    lines = []
    for counts, N, _ in CASES:
        passes = [-(-c // 16) for c in counts]
        lines.append(f"{len(counts)} {sum(passes)} {max(passes, default=0)} {N}")
    got = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split()
    for (counts, N, width), w in zip(CASES, got):
        assert int(w) == width, (counts[:4], len(counts), N, w, width)
    assert len(got) == len(CASES)
