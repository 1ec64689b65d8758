"""The places in LDS of the tokens that a workgroup's tiles of the gathered 8-bit product read, replayed on the CPU from the
header that the kernel takes them from."""
import os
import subprocess

import moe_dispatch_expert_amd as mk

# A run of tiles, i = 0, 1, ...: the tokens of tile i are read by every wave in the steps before its products; waves that are
# through with those steps load the tokens of tile i + 1, with no barrier in between for i = 0.  So two tiles that
# follow one another must not share a word, and all of them must lie in the table.
PROGRAM = r"""
#define __host__
#define __device__
#include <cstdio>
#include "grouped_args.h"
int main()
{
    using namespace mk;
    for (int i = 0; i < 8; ++i) {
        const int a = tile_tokens_at(i), b = tile_tokens_at(i + 1);
        if (kTokenRows < 256 || a < 0 || a + kTokenRows > kTokenTable || b < 0 || b + kTokenRows > kTokenTable ||
            (a < b + kTokenRows && b < a + kTokenRows)) {
            std::printf("tile %d at %d, the next at %d, of %d\n", i, a, b, kTokenTable);
            return 1;
        }
    }
    return 0;
}
"""


def test_tokens_of_consecutive_tiles_have_places_of_their_own(tmp_path):
    src = tmp_path / "tokens.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "tokens"
    csrc = os.path.join(os.path.dirname(mk.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
