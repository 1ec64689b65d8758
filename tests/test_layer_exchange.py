"""The LDS regions in which the few-token layer's waves exchange their sums, replayed on the CPU from the header that the
kernels take them from."""
import os
import subprocess

import moe_dispatch_expert_amd as mk

# One exchange writes and reads [at(par), at(par) + waves * R * 256) for a task of R weight tiles, and the next one takes the
# other half.  A wave that is through with the next task's K steps writes its sums while slower waves still read the
# present ones, so two consecutive exchanges must be disjoint for every pair of tile counts.
PROGRAM = r"""
#define __host__
#define __device__
#include <cstdio>
#include "layer_args.h"
int main()
{
    using namespace mk;
    const int tiles[] = {1, 2, 4};
    for (int par = 0; par < 2; ++par)
        for (int r : tiles)
            for (int next : tiles) {
                const int a = layer_exchange_at(par), a_end = a + kLayerWaves * r * 256;
                const int b = layer_exchange_at(par ^ 1), b_end = b + kLayerWaves * next * 256;
                if (a < 0 || b < 0 || a_end * 4 > kExchangeBytes || b_end * 4 > kExchangeBytes ||
                    (a < b_end && b < a_end)) {
                    std::printf("half %d of %d tiles [%d, %d) against %d tiles [%d, %d)\n", par, r, a, a_end, next, b, b_end);
                    return 1;
                }
            }
    return 0;
}
"""


def test_consecutive_exchanges_use_disjoint_regions(tmp_path):
    src = tmp_path / "exchange.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "exchange"
    csrc = os.path.join(os.path.dirname(mk.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
