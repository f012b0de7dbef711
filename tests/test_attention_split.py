"""What the host works out of a decode call's sizes before it launches (csrc/attn_split.h), compiled by itself: no GPU
needed."""

import os
import shutil
import subprocess

import pytest

import quantized_routed_expert_03_gb300 as qre

CSRC = os.path.join(os.path.dirname(qre.__file__), "csrc")
PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "attn_split.h"
int main(int argc, char** argv) {
  long long x[16] = {};
  for (int i = 2; i < argc; ++i) x[i - 2] = atoll(argv[i]);
  long long r = -1;
  if (!strcmp(argv[1], "join_counts")) r = qre::shared_join_counts(x[0], x[1], x[2]);
  if (!strcmp(argv[1], "join_ways")) r = qre::shared_join_ways(x[0], x[1], x[2], x[3], x[4], x[5], x[6]);
  if (!strcmp(argv[1], "ctas")) r = qre::decode_ctas(x[0], x[1], x[2], x[3]);
  if (!strcmp(argv[1], "room")) r = qre::decode_room(x[0], x[1], x[2]);
  printf("%lld", r);
}
"""


@pytest.fixture(scope="module")
def call(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    where = tmp_path_factory.mktemp("split")
    (where / "split.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(where / "split"), str(where / "split.cpp")],
                   check=True)

    def run(name, *args):
        out = subprocess.run([str(where / "split"), name, *map(str, args)], capture_output=True, text=True)
        assert out.returncode == 0, f"{name}{args} ended with {out.returncode}"
        return int(out.stdout)
    return run


def test_the_shared_join_counts_only_what_31_bits_hold(call):
    """The places of a call, and the first place of any unit, are at most queries * places * units."""
    for n, places, units in ((1, 5, 1), (64, 1030, 8), (128, 65541, 256), (128, 65541, 255), (1024, 8197, 8), (1024, 8197, 255),
                             (1024, 8197, 256), (2, 2 ** 30 - 1, 1), (1, 2 ** 31 - 1, 1), (1, 2 ** 31 - 1, 2), (15, 2 ** 27, 1),
                             (15, 2 ** 27, 2), (1, 2 ** 27 + 5, 1024)):
        assert call("join_counts", n, places, units) == (n * places * units <= 2 ** 31 - 1), (n, places, units)


def test_warps_of_the_shared_join_for_any_number_of_groups(call):
    def ways(n, heads, kv_heads, groups):
        return call("join_ways", n, heads, kv_heads, groups, 152, 256, 20)
    assert ways(4, 4, 2, 0) == 1 and ways(4096, 64, 8, 0) == 1          # no groups: nothing to divide by
    for n, groups in ((1, 1), (2, 4096), (4096, 4096), (4096, 1), (1, 4096)):
        for heads, kv_heads in ((1, 1), (1024, 1), (256, 256), (64, 8)):
            w = ways(n, heads, kv_heads, groups)
            assert w in (1, 2, 4, 8) and (w == 1 or n * heads * w // 2 <= 8 * 152)
    assert ways(3, 3, 1, 1) == 8 and ways(64, 32, 8, 1) == 1


def test_ctas_of_the_decode_kernel_that_fit(call):
    smem, low, other = 232448, 2 * 4 * 2 * 64 * 72, 2 * 4 * 2 * 4096    # two stages of four warps: 4 bits at 128, any 16 bits
    assert [call("ctas", 3, smem, 12 * (n + 1), low) for n in (1, 233, 234, 3476, 3477, 4096)] == [3, 3, 2, 2, 1, 1]
    assert [call("ctas", 3, smem, 24 * (n + 1), low) for n in (1, 116, 117, 1024)] == [3, 3, 2, 2]
    assert [call("ctas", 2, smem, b * (n + 1), other) for b, n in ((12, 1), (12, 4096), (24, 1024))] == [2, 2, 2]
    for most in (1, 2, 3):
        for of_queries in range(0, 50000, 1100):
            n = call("ctas", most, smem, of_queries, low)
            assert n == 1 or call("room", n, smem, of_queries) >= low
            assert n == most or call("room", n + 1, smem, of_queries) < low
