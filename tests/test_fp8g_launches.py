"""How the workgroups of a product with group scales are dealt among launches (CPU)."""
import shutil
import subprocess

import pytest

from tensor_transformer_mlp_02_amd import build as b


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("launches")
    (d / "launches.cpp").write_text("""
#include <cstdio>
#include <cstdlib>
#include "fp8g_plan.h"
int main(int, char** v) {  // blocks, the launch that fails
  int left = atoi(v[2]);
  const int r = tpmlp::g8_in_launches(atoll(v[1]), [&](int64_t first, int64_t count) {
    printf("%lld %lld\\n", (long long)first, (long long)count);
    return --left == 0 ? 7 : 0;
  });
  printf("%d", r);
}
""")
    exe = str(d / "launches")
    subprocess.run(["g++", "-std=c++17", "-I", b.CSRC, str(d / "launches.cpp"), "-o", exe], check=True)

    def run(blocks, fails=0):
        *rows, status = subprocess.run([exe, str(blocks), str(fails)], capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(map(int, r.split())) for r in rows], int(status)
    return run


@pytest.mark.parametrize("blocks", [0, 1, 1000, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, 1 << 24, (1 << 25) + 12345, (1 << 31) - 1])
def test_every_block_once(launches, blocks):
    rows, status = launches(blocks)
    assert status == 0
    at = 0
    for first, count in rows:
        assert first == at and 0 < count and count * 512 < 1 << 32      # threads of the largest workgroups
        at += count
    assert at == blocks


def test_a_failure_ends_it(launches):
    rows, status = launches(1 << 24, 2)
    assert len(rows) == 2 and status == 7
