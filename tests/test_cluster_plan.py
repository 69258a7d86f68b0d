"""Which cluster a small attention call gets, by the host's rule alone: compiled into a program
of its own, with rooms that a device could have."""
import os
import subprocess

import pytest

from rag_kv_cache_layer_gb300 import build as B

PROGRAM = r"""
#include <stdio.h>
#include "cb_paged_attn.cuh"
int main() {
  long long items, blocks;
  int sms, per_sm, parts, most, has, r[5];
  while (scanf("%lld %lld %d %d %d %d %d %d %d %d %d %d", &items, &blocks, &sms, &per_sm, &parts, &most, &has, r, r + 1,
               r + 2, r + 3, r + 4) == 12)
    printf("%d\n", cb::paged::plan_cluster(items, blocks, sms, per_sm, parts, most, has ? r : nullptr));
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "p.cu").write_text(PROGRAM)
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", os.path.join(B.ROOT, "include"), "-I", B.CSRC,
                    "-o", str(d / "p"), str(d / "p.cu")], check=True, capture_output=True)

    def run(items, blocks, room=None, sms=152, per_sm=1, parts=304, most=16):
        line = [items, blocks, sms, per_sm, parts, most, int(room is not None), *(room or [0] * 5)]
        return int(subprocess.run([str(d / "p")], input=" ".join(map(str, line)), capture_output=True, text=True, check=True).stdout)
    return run


def test_a_device_that_takes_all_clusters(plan):
    room = [152, 152, 144, 120, 112]
    for items, blocks, c in [(1, 1, 1), (1, 9, 2), (1, 64, 8), (1, 65, 16), (6, 128, 16), (7, 128, 8), (30, 32, 4), (152, 8, 1),
                             (153, 8, 0), (153, 800, 0)]:
        assert plan(items, blocks) == plan(items, blocks, room) == c, (items, blocks)


def test_a_device_without_large_clusters(plan):
    """A size that the device has no place for is not launched: a smaller one, or the line."""
    assert plan(1, 98, [152, 152, 144, 120, 0]) == 8
    assert plan(1, 60, [152, 152, 144, 0, 0]) == 4
    assert plan(1, 60, [152, 152, 0, 0, 0]) in (0, 2)
    assert plan(1, 4, [0, 0, 0, 0, 0]) == 0
    assert plan(1, 98, [0, 0, 0, 0, 0]) == 0


def test_a_device_with_room_for_fewer(plan):
    assert plan(6, 98, [152, 152, 144, 120, 112]) == 16
    assert plan(6, 98, [152, 152, 144, 120, 80]) == 8          # five clusters of 16
    assert plan(6, 98, [152, 152, 144, 40, 80]) in (0, 4)
    # (more room than the plan counts on changes nothing)
    assert plan(30, 64, [304, 304, 288, 240, 224]) == plan(30, 64)
