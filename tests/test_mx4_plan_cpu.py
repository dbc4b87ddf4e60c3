"""Which kernel the microscaled products and experts take, asked on the host (no GPU)."""
import os
import subprocess

import pytest

from mx4_plan_util import BLOCKS, WAYS

pytestmark = pytest.mark.cpu
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_quantize_amd", "csrc")
PROGRAM = r"""
#include <stdio.h>
#include "mx4_plan.hpp"
int main() {
    char kind;
    long long a[5];
    while (scanf(" %c %lld %lld %lld %lld %lld", &kind, a, a + 1, a + 2, a + 3, a + 4) == 6) {
        if (kind == 'b') {
            const w4::BlockPlan p = w4::block_plan(a[1], a[2], a[3], a[0], a[4]);
            const w4::BlockShape& s = (a[0] ? w4::kShapesX4 : w4::kShapes)[p.shape];
            printf("%d %d %d\n", s.bm, s.bn, p.parts);
        } else {
            const w4::MoeWay w = w4::moe_way(a[0], (int)a[2], a[1], a[3], a[4]);
            printf("%d\n", w.direct ? 0 : w.rows);
        }
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def ask(kind, cases):
        text = "".join(f"{kind} {' '.join(str(int(v)) for v in c)}\n" for c in cases)
        out = subprocess.run([str(d / "plan")], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def test_the_sizes_reach_every_block(plan):
    assert plan("b", BLOCKS) == list(BLOCKS.values())
    # every block that any size takes is among them, whole and (but for the least used) in pieces
    seen = {(c[0],) + b[:2] for c, b in BLOCKS.items()}
    cases = [(x4, M, N, K, ws) for x4 in (0, 1) for ws in (0, 1) for K in (32, 608, 4096, 11008)
             for N in (1, 100, 300, 1000, 4096, 11008, 50000) for M in (17, 50, 100, 200, 333, 700, 2048, 4097, 9000)]
    assert {(bool(c[0]),) + b[:2] for c, b in zip(cases, plan("b", cases))} == seen
    assert {(c[0],) + b[:2] for c, b in BLOCKS.items() if b[2] > 1} == seen
    assert {(c[0],) + b[:2] for c, b in BLOCKS.items() if b[2] == 1} == seen


def test_the_sizes_reach_every_way_of_the_experts(plan):
    assert plan("e", WAYS) == [(w,) for w in WAYS.values()]
    assert set(WAYS.values()) == {0, 8, 16, 64, 128}
