"""How a product with bias, activation and residual splits its depth decides the order of its sums, which is stated to
follow from sizes, strides and alignment alone. The plan is compiled here without CUDA, where it has no device to ask, and
its choices are checked over the sizes' range."""
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "diffusion_transformer_step_gb300", "csrc")

PROGRAM = """
#include <cstdio>
#include "linear_act_plan.h"
int main() {
  int rows, n, kblocks, lines;
  while (std::scanf("%d %d %d %d", &rows, &n, &kblocks, &lines) == 4) {
    const dit::LinearActPlan p = dit::linear_act_plan(rows, n, kblocks, lines != 0);
    std::printf("%d %d\\n", p.bn, p.splits);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cc").write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "plan.cc"), "-o", str(d / "plan")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        r = subprocess.run([str(d / "plan")], input="".join("%d %d %d %d\n" % c for c in cases), capture_output=True, text=True, check=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


def test_kernel_asks_no_device_for_its_splits():
    """The launching code takes its splits from the plan and from nothing that differs between devices."""
    with open(os.path.join(CSRC, "linear_act.cu")) as f:
        text = f.read()
    assert "linear_act_plan(" in text
    for word in ("Occupancy", "clusters_at_once", "cudaDeviceGetAttribute", "cudaGetDeviceProperties"):
        assert word not in text, word


def test_splits_fit_their_kernels(plan):
    """Every size has a plan that its kernel takes: up to eight splits of two 64-deep blocks at least for few rows, up to four of
    eight for wide tiles of 256, 192 or 128 columns, whose parts the ring has room for."""
    sides = (1, 2, 16, 33, 64, 65, 128, 129, 256, 257, 777, 4096, 8192, 1 << 20)
    cases = [(m, n, k, lines) for m, n in itertools.product(sides, sides) for k in (1, 2, 3, 15, 16, 31, 32, 64, 81, 1 << 14) for lines in (0, 1)]
    for (m, n, k, _), (bn, s) in zip(cases, plan(cases)):
        if m <= 128:
            assert bn == 0 and 1 <= s <= 8 and (s == 1 or k // s >= 2), (m, n, k, bn, s)
        else:
            assert bn in (128, 192, 256) and 1 <= s <= 4 and (s == 1 or k // s >= 8), (m, n, k, bn, s)


def test_known_choices(plan):
    """Both kernels, split and whole, on their lines and off them. Of clusters of 2, 3, 4, 6 and 7 CTAs 76, 46, 36, 23 and 15 run at
    once, twice as many up to 64 rows where fewer than three splits fit once."""
    want = {(1, 2560, 64, 1): (0, 6),      # 20 blocks of columns
            (1, 12288, 64, 1): (0, 2),     # 96, two CTAs per SM
            (64, 4096, 64, 1): (0, 4),     # 32
            (128, 4096, 64, 1): (0, 4),
            (33, 10007, 41, 0): (0, 3),    # 79, two CTAs per SM
            (128, 10007, 41, 0): (0, 1),   # the same, one
            (16, 8, 1, 1): (0, 1),         # a single block of depth
            (512, 4096, 64, 1): (128, 1),  # 64 tiles in one round
            (777, 1544, 81, 0): (192, 2),  # 36 tiles, as many clusters of two pairs
            (300, 9, 8192, 1): (128, 4),
            (8192, 12288, 64, 1): (256, 1)}
    assert dict(zip(want, plan(list(want)))) == want
