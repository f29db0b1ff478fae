"""Sizes of dit_text_attention at the corners of the documented ranges, without a GPU: every size
that the header allows gets an answer from the host-side plan, and a bounded one."""
import itertools
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A plan that dies takes the process with it, so the queries run in one of their own.
QUERY = """
import sys
from diffusion_transformer_step_gb300 import dit
for line in sys.stdin:
    print(dit.dit_text_attention_workspace(dit.make_text_attn(*map(int, line.split()))), flush=True)
"""


def _workspaces(cases):
    r = subprocess.run([sys.executable, "-c", QUERY], input="\n".join(" ".join(map(str, c)) for c in cases), text=True,
                       capture_output=True, cwd=ROOT)
    got = [int(x) for x in r.stdout.split()]
    assert r.returncode == 0 and len(got) == len(cases), (r.returncode, cases[len(got)], r.stderr[-500:])
    return got


@pytest.fixture(scope="module", autouse=True)
def built():
    from diffusion_transformer_step_gb300 import build_lib
    build_lib.build()


def test_sizes_whose_runs_pass_32_bits():
    """Longest keys x sequences x key heads x tiles of 16 rows at multiples of 2^46, where a run length
    of 32 bits would be zero, and from 2^45 on, where it would be negative."""
    got = _workspaces([(16384, 32, 8, 128, 1 << 21, 1 << 21, 1024, 1 << 21), (2048, 32, 8, 128, 1 << 21, 1 << 24, 1024, 1 << 24),
                       (16384, 1024, 1024, 64, 16384, 1 << 24, 1, 1 << 24), (16384, 512, 512, 64, 16384, 1 << 24, 1, 1 << 24)])
    # single tokens of so many sequences take one run each, which needs no parts
    assert got[2] == got[3] == 256


@pytest.mark.parametrize("heads_q,heads_k", [(1, 1), (64, 1), (44, 1), (32, 8), (1012, 23), (1024, 16), (1024, 1024)])
def test_workspace_at_the_corners(heads_q, heads_k):
    """Every combination of the smallest, ordinary and largest sizes.  The workspace is bounded: 16 bytes
    per pair of tiles of the list and its rows, 152 items' parts of 256 rows where keys are split over
    tiles, 32768 runs of 16 rows where they are split over runs."""
    cases = [(s, heads_q, heads_k, d, rq, rk, mq, mk) for s, d, rq, rk, mq, mk in itertools.product(
        (1, 63, 2048, 16384), (64, 128), (1, 4096, 1 << 28), (0, 1 << 21, 1 << 28), (1, 16, 1024, 1 << 24), (1, 1 << 21, 1 << 24))]
    for c, got in zip(cases, _workspaces(cases)):
        s, d, rq, mq = c[0], c[3], c[4], min(c[6], c[4])
        pairs = min(rq + s, s * -(-mq // 4))  # a pair of tiles holds four tokens or more
        parts = max(152 * 256, 32768 * 16) * (8 + 4 * d)
        assert 256 <= got <= 256 + 16 * pairs + parts + 1024, (c, got)
