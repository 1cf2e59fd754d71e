"""What the merge of cut units accepts, on the CPU: its workspace may hold anything where a wait gave up before a stretch
wrote its entry, and an entry that names no pieces or no head must not be followed.  The kernel's own test is compiled
for the host."""

import subprocess

import numpy as np
import pytest

from flashattention_attention_attn_b200 import build

SOURCE = r"""
#include <cstdio>
#include "prefill_fp8_sm100.cuh"
// lines of: stretch, kv heads, c0, hk, qoff, tok0, T
int main() {
  int c1, heads;
  attn::prefill8::Cut c;
  while (std::scanf("%d %d %d %d %d %d %d", &c1, &heads, &c.c0, &c.hk, &c.qoff, &c.tok0, &c.T) == 7)
    std::printf("%d\n", attn::prefill8::cut_ends_here(c, c1, heads) ? 1 : 0);
}
"""


@pytest.fixture(scope="module")
def ends_here(tmp_path_factory):
    at = tmp_path_factory.mktemp("merge")
    (at / "cut.cu").write_text(SOURCE)
    subprocess.run([build.nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1",
                    "--expt-relaxed-constexpr", "-I", build.CSRC, "-I", build.INCLUDE, "-o", str(at / "cut"),
                    str(at / "cut.cu")], check=True, capture_output=True)

    def call(rows):
        text = "\n".join(" ".join(str(int(x)) for x in r) for r in rows)
        out = subprocess.run([str(at / "cut")], input=text, capture_output=True, text=True, check=True)
        return [int(x) for x in out.stdout.split()]

    return call


def test_merge_follows_only_entries_whose_pieces_and_head_exist(ends_here):
    assert ends_here([(5, 8, -1, 0, 0, 0, 0),          # ends no cut unit
                      (5, 8, 0, 0, 0, 0, 70), (5, 8, 4, 7, 100, 64, 300), (1, 1, 0, 0, 0, 0, 1)]) == [0, 1, 1, 1]
    assert ends_here([(5, 8, 5, 0, 0, 0, 70), (5, 8, 6, 0, 0, 0, 70),          # no piece before this stretch
                      (5, 8, 0, 8, 0, 0, 70), (5, 8, 0, -1, 0, 0, 70),         # no such head
                      (0, 8, 0, 0, 0, 0, 70), (5, 8, -2 ** 31, 3, 0, 0, 70)]) == [0] * 6


def test_whatever_the_workspace_held_stays_inside_it(ends_here):
    """Random bits as entries: where the merge goes on, the slots it reads and the head it writes exist."""
    r = np.random.default_rng(0)
    rows = []
    for _ in range(4000):
        heads, c1 = int(r.integers(1, 9)), int(r.integers(0, 148))
        cut = [int(x) for x in r.integers(-2 ** 31, 2 ** 31, 5)]
        if r.random() < 0.7:  # small numbers too, so that some entries pass
            cut[:2] = [int(x) for x in r.integers(-3, 12, 2)]
        rows.append((c1, heads, *cut))
    got = ends_here(rows)
    assert len(got) == len(rows) and 0 < sum(got) < len(rows)
    for ok, (c1, heads, c0, hk, *_) in zip(got, rows):
        assert ok == (0 <= c0 < c1 and 0 <= hk < heads)
