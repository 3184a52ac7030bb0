"""Where the join of shared-prefix attention reads a row's parts, for spans that clusters wrote and for
spans that nobody wrote (after a wait that ran out the workspace holds anything there)."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "indexed_sparse_attention_indexer_gb300", "csrc")
M = 128

PROGRAM = r"""
#include <stdio.h>
#include "prefix_parts.h"
// lines of: spans of both kinds, clusters of both launches, rows of the groups, query head, query heads,
// first own slot -> whether both spans hold, the number of parts, their places (the first 600)
int main() {
  int x0, y0, x1, y1, c0, c1, r0, r1, at, vectors, slot0;
  while (scanf("%d %d %d %d %d %d %d %d %d %d %d", &x0, &y0, &x1, &y1, &c0, &c1, &r0, &r1, &at, &vectors, &slot0) == 11) {
    const dsi::Span a(x0, y0, c0), b(x1, y1, c1);
    const int n = a.pieces + b.pieces;
    printf("%d %d", a.pieces > 0 && b.pieces > 0, n);
    for (int j = 0; j < n && j < 600; ++j)
      printf(" %lld", (long long)dsi::part_place(a, b, j, r0, r1, at, vectors, slot0, 128));
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    at = tmp_path_factory.mktemp("parts")
    (at / "parts.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(at / "parts.cpp"), "-o", str(at / "parts")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        got = subprocess.run([str(at / "parts")], input=text, capture_output=True, text=True, check=True)
        lines = [[int(v) for v in line.split()] for line in got.stdout.splitlines()]
        assert len(lines) == len(cases)
        return lines
    return run


def test_written_spans(places):
    """Whole groups stand in the rows' places; pieces in the first slot of a cluster but for the one
    that starts the group, which has the second."""
    got = places([(3, 3, 5, 5, 8, 8, 17, 40, 6, 100, 0),
                  (3, 5, 0, 0, 8, 8, 17, 40, 6, 100, 0),
                  (0, 0, 6, 7, 8, 8, 17, 40, 6, 100, 0),
                  (0, 75, 10, 12, 76, 70, 1, 127, 0, 1, 152)])
    assert got[0] == [1, 2, -7, -107]
    assert got[1] == [1, 4, 7 * M + 17, 8 * M + 17, 10 * M + 17, -107]
    assert got[2] == [1, 3, -7, 13 * M + 40, 14 * M + 40]
    first = [(2 * k + (k == 0)) * M + 1 for k in range(76)]
    assert got[3] == [1, 79] + first + [(152 + 21) * M + 127, (152 + 22) * M + 127, (152 + 24) * M + 127]


def test_unwritten_spans(places):
    """Whatever the spans hold, no place lies outside the workspace and no row has more parts than clusters."""
    rng = random.Random(7)
    edge = [-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 75, 76, 77, 0x3f800000, 0x7fc00000, 2 ** 31 - 2, 2 ** 31 - 1]
    cases = []
    for _ in range(4000):
        slots = rng.choice([1, 2, 76, 128])
        c = [rng.randint(1, slots), rng.randint(1, slots)]
        value = lambda: (rng.randint(0, slots) if rng.random() < 0.8 else                      # noqa: E731
                         rng.choice([rng.choice(edge), rng.randint(-2 ** 31, 2 ** 31 - 1)]))
        vectors = rng.choice([1, 64, 2 ** 30 - 1])
        cases.append((value(), value(), value(), value(), *c, rng.randrange(M), rng.randrange(M), rng.randrange(vectors),
                      vectors, rng.choice([0, 2 * slots])))
    refused = 0                                # (both kinds are drawn)
    for case, (ok, n, *at) in zip(cases, places(cases)):
        x0, y0, x1, y1, c0, c1, _, _, _, vectors, slot0 = case
        good = [0 <= x <= y < c for x, y, c in ((x0, y0, c0), (x1, y1, c1))]
        assert ok == all(good) and n == len(at) == good[0] * (y0 - x0 + 1) + good[1] * (y1 - x1 + 1)
        most = max(2 * c0, slot0 + 2 * c1) * M
        assert all(-2 * vectors <= p < most for p in at), case
        refused += not ok
    assert 1000 < refused < 4000
