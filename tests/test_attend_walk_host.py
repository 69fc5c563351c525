"""The division of attention's work (csrc/attend_walk.cuh), compiled for the CPU and held against an enumeration: every unit's tiles are taken
once and in order, the runs are equal to within one, the keys of each row and the edges are right, and the CTAs of a cut unit are found."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include <vector>
#include "%s"
using namespace fp8gb::attend;
struct Src {
  std::vector<int> st, len;
  int tokens, capacity, seqs;
  Seq seq(int s) const { return seq_of(st[s], st[s + 1], len[s], tokens, capacity); }
};
int main() {
  int seqs, tokens, capacity, heads, per, window, ctas;
  while (scanf("%%d %%d %%d %%d %%d %%d %%d", &seqs, &tokens, &capacity, &heads, &per, &window, &ctas) == 7) {
    Src s;
    s.tokens = tokens, s.capacity = capacity, s.seqs = seqs;
    s.st.resize(seqs + 1), s.len.resize(seqs);
    for (int& x : s.st) if (scanf("%%d", &x) != 1) return 1;
    for (int& x : s.len) if (scanf("%%d", &x) != 1) return 1;
    long long total = 0;
    for (int i = 0; i < seqs; ++i) { Seq q = s.seq(i); for (int b = 0; b * per < q.n; ++b) total += (long long)heads * items_of(q, b, per, window); }
    int runs = total < ctas ? (int)total : ctas;
    printf("total %%lld\n", total);
    for (int c = 0; c < runs; ++c) {
      // the start, by walking
      Place at{0, 0, 0, 0, begin_of(total, c, runs), begin_of(total, c + 1, runs)};
      long long x = 0;
      bool found = false;
      for (int i = 0; i < seqs && !found; ++i) { Seq q = s.seq(i); for (int h = 0; h < heads && !found; ++h) for (int b = 0; b * per < q.n && !found; ++b) {
        int n = items_of(q, b, per, window);
        if (at.item < x + n) { at.seq = i, at.head = h, at.block = b, at.off = (int)(at.item - x), found = true; }
        x += n; } }
      for (Walk<Src> k(s, at, heads, per, window); k.live(); k.next()) {
        long long unit = k.at.item - k.at.off;
        Keys half = k.part_of(0, (per + 1) / 2);
        printf("%%d %%d %%d %%d %%d %%d %%d %%d %%d %%d %%d %%d %%d", c, k.at.seq, k.at.head, k.at.block, k.a, k.b, (int)k.first(), (int)k.last(), cta_of(total, unit, runs),
               cta_of(total, unit + k.items - 1, runs), k.filled, half.lo, half.hi);
        for (int t = k.a; t < k.b; ++t) printf(" %%d", (int)k.edge(t));
        printf("\n");
      }
    }
    printf("end\n");
  }
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("walk")
    (d / "w.cpp").write_text(SOURCE % os.path.join(ROOT, "fp8_mixed_precision_saturating_gb300", "csrc", "attend_walk.cuh"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", str(d / "w.cpp"), "-o", str(d / "w")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c[:7])) + "\n" + " ".join(map(str, c[7])) + "\n" + " ".join(map(str, c[8])) for c in cases)
        out = subprocess.run([str(d / "w")], input=text, capture_output=True, text=True, check=True).stdout
        return [block.strip().split("\n") for block in out.split("end\n")[:-1]]
    return run


def sequences(seqs, tokens, capacity, st, length):
    for s in range(seqs):
        first, end = min(max(st[s], 0), tokens), min(max(st[s + 1], 0), tokens)
        yield max(end - first, 0), max(length[s], 0)


def tiles(rows):
    """Tiles that any of the rows' key ranges touches, from the first row's beginning to the last one's end."""
    lo, hi = rows[0][0], rows[-1][1]
    return list(range(min(lo // 128, -(-hi // 128)), -(-hi // 128)))


def test_walks(walk):
    rng = random.Random(3)
    cases = []
    for _ in range(300):
        seqs, heads, per = rng.randint(1, 9), rng.randint(1, 4), rng.choice([1, 2, 5, 16, 42, 64, 128, 256])
        new = [rng.choice([0, 1, 1, rng.randint(0, 5), rng.randint(0, 700)]) for _ in range(seqs)]
        length = [n + rng.choice([-n - 3, -(n // 2), 0, 0, rng.randint(0, 40), rng.randint(0, 2000)]) for n in new]
        st = [0]
        for n in new:
            st.append(st[-1] + n)
        if rng.random() < 0.2:
            st[rng.randrange(seqs + 1)] += rng.randint(-400, 400)
        tokens = max(0, sum(new) + rng.choice([0, 0, 5, -3]))
        cases.append((seqs, tokens, rng.choice([128, 1024, 4096, 1 << 30]), heads, per, rng.choice([0, 0, 1, 100, 128, 1000]), rng.choice([1, 2, 7, 152]), st, length))
    for case, lines in zip(cases, walk(cases)):
        seqs, tokens, capacity, heads, per, window, ctas, st, length = case
        want = []  # (seq, head, block, tile or None, edge, tiles of the first half)
        for s, (n, total) in enumerate(sequences(seqs, tokens, capacity, st, length)):
            seen = min(total, capacity)
            rows = []
            for i in range(n):
                p = max(total - n + i, -1)
                rows.append((max(p + 1 - window, 0) if window else 0, min(p + 1, seen)))
            for h in range(heads):
                for b in range(-(-n // per)):
                    mine = rows[b * per:(b + 1) * per]
                    some = tiles(mine)
                    half = tiles(mine[:(per + 1) // 2])
                    for t in some or [None]:
                        edge = t is not None and any(lo > t * 128 or hi < t * 128 + 128 for lo, hi in mine)
                        want.append((s, h, b, t, edge, half, len(some) or 1))
        assert lines[0] == f"total {len(want)}"
        runs, got, filled, owner = {}, [], {}, {}
        half_of = {w[:4]: set(w[5]) for w in want}
        for line in lines[1:]:
            c, s, h, b, a, e, first, last, c0, c1, f, lo, hi, *edges = map(int, line.split())
            assert f == filled.get(c, 0)
            filled[c] = f + (a < e)
            owner.setdefault((s, h, b), []).append((c, first, last, c0, c1))
            for t, x in zip(range(a, e), edges):
                got.append((s, h, b, t, bool(x)))
                assert (lo <= t < hi) == (t in half_of[s, h, b, t])
            if a == e:
                got.append((s, h, b, None, False))
            runs[c] = runs.get(c, 0) + max(e - a, 1)
        assert got == [w[:5] for w in want]
        if want:
            assert len(runs) == min(ctas, len(want)) and max(runs.values()) - min(runs.values()) <= 1
        for parts in owner.values():
            assert [p[0] for p in parts] == list(range(parts[0][0], parts[-1][0] + 1))  # no CTA between them is without a part
            assert all(p[3:] == (parts[0][0], parts[-1][0]) for p in parts)
            assert [p[1] for p in parts] == [1] + [0] * (len(parts) - 1) and [p[2] for p in parts] == [0] * (len(parts) - 1) + [1]


def test_far_positions(walk):
    """Lengths near the end of 32 bits."""
    big = (1 << 31) - 1
    lines = walk([(1, 3, 0x7FFFFF00, 1, 2, 1, 2, [0, 3], [big]), (1, 3, 0x7FFFFF00, 1, 2, big, 1, [0, 3], [-big]), (1, 3, 1000, 1, 1, 300, 1, [0, 3], [big])])
    assert lines[0][0] == "total 2" and lines[1][0] == "total 2" and lines[2][0].startswith("total")
