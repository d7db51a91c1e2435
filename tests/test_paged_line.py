"""How mkv_paged_attention cuts the line of key blocks over the CTAs: the rule's own arithmetic (csrc/mkv_line.h, compiled
for the host) walked over every tile in turn."""
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "geometric_kv_cache_gb300", "csrc")
CTAS = 152
FEW, CHUNK = (CTAS, 1, 3, 3), (CTAS, 4, 6, 32)  # the rules of the two forms (CTAs, LineRule), for blocks of 128 keys

# Reads lines "ctas min_units slack uneven n len_1 .. len_n"; writes "units parts moved begin_0 .. begin_parts" and per tile of
# more than one part "tile first last" as part_of has them.
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "mkv_line.h"
using mkv::LineCut;
int main()
{
    int ctas, n;
    mkv::LineRule rule;
    while (std::scanf("%d %d %d %d %d", &ctas, &rule.min_units, &rule.slack, &rule.uneven, &n) == 5) {
        std::vector<int> len(n);
        int units = 0, tiles = 0;
        for (int &x : len) {
            if (std::scanf("%d", &x) != 1) return 1;
            units += x;
            tiles += x > 0;
        }
        const LineCut cut = LineCut::make(units, tiles, ctas, rule);
        std::vector<int> shift(cut.parts + 1, 0), begin(cut.parts + 1);
        const bool move = cut.hopeful();
        int off = 0;
        if (move)
            for (int x : len) {
                if (x > 0 && cut.movable(x))
                    for (int c = cut.part_from(off); c < cut.parts && cut.begin(c) < off + x; ++c)
                        shift[c] = LineCut::moved(cut.begin(c), off, x) - cut.begin(c);
                off += x;
            }
        int longest = 0;
        for (int c = 0; c < cut.parts; ++c) {
            const int l = cut.begin(c + 1) + shift[c + 1] - cut.begin(c) - shift[c];
            longest = l > longest ? l : longest;
        }
        const bool moved = move && cut.fits(longest);
        std::printf("%d %d %d", cut.units, cut.parts, (int)moved);
        for (int c = 0; c <= cut.parts; ++c) std::printf(" %d", cut.begin(c) + (moved ? shift[c] : 0));
        off = 0;
        for (int i = 0; i < n; off += len[i++])
            if (len[i] > 0) std::printf(" %d %d %d", i, cut.part_of(off), cut.part_of(off + len[i] - 1));
        std::printf("\n");
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("line")
    (d / "line.cc").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, "-o", str(d / "line"), str(d / "line.cc")],
                   check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, (*head, len(tiles), *tiles))) for head, tiles in cases)
        out = subprocess.run([str(d / "line")], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(cases)
        res = []
        for line in out:
            v = [int(x) for x in line.split()]
            res.append(dict(units=v[0], parts=v[1], moved=bool(v[2]), begin=v[3:4 + v[1]],
                            tiles=[tuple(v[i:i + 3]) for i in range(4 + v[1], len(v), 3)]))
        return res

    return run


def _parts(r):
    return [b - a for a, b in zip(r["begin"], r["begin"][1:])]


def test_any_line_is_covered_once_and_no_part_is_much_longer_than_its_share(cut):
    rng = random.Random(1)
    cases = []
    for _ in range(4000):
        most = rng.choice([1, 3, 10, 40, 3000, 40000])
        tiles = [rng.choice([0, 1, rng.randint(0, most), rng.randint(0, most)]) for _ in range(rng.choice([1, 5, 30, 152, 400]))]
        if rng.random() < 0.3:
            tiles = [most] * len(tiles)
        slack = rng.choice([0, 3, 6, 12])
        cases.append(((rng.choice([1, 7, 20, CTAS]), rng.choice([1, 4]), slack, rng.choice([slack, 32])), tiles))
    kinds = set()
    for (head, tiles), r in zip(cases, cut(cases)):
        ctas, min_units, slack, uneven = head
        units, parts = sum(tiles), r["parts"]
        assert r["units"] == units and 1 <= parts <= ctas
        assert r["begin"][0] == 0 and r["begin"][-1] == units and all(x >= 0 for x in _parts(r))
        longest = max(_parts(r))
        # equal parts, or none beyond its share by as much as the rule allows
        assert longest <= -(-units // parts) if not r["moved"] else (longest - units / parts) * ctas < uneven * parts
        kinds.add(r["moved"])
        # a cut tile's first and last part, as the joining code finds them
        off, held = 0, dict((i, (a, b)) for i, a, b in r["tiles"])
        for i, n in enumerate(tiles):
            if n:
                inside = [c for c in range(parts) if r["begin"][c] < off + n and r["begin"][c + 1] > off]
                if len(inside) > 1:
                    assert held[i] == (inside[0], inside[-1]) and inside == list(range(inside[0], inside[-1] + 1))
                    assert not r["moved"] or n > units // parts + slack
            off += n
    assert kinds == {False, True}


def test_largest_line(cut):
    for tiles in ([2 ** 31 - 1], [2 ** 30, 2 ** 30 - 1], [2 ** 23] * 200, [1] * 3 + [2 ** 31 - 4]):
        r, = cut([(FEW, tiles)])
        assert sum(_parts(r)) == sum(tiles) and max(_parts(r)) <= -(-sum(tiles) // CTAS) + 3


def _blocks(rng, n, lo, hi, keys):
    return [-(-rng.randint(lo, hi) // keys) for _ in range(n)]


@pytest.mark.parametrize("lists,lo,hi", [(152, 4096, 16384), (304, 4096, 16384), (144, 1024, 8192), (456, 500, 2000)])
@pytest.mark.parametrize("rule", [FEW, CHUNK])
def test_ragged_lists_as_many_as_the_ctas(cut, rule, lists, lo, hi):
    # whole tiles on average, but the longest are several times the shortest
    for seed in range(20):
        r, = cut([(rule, _blocks(random.Random(seed), lists, lo, hi, 128))])
        assert max(_parts(r)) < r["units"] / r["parts"] + rule[3]


@pytest.mark.parametrize("tokens,heads", [(2432, 8), (4864, 8), (608, 32), (16384, 8)])
def test_fresh_prompts(cut, tokens, heads):
    # 256 rows of a group of 4: 64 tokens to a tile, each list's tiles see ever more blocks of 128 keys
    tiles = [-(-64 * (i + 1) // 128) for i in range(tokens // 64)] * heads
    r, = cut([(CHUNK, tiles)])
    assert max(_parts(r)) < r["units"] / r["parts"] + CHUNK[3]


@pytest.mark.parametrize("rule,tiles,moved", [(FEW, [8] * 128, True), (CHUNK, [8] * 128, True), (FEW, [8] * 512, False),
                                              (CHUNK, [8] * 512, True), (CHUNK, [16] * 32, False), (FEW, [2] * 128, True)])
def test_equal_tiles_as_measured(cut, rule, tiles, moved):
    r, = cut([(rule, tiles)])
    assert r["moved"] == moved
    if moved:
        assert set(_parts(r)) <= {k * tiles[0] for k in range(10)}


def test_the_rules_here_are_the_kernels():
    few, chunk = (open(os.path.join(CSRC, f)).read() for f in ("mkv_attention.cu", "mkv_attention_chunk.cu"))
    assert "kLine = {%d, %d, %d};" % FEW[1:] in few
    assert "kSlackKeys = %d, kUnevenKeys = %d;" % (128 * CHUNK[2], 128 * CHUNK[3]) in chunk
    assert "kMinBlocks = %d;" % CHUNK[1] in chunk
