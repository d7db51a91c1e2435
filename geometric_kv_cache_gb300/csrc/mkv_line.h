// Where the line of key blocks of mkv_paged_attention is cut (internal; plain
// arithmetic for host and device, so that it can be tested without a GPU).
//
// All tiles' units stand on one line, tile after tile. Part c of `parts` equal
// ones begins at floor(c units / parts). Where whole tiles, of which some CTAs
// get more than others, cost less than equal parts, the cuts move to the nearer
// ends of their tiles (not in tiles longer than a part and the slack): the parts
// of cut tiles have to be begun, written, read and joined. Both an average and the
// longest part decide: lists of uneven length can pass for whole tiles on average
// and leave one CTA 1.7 times its share.
// Measured (us, equal parts / whole tiles, 128 dims, bf16, blocks of 128 keys):
// equal tiles: 128 of 8 blocks, 16 rows 21 / 15.5, 256 rows 49 / 30; 512 of 8, 16 rows
// 61 / 66.5 (5 blocks more), 256 rows 113 / 102; 32 of 16, 256 rows 30 / 44 (12 more);
// lists of uneven length, one row: 152 of 4K-16K tokens 130 / 191 (longest part 49 to 68
// blocks more), 304 of them 240 / 310; 256 rows: the 152 194 / 260, 304 of 1K-4K 136 / 132
// (about 20 more), 152 of 2K-8K 146 / 145 (22 to 35), 304 of 2K-8K 205 / 222 (about 40);
// triangles of fresh prompts, 8 lists: 2432 tokens 105 / 91 (14 more), 4864 263 / 242 (26).
// (9728 tokens, 49 more, are 728 / 698: their longest parts are those with the fewest
// tiles to begin, which the rule does not see.) Looking at the longest part takes 0.3 to
// 0.5 us where the average allows whole tiles, 2 us over more tiles than threads.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MKV_HD __host__ __device__ __forceinline__
#else
#define MKV_HD inline
#endif

namespace mkv {

// slack: the units by which a CTA may have more than its share before joining
// costs less, with tiles of equal length (less where fewer parts would be
// joined). uneven: the same for the longest part that moved cuts really leave.
struct LineRule {
    int min_units;  // least units of a part while there are fewer tiles than CTAs
    int slack, uneven;
};

struct LineCut {
    int units, tiles;  // the line's length, the tiles on it
    int ctas, parts;   // parts <= ctas <= 512
    LineRule rule;
    int share, rest;   // units / parts and what is left
    uint32_t over;     // ceil(2^32 / parts), the one division: every CTA does this before it can begin

    // n / parts (the estimate is at most one too high)
    MKV_HD int by_parts(int n) const
    {
        const uint32_t q = parts == 1 ? (uint32_t)n : (uint32_t)((uint64_t)over * (uint32_t)n >> 32);
        return (int)(q - (q * (uint32_t)parts > (uint32_t)n ? 1u : 0u));
    }
    static MKV_HD LineCut make(int units, int tiles, int ctas, LineRule rule)
    {
        LineCut k;
        k.units = units;
        k.tiles = tiles;
        k.ctas = ctas;
        k.rule = rule;
        const int want = units / rule.min_units > tiles ? units / rule.min_units : tiles;
        k.parts = want < 1 ? 1 : want < ctas ? want : ctas;
        k.over = 0xFFFFFFFFu / (uint32_t)k.parts + 1u;  // (0 for one part)
        k.share = k.by_parts(units);
        k.rest = units - k.share * k.parts;
        return k;
    }
    MKV_HD int begin(int c) const
    {
        if (c >= parts) return units;
        return share * c + (int)((uint64_t)over * (uint32_t)(rest * c) >> 32);  // (exact: rest c < 2^18)
    }
    // The lowest part that begins at unit u or later. (The estimates here are off by less than one part.)
    MKV_HD int part_from(int u) const
    {
        int c = (int)((float)u * (float)parts / (float)units) - 1;
        for (c = c < 0 ? 0 : c; c < parts && begin(c) < u; ++c) {}
        return c;
    }
    // The part (of equal ones) that unit u is in.
    MKV_HD int part_of(int u) const
    {
        int c = (int)((float)u * (float)parts / (float)units) + 1;
        for (c = c < parts ? c : parts - 1; begin(c) > u; --c) {}
        return c;
    }
    // Whether moved cuts cost less, going by tiles of average length, none of them cut.
    MKV_HD bool hopeful() const
    {
        const int last = tiles - by_parts(tiles) * parts, idle = last > 0 ? parts - last : 0;  // places for a tile that stay empty
        return (long long)idle * units * ctas < (long long)rule.slack * tiles * parts * parts;
    }
    // Whether they do, going by the longest part that they leave.
    MKV_HD bool fits(int longest) const
    {
        return ((long long)longest * parts - units) * ctas < (long long)rule.uneven * parts * parts;
    }
    MKV_HD bool movable(int len) const { return len <= share + rule.slack; }  // the cuts in a tile of len units
    // Where the cut at u in the tile [off, off + len) moves to.
    static MKV_HD int moved(int u, int off, int len) { return 2 * (u - off) < len ? off : off + len; }
};

}  // namespace mkv
