// The division of the head's products among pairs of SMs, walked on the host (test_head_division.py).
#include <vector>

#include "zero_head.cuh"

using namespace zero;

// 0: every stage of every tile is one pair's once, tiles' places are all places once, parts have a
// place of their own inside the workspace, and the join adds exactly a tile's parts in order.
template <int PASS>
static int check(int counted, int cols, int columns, int pairs, int band)
{
    HeadArgs a{};
    a.cols = cols;
    a.count_v = columns;
    a.pairs = pairs;
    a.band = band;
    uint16_t some;
    a.dx = &some;
    const HeadShape s = head_shape<PASS>(a, counted);
    const uint32_t tiles = s.tm * s.tn, places = head_band<PASS>(a);
    // places that the workspace has: of the largest call of these sizes
    int64_t most = (int64_t)(tiles < ZERO_HD_PAIRS ? tiles : ZERO_HD_PAIRS) * (s.steps / ZERO_HD_PART);
    if (most > ZERO_HD_ROUNDS * ZERO_HD_PAIRS) most = ZERO_HD_ROUNDS * ZERO_HD_PAIRS;
    std::vector<uint8_t> seen((size_t)tiles * s.steps, 0), place(tiles, 0), slots(ZERO_HD_ROUNDS * ZERO_HD_PAIRS, 0);
    if (pairs > ZERO_HD_PAIRS || s.runs * s.run < s.steps || (PASS == HEAD_LOGITS && s.run > ZERO_HD_RUN)) return 1;
    for (uint32_t t = 0; t < tiles; t++) {
        uint32_t i, j;
        head_place(places, s, t, i, j);
        if (i >= s.tm || j >= s.tn || place[i * s.tn + j]++) return 2;
    }
    for (int p = 0; p < pairs; p++) {
        HeadSegment g;
        int within = 0;                              // runs of the tile so far
        uint32_t i = 0;
        for (; head_segment<PASS>(a, s, p, i, g); i++) {
            if (g.tile >= tiles || g.s0 < 0 || g.s1 <= g.s0 || g.s1 > (int)s.steps) return 3;
            for (int t = g.s0; t < g.s1; t++)
                if (seen[(size_t)g.tile * s.steps + t]++) return 4;
            if (g.first != (within == 0)) return 5;
            within = g.last ? 0 : within + 1;
            const bool whole = g.first && g.last && g.s0 == 0 && g.s1 == (int)s.steps;
            if (PASS >= HEAD_INPUT && (g.slot < 0) != whole) return 6;
            if (PASS < HEAD_INPUT && g.slot >= 0) return 6;
            if (g.slot >= 0 && (g.slot >= most || slots[g.slot]++)) return 7;
            if (g.slot >= 0) {                       // the join adds parts q, q + rest, ... of tile q in the axis's order
                const uint32_t q = g.tile - s.waves * a.pairs;
                if (g.tile < s.waves * a.pairs || g.slot % (int)s.rest != (int)q || g.slot / s.rest >= s.ranges) return 8;
                if (g.s0 != (int)(g.slot / s.rest * s.steps / s.ranges)) return 9;
            }
        }
        if (within) return 10;
        if (PASS == HEAD_INPUT && i != head_inputs(a, s, p)) return 13;
    }
    for (uint8_t n : seen)
        if (n != 1) return 11;
    // parts are cut only where the host launches the join
    if (PASS >= HEAD_INPUT && s.ranges > 1 && s.steps < 2 * ZERO_HD_PART) return 12;
    return 0;
}

extern "C" int head_check(int pass, int counted, int cols, int columns, int pairs, int band)
{
    switch (pass) {
    case HEAD_LOGITS: return check<HEAD_LOGITS>(counted, cols, columns, pairs, band);
    case HEAD_GRADIENT: return check<HEAD_GRADIENT>(counted, cols, columns, pairs, band);
    case HEAD_INPUT: return check<HEAD_INPUT>(counted, cols, columns, pairs, band);
    default: return check<HEAD_WEIGHT>(counted, cols, columns, pairs, band);
    }
}
