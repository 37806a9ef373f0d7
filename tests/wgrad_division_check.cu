// wgrad_division_check.cu -- test helper (built by tests/test_wgrad_division.py): the weight
// gradient's division of work, walked on the host, against the workspace that a caller is told to
// bring.  Nothing here runs on a GPU.
#include "zero_wgrad.cu"

// Bytes of the workspace up to the end of the farthest slot that a call keeps sums in (those
// before the slots if it keeps none), for a device of `pairs` pairs.  *stages: how often the
// segments cover the tiles' stages (tiles x stages if each once, in order), -1 if a tile's or
// part's runs do not follow one another.
extern "C" uint64_t wgrad_reach(int64_t tokens, int64_t n, int64_t k, int grad_dtype, int pairs, int64_t* stages,
                                int* longest_run)
{
    WgradArgs a{};
    a.tokens = tokens;
    a.n = n;
    a.k = k;
    a.grad_dtype = grad_dtype;
    divide(a, pairs);
    int64_t far = 0;
    bool good = true;
    *stages = 0;
    *longest_run = 0;
    for (int pair = 0; pair < (a.waves > 0 ? a.pairs : a.rest_pairs); pair++) {
        WgradSegment g, last{};
        last.last = true;
        for (uint32_t i = 0; wgrad_segment(a, (uint32_t)pair, i, g); i++) {
            *stages += g.s1 - g.s0;
            if (g.s1 - g.s0 > *longest_run) *longest_run = g.s1 - g.s0;
            good = good && g.s1 > g.s0 && g.s1 <= a.steps && g.tile < a.tiles_n * a.tiles_k && g.first == last.last;
            if (!g.first) good = good && g.tile == last.tile && g.slot == last.slot && g.s0 == last.s1;
            if (wgrad_kept(g) && wgrad_slot(g, (uint32_t)pair) + 1 > far) far = wgrad_slot(g, (uint32_t)pair) + 1;
            last = g;
        }
        good = good && last.last;
    }
    if (!good) *stages = -1;
    return (uint64_t)(256 + sums_bytes(n) + far * ZERO_WG_SLOT * 4);
}
