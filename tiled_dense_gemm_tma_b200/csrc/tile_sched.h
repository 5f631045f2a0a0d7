// tile_sched.h -- work-distribution arithmetic shared by the kernels and their
// launchers: the stream-K split of the weight-streaming kernels, the grouped
// tile raster of the persistent kernels, and the split-K ranges of the fp32
// FFMA kernel.  Plain C++ with no CUDA types, so that the host tests build it
// with g++ and check every partition it produces.
#pragma once

#if defined(__CUDACC__)
#define TG_HD __host__ __device__ __forceinline__
#else
#define TG_HD inline
#endif

namespace tg {

TG_HD int sched_min(int a, int b) {
#if defined(__CUDA_ARCH__)
    return min(a, b);
#else
    return a < b ? a : b;
#endif
}

TG_HD int sched_max(int a, int b) {
#if defined(__CUDA_ARCH__)
    return max(a, b);
#else
    return a > b ? a : b;
#endif
}

// ---------------------------------------------------------------- stream-K
// U work units (column group t owns units [t*KB, t*KB + KB)) are cut into G
// contiguous ranges, CTA c taking [sk_begin(c), sk_begin(c + 1)).  Range
// sizes are floor(U/G) or ceil(U/G); with G <= U none is empty.

TG_HD int sk_begin(int c, int U, int G) {
    return static_cast<int>((static_cast<long long>(c) * U) / G);
}

// CTA whose range holds unit u (0 <= u < U).  When G > U some ranges are
// empty; the owner is the one non-empty range that holds u.  The first guess
// floor(u*G/U) never lies past the owner (its range starts at or before u),
// so the upward step does the work; the downward one only guards the guess.
TG_HD int sk_owner(int u, int U, int G) {
    int c = static_cast<int>((static_cast<long long>(u) * G) / U);
    while (c + 1 < G && sk_begin(c + 1, U, G) <= u) ++c;
    while (c > 0 && sk_begin(c, U, G) > u) --c;
    return c;
}

// Launch plan of a weight-streaming kernel: T column groups of gn columns,
// KB k-units of bk rows each, U = T*KB units over G = min(U, num_sms) CTAs,
// and J = the most ranges (segments) any one column group is cut into, which
// sizes its split-K partial slots.
struct SkPlan {
    long long T, KB, U, G, J;
};

// False when U does not fit the kernels' int unit indices.
inline bool sk_plan(long long N, long long K, int gn, int bk, int num_sms, SkPlan* p) {
    p->T = (N + gn - 1) / gn;
    p->KB = (K + bk - 1) / bk;
    p->U = p->T * p->KB;
    if (p->U > 0x7fffffffll) return false;
    p->G = p->U < num_sms ? p->U : num_sms;
    p->J = 1;
    const int U = static_cast<int>(p->U), G = static_cast<int>(p->G);
    for (long long t = 0; t < p->T; ++t) {
        const long long n = sk_owner(static_cast<int>(t * p->KB + p->KB - 1), U, G) -
                            sk_owner(static_cast<int>(t * p->KB), U, G) + 1;
        if (n > p->J) p->J = n;
    }
    return true;
}

// ------------------------------------------------- split-K inside a cluster
// The alternative to stream-K when T column groups times a small split S
// fill the GPU: group t goes to the S CTAs of cluster t, and rank r of the
// cluster takes the k-units [t*KB + cl_begin(r), t*KB + cl_begin(r + 1)).
// The ranks then sum their partials through distributed shared memory, each
// rank owning gn/S columns of the group.

TG_HD int cl_begin(int r, int KB, int S) {
    return static_cast<int>((static_cast<long long>(r) * KB) / S);
}

// The split S in {8, 4, 2, 1} for T groups of gn columns and KB k-units, or 0
// (use stream-K): the largest S with no empty range (S <= KB), whole 32-column
// warp slices per owner (gn a multiple of 32*S), T*S <= cap CTAs, and T*S at
// least three quarters of num_sms (fewer CTAs would leave HBM bandwidth
// unused).  `max_s` bounds S (a smaller maximum cluster on the device).
inline int cl_split(long long T, long long KB, int gn, long long cap, int num_sms, int max_s) {
    for (int S = 8; S >= 1; S >>= 1) {
        if (S > max_s || S > KB || gn % (32 * S) != 0 || T * S > cap) continue;
        return T * S * 4 >= 3ll * num_sms ? S : 0;
    }
    return 0;
}

// ------------------------------------------- hybrid schedule of the pairs
// The persistent CTA-pair kernel hands out work items round-robin to its
// npairs pairs.  Whole tiles fill the full waves; when the R tiles left for
// the last wave would leave at least half of the pairs idle (2R <= npairs),
// each of them is split into two halves of its k-blocks, so the last wave
// takes about half a tile's time.  tail_dp() is the number of items that
// are whole tiles (all tiles when there is no split).

TG_HD int tail_split(int num_tiles, int npairs, int num_kb) {
    const int R = num_tiles % npairs;
    return (R > 0 && 2 * R <= npairs && num_kb >= 2) ? 2 : 1;
}

TG_HD int tail_dp(int num_tiles, int npairs, int S) {
    return S > 1 ? num_tiles - num_tiles % npairs : num_tiles;
}

TG_HD int tail_items(int num_tiles, int dp, int S) { return dp + (num_tiles - dp) * S; }

// Item w -> tile t, k-blocks [kb0, kb1), and the half z (-1 for a whole tile).
TG_HD void tail_item(int w, int dp, int S, int num_kb, int& t, int& kb0, int& kb1, int& z) {
    if (S <= 1 || w < dp) {
        t = w;
        kb0 = 0;
        kb1 = num_kb;
        z = -1;
        return;
    }
    const int i = (w - dp) / S;
    z = (w - dp) - i * S;
    t = dp + i;
    kb0 = static_cast<int>((static_cast<long long>(z) * num_kb) / S);
    kb1 = static_cast<int>((static_cast<long long>(z + 1) * num_kb) / S);
}

// ------------------------------------------------------------ tile raster
// Linear tile index t of an ntm x ntn tile grid -> (tm, tn).  Tiles are taken
// in bands of group_m tile rows (the last band may be shorter); inside a band
// the index runs down the rows of one tile column, then to the next column,
// so CTAs working at the same time share the band's A rows and a few B
// columns in L2.
TG_HD void tile_coords(int t, int ntm, int ntn, int group_m, int& tm, int& tn) {
    const int per_group = group_m * ntn;
    const int g = t / per_group;
    const int first_m = g * group_m;
    const int gsz = sched_min(ntm - first_m, group_m);
    const int local = t - g * per_group;
    tm = first_m + local % gsz;
    tn = local / gsz;
}

// ------------------------------------------------------ groups of rows
// The experts' products: a group of `rows` > 0 consecutive rows is cut into
// grp_tiles(rows) tiles, as few as 256 rows a tile allow.  An MMA takes
// widths in units of 32 rows: the group's units are dealt out evenly, so that
// no more than the last unit is padding (1348 rows are 256 + 5 x 224, not
// 6 x 256, nor 5 x 256 + 96).

TG_HD int grp_tiles(int rows) { return (rows - 1) / 256 + 1; }

// Tile i of the group: its first row in the group and its MMA width (a
// multiple of 32, at most 256; the last tile may hold fewer rows).  `tiles`: how
// many there are where that is not grp_tiles(rows), from it to rows / 32.
TG_HD void grp_tile(int rows, int i, int& at, int& width, int tiles = 0) {
    const int nt = tiles ? tiles : grp_tiles(rows), units = (rows - 1) / 32 + 1;
    const int each = units / nt, more = units - each * nt;     // the first `more` tiles take one more
    at = 32 * (i * each + sched_min(i, more));
    width = 32 * (each + (i < more ? 1 : 0));
}

// The last wave of T tiles on npairs pairs: where its R = T mod npairs tiles
// leave at least half (three quarters) of the pairs idle, each is cut into 2
// (at most `most`: 4) narrower ones, pieces of at least 64 rows.  The pieces
// of a tile add the same terms in the same order as the whole one.
TG_HD int grp_pieces(int T, int npairs, int most) {
    const int R = T % npairs;
    return R == 0 ? 1 : (most >= 4 && 4 * R <= npairs) ? 4 : 2 * R <= npairs ? 2 : 1;
}

// Width of the pieces of a tile of `width` rows (a multiple of 32).
TG_HD int grp_piece_width(int width, int pieces) {
    const int w = ((width - 1) / pieces + 32) / 32 * 32;
    return w < 64 ? sched_min(64, width) : w;
}

// Clocks of a 256-byte-deep stage of a tile of `width` rows of 4-bit products, as
// measured: its MMAs and what a stage costs besides, or the time that five stages
// in flight take to come round.
TG_HD int mx4_stage_clocks(int width) { return sched_max(2 * width + 70, sched_min(500, 372 + width)); }

// Row tiles of one group of all rows, a known number of them: as many as make
// the waves of tiles over npairs pairs take the least time, if that is a
// twentieth less than with the fewest.  1536 rows on 20 column tiles: 7 tiles of up
// to 224 rows (140 on 74 pairs, two waves) and not 6 of 256 (120, two waves):
// 26.6 -> 24.6 us with 4096 columns.
inline int mx4_even_tiles(long long rows, long long ntl, int npairs) {
    const long long least = (rows - 1) / 256 + 1, units = (rows - 1) / 32 + 1;
    long long best = least, cost = -1;
    if (least * ntl >= 16ll * npairs) return static_cast<int>(least);     // one wave of many
    for (long long nt = least; nt <= least + least / 3 + 1 && nt <= units; ++nt) {
        const int width = static_cast<int>(32 * ((units - 1) / nt + 1));
        const long long tiles = nt * ntl, rest = tiles % npairs;
        long long c = tiles / npairs * mx4_stage_clocks(width);
        if (rest) c += mx4_stage_clocks(grp_piece_width(width, grp_pieces(static_cast<int>(rest), npairs, 4)));
        if (cost < 0 || c < (best == least ? cost - cost / 20 : cost)) {
            cost = c;
            best = nt;
        }
    }
    return static_cast<int>(best);
}

// Rows [r0, r1) of group e from the offsets (ng + 1 of them), clamped to
// 0 <= r0 <= r1 <= M so that no offset leads outside the matrices; group ng
// is the rows behind the last one.
TG_HD void grp_rows(const int* offsets, int e, int ng, int M, int& r0, int& r1) {
    if (!offsets) {                        // one group of all rows
        r0 = e == 0 ? 0 : M;
        r1 = M;
        return;
    }
    r0 = sched_min(sched_max(offsets[e], 0), M);
    r1 = e < ng ? sched_min(sched_max(offsets[e + 1], r0), M) : M;
}

// ------------------------------------------------------- fp32 split-K
// Number of k ranges per output tile: 1 when the tiles already fill the SMs;
// otherwise enough to fill them, with at most 8 ranges and no more ranges than
// kb_all / 8 (so a range averages at least 8 k-slices).
inline int ffma_splits(long long tiles, long long kb_all, int num_sms) {
    long long s = 1;
    if (tiles < num_sms) {
        s = num_sms / tiles;
        if (s > kb_all / 8) s = kb_all / 8;
        if (s > 8) s = 8;
        if (s < 1) s = 1;
    }
    return static_cast<int>(s);
}

// Split-K ranges over kb_all k-slices: range z is [z * kb_per, z * kb_per +
// ffma_range_len(z * kb_per, kb_per, kb_all)), kb_per = ffma_kb_per(kb_all,
// splits) = ceil(kb_all / splits).  Every range is kb_per long except a
// shorter last one, which is never empty for a split count from ffma_splits.
TG_HD int ffma_kb_per(int kb_all, int splits) { return (kb_all + splits - 1) / splits; }

TG_HD int ffma_range_len(int kb0, int kb_per, int kb_all) {
    return sched_max(0, sched_min(kb_all, kb0 + kb_per) - kb0);
}

}  // namespace tg
