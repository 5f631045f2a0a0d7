// Host checks of the group arithmetic of tile_sched.h: each entry point walks
// a parameter grid, counts what it checked in *checked and returns how many
// checks failed.  Built with g++ by test_group_sched_host.py.
#include "tile_sched.h"

#include <algorithm>
#include <vector>

using namespace tg;

extern "C" {

// The row tiles of a group, whole or in pieces: they tile [0, rows) in order,
// whole ones are not empty, widths are multiples of 32 in [32, 256] as an MMA
// takes them, their sum pads less than 32 rows, and pieces are no wider than
// their tile.
long long check_group_tiles(int max_rows, long long* checked) {
    long long bad = 0, n = 0;
    for (int rows = 1; rows <= max_rows; ++rows) {
        const int nt = grp_tiles(rows);
        ++n; bad += nt != (rows + 255) / 256;
        for (int pieces : {1, 2, 4}) {
            int end = 0, sum = 0;
            for (int t = 0; t < nt; ++t) {
                int at, w;
                grp_tile(rows, t, at, w);
                ++n; bad += w % 32 != 0 || w < 32 || w > 256 || at >= rows || at != sum;
                sum += w;
                const int pw = grp_piece_width(w, pieces);
                ++n; bad += pw % 32 != 0 || pw < 32 || pw > w || pw * pieces < w;
                // as the kernel walks them
                const int m1 = std::min(rows, at + w);
                for (int i = 0; i < pieces; ++i) {
                    const int a = at + i * pw, b = std::min(m1, a + pw);
                    if (a >= b) continue;
                    ++n; bad += a != end;
                    end = b;
                }
            }
            ++n; bad += end != rows || sum - rows >= 32;
        }
    }
    *checked = n;
    return bad;
}

// Large row counts: no overflow.
long long check_group_large(long long* checked) {
    long long bad = 0, n = 0;
    for (int rows : {2147483647, 2147483393, 1 << 30}) {
        const int nt = grp_tiles(rows);
        ++n; bad += nt != static_cast<int>((static_cast<long long>(rows) + 255) / 256);
        for (int t : {0, 1, nt / 2, nt - 1}) {
            int at, w;
            grp_tile(rows, t, at, w);
            ++n; bad += at < 0 || at >= rows || (w != 256 && w != 224);
        }
    }
    *checked = n;
    return bad;
}

// The schedule of T tiles on npairs pairs: every tile once, whole before dp,
// all its pieces after; pieces only where they fit one wave.
long long check_group_schedule(int max_tiles, int max_pairs, long long* checked) {
    long long bad = 0, n = 0;
    for (int np = 1; np <= max_pairs; ++np)
        for (int T = 1; T <= max_tiles; ++T)
            for (int most : {2, 4}) {
                const int pieces = grp_pieces(T, np, most);
                const int dp = tail_dp(T, np, pieces), items = tail_items(T, dp, pieces);
                ++n; bad += pieces < 1 || pieces > most;
                if (pieces > 1) { ++n; bad += dp % np != 0 || items - dp > np || items <= dp; }
                std::vector<int> seen(T, 0);
                for (int i = 0; i < items; ++i) {
                    const int w = i < dp ? i : dp + (i - dp) / pieces;
                    ++n; bad += w < 0 || w >= T;
                    if (w >= 0 && w < T) seen[w] += i < dp ? pieces : 1;
                }
                for (int c : seen) { ++n; bad += c != pieces; }
            }
    *checked = n;
    return bad;
}

// Rows of groups from any offsets: inside [0, M], in order; from proper ones
// exactly theirs, and the rows behind the last group as one more.
long long check_group_rows(long long* checked) {
    long long bad = 0, n = 0;
    const int lo = -2147483647 - 1, hi = 2147483647;
    for (int M : {1, 5, 100, hi})
        for (int a : {lo, -1, 0, 3, 100, hi})
            for (int b : {lo, 0, 4, 50, hi}) {
                const int off[3] = {a, b, a};
                for (int e = 0; e <= 2; ++e) {
                    int r0, r1;
                    grp_rows(off, e, 2, M, r0, r1);
                    ++n; bad += r0 < 0 || r1 < r0 || r1 > M;
                }
            }
    const int off[4] = {0, 3, 3, 9};
    const int want[4][2] = {{0, 3}, {3, 3}, {3, 9}, {9, 12}};
    for (int e = 0; e <= 3; ++e) {
        int r0, r1;
        grp_rows(off, e, 3, 12, r0, r1);
        ++n; bad += r0 != want[e][0] || r1 != want[e][1];
        grp_rows(nullptr, e > 0, 1, 12, r0, r1);
        ++n; bad += r0 != (e ? 12 : 0) || r1 != 12;
    }
    *checked = n;
    return bad;
}

}  // extern "C"
