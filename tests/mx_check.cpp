// Host checks of the arithmetic behind routing and the 4-bit products: each entry
// point counts what it checked in *checked and returns how many checks failed.
// Built with g++ by test_mxfp4_host.py.
#include "route.h"
#include "tile_sched.h"

#include <algorithm>
#include <vector>

using namespace tg;

extern "C" {

float slack(int sigmoid, float highest, float size, int values) { return route_slack(sigmoid, highest, size, values); }

// Row tiles of one group in any number that mx4_even_tiles gives: they tile the
// rows in order, in widths an MMA takes, and cost no more than the fewest do.
long long check_even_tiles(long long* checked) {
    long long bad = 0, n = 0;
    for (long long rows : {1, 31, 32, 129, 200, 256, 257, 500, 1000, 1536, 3000, 4096, 8192, 100000, 2147482623})
        for (long long ntl : {1, 2, 5, 20, 32, 74, 300})
            for (int np : {1, 66, 74}) {
                const int nt = mx4_even_tiles(rows, ntl, np);
                const long long units = (rows - 1) / 32 + 1;
                ++n; bad += nt < grp_tiles(static_cast<int>(rows)) || nt > units;
                if (rows > 100000) continue;
                int end = 0;
                for (int t = 0; t < nt; ++t) {
                    int at, w;
                    grp_tile(static_cast<int>(rows), t, at, w, nt);
                    ++n; bad += at != end || w % 32 != 0 || w < 32 || w > 256 || at >= rows;
                    end = at + w;
                }
                ++n; bad += end < rows || end - rows >= 32;
            }
    ++n; bad += mx4_even_tiles(1536, 20, 74) != 7 || mx4_even_tiles(8192, 32, 74) != 32;
    *checked = n;
    return bad;
}

// How a warp's lanes share a row: every expert in one lane, in order of lanes,
// a group in lanes of its own; at most 64 to a lane.
long long check_route_lanes(long long* checked) {
    long long bad = 0, n = 0;
    for (int groups = 1; groups <= 32; ++groups)
        for (int per = 1; per * groups <= 1024; ++per) {
            const int lanes = route_lanes(groups), v = route_values(per * groups, groups);
            int V = 1;
            while (V < v) V *= 2;
            ++n; bad += lanes < 1 || (lanes & (lanes - 1)) != 0 || lanes * groups > 32 || V > 64;
            int next = 0;
            for (int lane = 0; lane < 32; ++lane) {
                const int group = lane / lanes, off = lane % lanes * V, first = group * per + off;
                const int live = group < groups ? std::max(0, std::min(V, per - off)) : 0;
                for (int i = 0; i < live; ++i) { ++n; bad += first + i != next++; }
            }
            ++n; bad += next != per * groups;
        }
    *checked = n;
    return bad;
}

// Where a warp puts the scale words of 128 rows (order_scales): reading row
// behind row and writing word behind word, lane i's 16 bytes of word w are those of
// rows i, 32 + i, 64 + i and 96 + i.
long long check_scale_places(long long* checked) {
    long long bad = 0, n = 0;
    for (int Q : {1, 2}) {
        std::vector<int> tile(128 * 4 * Q), out(128 * 4 * Q, -1);      // words
        for (int r = 0; r < 128; ++r)
            for (int w = 0; w < 4 * Q; ++w) tile[r * 4 * Q + w] = r * 100 + w;
        for (int lane = 0; lane < 32; ++lane)
            for (int c = 0; c < 4; ++c)
                for (int h = 0; h < Q; ++h)
                    for (int j = 0; j < 4; ++j)
                        out[((4 * h + j) * 512 + lane * 16) / 4 + c] = tile[((32 * c + lane) * 16 * Q + 16 * h) / 4 + j];
        for (int w = 0; w < 4 * Q; ++w)
            for (int lane = 0; lane < 32; ++lane)
                for (int c = 0; c < 4; ++c) { ++n; bad += out[w * 128 + lane * 4 + c] != (32 * c + lane) * 100 + w; }
    }
    *checked = n;
    return bad;
}

}  // extern "C"
