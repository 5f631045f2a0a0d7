// Host check of the weight gradient's k blocks (tile_sched.h), built with g++
// by test_group_window_host.py.
#include "tile_sched.h"

#include <vector>

using namespace tg;

extern "C" {

// What the kernel's copies and MMA steps make of groups of 1 to max_rows
// rows: a box of 64 rows starts z = grp_zero_rows rows before the window of 64
// rows that begins at the block's first row, and steps of 16 rows before
// z / 16 are skipped.  Every row of the group enters once, none from outside
// it does, and a skipped step holds zeros alone.
long long check_windows(int max_rows, long long* checked) {
    constexpr int BK = 64, STEP = 16, R0 = 1000;
    long long bad = 0, n = 0;
    for (int rows = 1; rows <= max_rows; ++rows) {
        std::vector<int> seen(rows, 0);
        const int blocks = (rows + BK - 1) / BK;
        for (int kb = 0; kb < blocks; ++kb) {
            const int z = grp_zero_rows(rows, kb, BK), first = R0 + kb * BK;
            ++n; bad += z < 0 || z >= BK || (kb < blocks - 1 && z != 0);
            for (int i = 0; i < BK; ++i) {
                const int w = i - z;                      // row of the window
                const bool zero = w < 0 || w >= BK, skipped = i / STEP < z / STEP;
                ++n; bad += skipped && !zero;
                if (zero || skipped) continue;
                const int row = first + w - R0;
                ++n; bad += row < 0 || row >= rows;
                if (row >= 0 && row < rows) ++seen[row];
            }
        }
        for (int c : seen) { ++n; bad += c != 1; }
    }
    // the largest group: no overflow
    const int big = 2147482623, last = (big - 1) / BK;
    ++n; bad += grp_zero_rows(big, last, BK) != (last + 1) * static_cast<long long>(BK) - big;
    ++n; bad += grp_zero_rows(big, 0, BK) != 0;
    *checked = n;
    return bad;
}

}  // extern "C"
