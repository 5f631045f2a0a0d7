// block_scales.cuh -- the scale bytes of microscaled 4-bit rows on their way to
// tensor memory (gemm_group.cuh, gemm_skinny.cuh).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace tg {

// 16 scale bytes of a row at `p`, zero from the `left`-th on; `rows` rows are
// left in the matrix, this one included (none: all zero).  Rows are a multiple
// of 16 bytes apart, so that only the last one may end before its 16 bytes.
__device__ __forceinline__ uint4 load_blocks(const uint8_t* p, int left, int rows) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (rows <= 0) return v;
    if (left >= 16) return __ldg(reinterpret_cast<const uint4*>(p));
    if (rows > 1) {
        v = __ldg(reinterpret_cast<const uint4*>(p));
        uint32_t* w = &v.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int keep = left - 4 * j;
            if (keep < 4) w[j] = keep > 0 ? w[j] & ((1u << (8 * keep)) - 1) : 0;
        }
        return v;
    }
    uint32_t* w = &v.x;
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (j < left) w[j / 4] |= static_cast<uint32_t>(__ldg(p + j)) << (8 * (j % 4));
    return v;
}

}  // namespace tg
