// block_scales.cuh -- the scale bytes of microscaled 4-bit rows on their way to
// tensor memory (gemm_group.cuh, gemm_skinny.cuh).
//
// A row's scales lie in memory along k, 16 bytes for 512 k.  An MMA takes
// those of 128 k (a word) from four columns of tensor memory: row 32c + i in
// lane i, column c.  The copy engine brings 16 bytes of 128 rows, 16 bytes
// apart (zeros past a row's last block and past the last row: the zeros beside
// them must not meet a NaN); a warp turns word w of row 32c + i into word c of
// lane i of the w-th 512 bytes, which tmem_cp_scales then copies as they are.
#pragma once
#include "ptx.cuh"

namespace tg {

constexpr int kScaleTile = 128 * 16;

// In place: lane i owns the 16 bytes of rows i, 32 + i, 64 + i and 96 + i before
// and its 16 bytes of the four words after, which are the same places.
__device__ __forceinline__ void order_scales(uint32_t tile, int lane) {
    const uint32_t at = tile + lane * 16;
    uint4 v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w) : "r"(at + c * 512) : "memory");
    auto put = [&](int w, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + w * 512), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    };
    put(0, v[0].x, v[1].x, v[2].x, v[3].x);
    put(1, v[0].y, v[1].y, v[2].y, v[3].y);
    put(2, v[0].z, v[1].z, v[2].z, v[3].z);
    put(3, v[0].w, v[1].w, v[2].w, v[3].w);
}

}  // namespace tg
