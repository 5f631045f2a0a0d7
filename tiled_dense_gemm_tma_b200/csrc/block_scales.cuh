// block_scales.cuh -- the scale bytes of microscaled 4-bit rows on their way to
// tensor memory (gemm_group.cuh, gemm_skinny.cuh).
//
// A row's scales lie in memory along k, 4 bytes (a word) for 128 k.  An MMA
// takes a word of each row from four columns of tensor memory: row 32c + i in lane
// i, column c.  4 or 8 words of 128 rows are brought row behind row (zeros past a
// row's last block and past the last row: the zeros beside them must not meet a
// NaN); a warp puts word w of row 32c + i at word c of lane i of
// the w-th 512 bytes, which tmem_cp_scales then copies as they are.
#pragma once
#include "ptx.cuh"

namespace tg {

// The tile of 128 rows of 4 * Q words at `tile`, in place.  Lane i reads rows i,
// 32 + i, 64 + i and 96 + i, all lanes before the first writes.
template <int Q>
__device__ __forceinline__ void order_scales(uint32_t tile, int lane) {
    uint4 v[4][Q];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int h = 0; h < Q; ++h)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[c][h].x), "=r"(v[c][h].y), "=r"(v[c][h].z), "=r"(v[c][h].w)
                         : "r"(tile + (32 * c + lane) * 16 * Q + 16 * h) : "memory");
    __syncwarp();
    auto put = [&](int w, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(tile + w * 512 + lane * 16), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    };
#pragma unroll
    for (int h = 0; h < Q; ++h) {
        put(4 * h, v[0][h].x, v[1][h].x, v[2][h].x, v[3][h].x);
        put(4 * h + 1, v[0][h].y, v[1][h].y, v[2][h].y, v[3][h].y);
        put(4 * h + 2, v[0][h].z, v[1][h].z, v[2][h].z, v[3][h].z);
        put(4 * h + 3, v[0][h].w, v[1][h].w, v[2][h].w, v[3][h].w);
    }
}

// 16 bytes from global to shared memory, the first `bytes` (0..16) of them read
// and the rest zero, completing at cp_async_wait of the same thread.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Start bringing 32 bytes from byte k on of the rows row0 .. row0 + 127 of
// `rows` rows of `blocks` bytes, `ld` apart.
__device__ __forceinline__ void load_scales(uint32_t tile, const uint8_t* base, int row0, int rows, long long ld,
                                            int k, int blocks, int lane) {
    const int at = k + 16 * (lane & 1);
    const int bytes = min(16, max(0, blocks - at));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = row0 + 16 * i + (lane >> 1);
        const bool in = r < rows && bytes > 0;
        cp_async_16(tile + (16 * i * 32 + lane * 16), in ? base + r * ld + at : base, in ? bytes : 0);
    }
}

}  // namespace tg
