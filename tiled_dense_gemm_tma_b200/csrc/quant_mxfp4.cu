// quant_mxfp4.cu -- rows of 16-bit values to microscaled 4-bit floating point
// and back: the operands of the 4-bit products.
//
// 32 consecutive values of a row are a block.  With top its largest magnitude,
//
//   E = floor(log2(top)) - 2 + 127 (at least 0),   q[k] = E2M1(x[k] * 2^(127 - E))
//
// rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code,
// magnitudes above 6 (they are below 8) to 6.  A block of zeros gets E = 0; one
// that holds an infinity or a NaN gets E = 255, the format's NaN, and codes 0.
//
// floor(log2(top)) + 127 is the exponent field of top in fp32, where top is
// normal; a subnormal top (bfloat16 only) has field 0 and is below 2^-126, so
// that E is 0 either way.  The product with a power of two is exact (it can
// only underflow where the result rounds to 0 all the same), so the one rounding
// is that to E2M1, by the conversion instruction: the code is the one that the
// formula gives in real arithmetic.
//
// A warp takes UNROLL x 256 consecutive values of a row, a lane eight at a
// time; four neighbouring lanes hold a block, and its maximum takes two
// shuffles.  Units that lie wholly inside the row have no checks.  Bound by HBM:
// 16384 x 8192 bf16 values take 51 us to 4 bits (6.6 TB/s; 57 with the checks in
// every unit, when the issue of instructions was at 80 %), 54 us back (6.3 TB/s; 80
// with a thread to eight values and one load in flight).  Figures of event times,
// of which an empty call is 6.
#include "host.cuh"
#include "launch.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tg {

namespace {

template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Eight values to eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float2 (&x)[4]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
    return r;
}

// Eight codes to four pairs of fp16 values (exact).
__device__ __forceinline__ void values8(uint32_t q, __half2 (&h)[4]) {
    uint32_t r[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(q));
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2*>(&r[i]);
}

// 16-byte vector v of a row of K values, zero past its end.
__device__ __forceinline__ uint4 load_vec(const uint16_t* row, int v, int K) {
    const int left = K - 8 * v;
    if (left >= 8) return __ldg(reinterpret_cast<const uint4*>(row) + v);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < left) w[j >> 1] |= static_cast<uint32_t>(__ldg(row + 8ll * v + j)) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A 64-bit division only where the number needs it.
__device__ __forceinline__ long long row_of(long long unit, int per_row) {
    if (unit < (1ll << 32)) return static_cast<uint32_t>(unit) / static_cast<uint32_t>(per_row);
    return unit / per_row;
}

// What a block's largest magnitude (bits of the type) makes of it: E, and the
// power of two that its values are multiplied by.
template <bool BF16>
__device__ __forceinline__ uint32_t block_scale(uint32_t top, float& up) {
    const int field = static_cast<int>(__float_as_uint(widen2<BF16>(top).x) >> 23);
    const int E = max(field - 2, 0);
    up = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);
    return E;
}

// PLACES: each row goes to the rows pos[row * topk ..] of the output, as zeros
// to those from *kept on; else to its own.
template <bool BF16, bool PLACES, int UNROLL>
__global__ void __launch_bounds__(256)
quant_mxfp4_kernel(long long units, int per_row, int K, const uint16_t* __restrict__ X, long long ldx, int topk,
                   long long rows_out, const int* __restrict__ pos, const int* __restrict__ kept,
                   uint8_t* __restrict__ Q, long long ldq, uint8_t* __restrict__ S, long long lds) {
    const int lane = threadIdx.x & 31;
    const long long unit = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (unit >= units) return;
    const long long row = row_of(unit, per_row);
    const int first = static_cast<int>(unit - row * per_row) * (32 * UNROLL), v0 = first + lane;
    const bool whole = first + 32 * UNROLL <= K >> 3;        // warp-uniform
    const int nvec = (K + 7) >> 3;
    const uint16_t* x = X + row * ldx;
    uint4 v[UNROLL];
    if (whole) {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(x) + v0 + 32 * i);
    } else {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
            v[i] = v0 + 32 * i < nvec ? load_vec(x, v0 + 32 * i, K) : make_uint4(0, 0, 0, 0);
    }
    uint32_t code[UNROLL], exps[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        // largest magnitude as a bit pattern, infinity and NaN above all values
        uint32_t top2 = __vimax3_u16x2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu, v[i].z & 0x7fff7fffu);
        top2 = __vmaxu2(top2, v[i].w & 0x7fff7fffu);
        top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 1));
        top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 2));
        const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
        const bool bad = top >= (BF16 ? 0x7f80u : 0x7c00u);
        float up;
        const uint32_t E = block_scale<BF16>(top, up);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = widen2<BF16>(w[j]);
            f[j].x *= up;
            f[j].y *= up;
        }
        code[i] = bad ? 0u : codes8(f);
        exps[i] = bad ? 255u : E;
    }
    const int bytes = (K + 1) >> 1;
    // Rows for several places: lane l of the first eight takes scales 4 l .. 4 l + 3 of
    // the unit, one store a place and not four (8191 x 2040 to six places 22.5 -> 18.4
    // us; to one place nothing is gained).
    constexpr bool WORDS = PLACES && UNROLL == 4;
    uint32_t word = 0;
    if constexpr (WORDS) {
        const uint32_t own = exps[0] | exps[1] << 8 | exps[2] << 16 | exps[3] << 24;    // blocks m, 8 + m, ... of lane 4 m
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t o = __shfl_sync(0xffffffffu, own, 16 * (lane & 1) + 4 * j);
            word |= (o >> (8 * ((lane >> 1) & 3)) & 0xffu) << (8 * j);
        }
    }
    const int blocks = (K + 31) >> 5, b0 = (first >> 2) + 4 * lane;
    auto write_scales = [&](uint8_t* s, uint32_t w) {
        if (lane >= 8) return;
        if (b0 + 4 <= blocks) {
            *reinterpret_cast<uint32_t*>(s + b0) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (b0 + j < blocks) s[b0 + j] = static_cast<uint8_t>(w >> (8 * j));
        }
    };
    auto write = [&](long long r, bool live) {
        uint8_t* q = Q + r * ldq;
        uint8_t* s = S + r * lds;
        if (whole) {
            uint32_t* q4 = reinterpret_cast<uint32_t*>(q) + v0;
            uint8_t* s1 = s + (v0 >> 2);
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                q4[32 * i] = live ? code[i] : 0u;
                if (!WORDS && (lane & 3) == 0) s1[8 * i] = static_cast<uint8_t>(live ? exps[i] : 0u);
            }
            if constexpr (WORDS) write_scales(s, live ? word : 0u);
            return;
        }
        if constexpr (WORDS) write_scales(s, live ? word : 0u);
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int vi = v0 + 32 * i;
            const uint32_t c = live ? code[i] : 0u;
            const int left = bytes - 4 * vi;
            if (left >= 4) {
                reinterpret_cast<uint32_t*>(q)[vi] = c;
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (j < left) q[4ll * vi + j] = static_cast<uint8_t>(c >> (8 * j));
            }
            if (!WORDS && (lane & 3) == 0 && left > 0) s[vi >> 2] = static_cast<uint8_t>(live ? exps[i] : 0u);
        }
    };
    if constexpr (PLACES) {
        const int live = __ldg(kept);
        for (int j = 0; j < topk; ++j) {
            const int r = __ldg(pos + row * topk + j);
            if (r >= 0 && r < rows_out) write(r, r < live);
        }
    } else {
        write(row, true);
    }
}

// The same units of a row a warp, back.
template <bool BF16, int UNROLL>
__global__ void __launch_bounds__(256)
dequant_mxfp4_kernel(long long units, int per_row, int K, const uint8_t* __restrict__ Q, long long ldq,
                     const uint8_t* __restrict__ S, long long lds, uint16_t* __restrict__ Y, long long ldy) {
    const int lane = threadIdx.x & 31;
    const long long unit = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (unit >= units) return;
    const long long row = row_of(unit, per_row);
    const int first = static_cast<int>(unit - row * per_row) * (32 * UNROLL), v0 = first + lane;
    const bool whole = first + 32 * UNROLL <= K >> 3;        // warp-uniform
    const uint8_t* q = Q + row * ldq;
    const uint8_t* s = S + row * lds;
    uint32_t c[UNROLL], E[UNROLL];
    if (whole) {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            c[i] = __ldg(reinterpret_cast<const uint32_t*>(q) + v0 + 32 * i);
            E[i] = __ldg(s + (v0 >> 2) + 8 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int v = v0 + 32 * i, left = K - 8 * v;
            c[i] = E[i] = 0;
            if (left > 0) E[i] = __ldg(s + (v >> 2));
            if (left >= 8) {
                c[i] = __ldg(reinterpret_cast<const uint32_t*>(q) + v);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (2 * j < left) c[i] |= static_cast<uint32_t>(__ldg(q + 4ll * v + j)) << (8 * j);
            }
        }
    }
    uint16_t* y = Y + row * ldy;
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int v = v0 + 32 * i, left = K - 8 * v;
        const float up = __uint_as_float(E[i] == 0 ? 0x00400000u : E[i] == 255 ? 0x7fc00000u : E[i] << 23);
        __half2 h[4];
        values8(c[i], h);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            if constexpr (BF16) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * up, f.y * up);
                o[j] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                const __half2 b = __floats2half2_rn(f.x * up, f.y * up);
                o[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        if (whole || left >= 8) {
            reinterpret_cast<uint4*>(y)[v] = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) y[8ll * v + j] = static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1)));
        }
    }
}

constexpr long long kMaxBlocks = 0x7fffffffll;

// Few values, or short rows: more warps, each with less to wait for.
bool few_values(int64_t M, int64_t K) { return K <= 256 || M * ((K + 1023) / 1024) < 148 * 16; }

template <bool BF16, int UNROLL>
int back(int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* scales, int64_t lds, void* Y, int64_t ldy,
         cudaStream_t s) {
    const long long per_row = (K + 256 * UNROLL - 1) / (256 * UNROLL), units = M * per_row;
    if ((units + 7) / 8 > kMaxBlocks) return kUnsupported;
    dequant_mxfp4_kernel<BF16, UNROLL><<<static_cast<unsigned>((units + 7) / 8), 256, 0, s>>>(
        units, static_cast<int>(per_row), static_cast<int>(K), Q, ldq, scales, lds, static_cast<uint16_t*>(Y), ldy);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

template <bool BF16, bool PLACES, int UNROLL>
int start(int64_t M, int64_t K, const void* X, int64_t ldx, int topk, const int* pos, const int* kept, uint8_t* Q,
          int64_t ldq, uint8_t* scales, int64_t lds, cudaStream_t s) {
    const long long per_row = (K + 256 * UNROLL - 1) / (256 * UNROLL), units = M * per_row;
    if ((units + 7) / 8 > kMaxBlocks) return kUnsupported;
    quant_mxfp4_kernel<BF16, PLACES, UNROLL><<<static_cast<unsigned>((units + 7) / 8), 256, 0, s>>>(
        units, static_cast<int>(per_row), static_cast<int>(K), static_cast<const uint16_t*>(X), ldx, topk,
        M * topk, pos, kept, Q, ldq, scales, lds);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

template <bool BF16, bool PLACES>
int pick(int64_t M, int64_t K, const void* X, int64_t ldx, int topk, const int* pos, const int* kept, uint8_t* Q,
         int64_t ldq, uint8_t* scales, int64_t lds, cudaStream_t s) {
    if (few_values(M, K))
        return start<BF16, PLACES, 1>(M, K, X, ldx, topk, pos, kept, Q, ldq, scales, lds, s);
    return start<BF16, PLACES, 4>(M, K, X, ldx, topk, pos, kept, Q, ldq, scales, lds, s);
}

}  // namespace

int launch_quant_mxfp4(int64_t M, int64_t K, const void* X, int64_t ldx, int bf16, int topk, const int* pos,
                       const int* kept, uint8_t* Q, int64_t ldq, uint8_t* scales, int64_t lds, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pos)
        return bf16 ? pick<true, true>(M, K, X, ldx, topk, pos, kept, Q, ldq, scales, lds, s)
                    : pick<false, true>(M, K, X, ldx, topk, pos, kept, Q, ldq, scales, lds, s);
    return bf16 ? pick<true, false>(M, K, X, ldx, 1, nullptr, nullptr, Q, ldq, scales, lds, s)
                : pick<false, false>(M, K, X, ldx, 1, nullptr, nullptr, Q, ldq, scales, lds, s);
}

int launch_dequant_mxfp4(int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* scales, int64_t lds,
                         void* Y, int64_t ldy, int bf16, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (few_values(M, K))
        return bf16 ? back<true, 1>(M, K, Q, ldq, scales, lds, Y, ldy, s) : back<false, 1>(M, K, Q, ldq, scales, lds, Y, ldy, s);
    return bf16 ? back<true, 4>(M, K, Q, ldq, scales, lds, Y, ldy, s) : back<false, 4>(M, K, Q, ldq, scales, lds, Y, ldy, s);
}

}  // namespace tg
