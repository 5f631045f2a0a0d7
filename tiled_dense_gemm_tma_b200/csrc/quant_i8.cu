// quant_i8.cu -- rows of 16-bit values to signed 8-bit integers with one
// scale per row: the activation side of the 8-bit product.
//
//   top = max_k |x[k]|,  scale = top / 127,  q[k] = rint(x[k] * 127 / top)
//
// (ties to even; a row of zeros gets scale 0 and q = 0; a row with an
// infinity or a NaN gets scale NaN and q = 0, so that what is multiplied with
// it is NaN).
//
// The integer is exactly the one that the formula names in real arithmetic.
// With x of at most 11 significant bits, x * 127 has at most 18, and
// x * 127 / top is either exactly halfway between two integers or at least
// 2^-19 of itself away from it; r = x * inv with inv = 127 / top in fp32 is
// off by 2^-24 of itself (r is never rounded: one fused multiply-add rounds
// it to the integer, another gives its distance from it), so rint(r) is right
// unless r lies within 2^-11 of halfway (127 * 2^-24 is less).  Those few values, and rows whose
// 127 / top could overflow, take the division, which is off by 2^-24 of the
// quotient and keeps exact halves exact.
//
// Bound by HBM: 2 bytes in and 1 out per value.  One group of threads per row
// keeps the row in registers between the maximum and the rounding; rows
// longer than that (16384 values) are read twice, the second time from L2.
#include "host.cuh"
#include "launch.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tg {

namespace {

constexpr int kVec = 4;                 // 16-byte vectors a thread keeps

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpair(uint64_t d) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Eight values -> eight integers.
template <bool BF16>
__device__ __forceinline__ uint2 round8(const uint4& v, float inv, float top, bool divide) {
    constexpr float kMagic = 12582912.f;             // 1.5 * 2^23: adding it leaves rint(r) in the low bits
    const uint64_t magic = pair(kMagic, kMagic), inv2 = pair(inv, inv);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t t[8];
    float off = 0.f;                                 // largest distance from an integer
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = widen<BF16>(w[j]);
        const uint64_t x2 = pair(x.x, x.y);
        const uint64_t s2 = fma2(x2, inv2, magic);
        const float2 s = unpair(s2);
        t[2 * j] = __float_as_uint(s.x);
        t[2 * j + 1] = __float_as_uint(s.y);
        const float2 d = unpair(fma2(x2, inv2, sub2(magic, s2)));       // r - rint(r)
        off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
    }
    if (divide || off > 0.5f - 0x1p-11f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = widen<BF16>(w[j]);
            t[2 * j] = __float_as_uint(__fdiv_rn(x.x * 127.f, top) + kMagic);
            t[2 * j + 1] = __float_as_uint(__fdiv_rn(x.y * 127.f, top) + kMagic);
        }
    }
    uint2 o;
    o.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
    return o;
}

// TPR threads per row, a block of max(TPR, 128).  FITS: the row's vectors fit
// the threads' registers.  From 128 threads on three quarters of the SM's
// threads are asked for (40 registers a thread and not 47): 4096 rows of 16384
// values 47 us against 54, of 8192 27 both ways; one-warp rows of 1024 lose by
// it (18.2 against 16.7).  Event times; an empty call reads 7 to 8 us there.
template <bool BF16, int TPR, bool FITS>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR < 128 ? 1 : 1536 / TPR)
quant_i8_kernel(int M, int K, const uint16_t* __restrict__ X, long long ldx, int8_t* __restrict__ Q,
                long long ldq, float* __restrict__ scales) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;   // rows per block
    constexpr int WPR = TPR / 32;
    const int t = threadIdx.x % TPR;
    const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / TPR;
    if (row >= M) return;                            // whole warps: a row has whole warps
    const uint16_t* x = X + row * ldx;
    const int nv = K >> 3, tail = K & 7;             // whole vectors, values after them
    auto load = [&](int v) -> uint4 {
        if (v < nv) return __ldg(reinterpret_cast<const uint4*>(x) + v);
        uint32_t w[4] = {0, 0, 0, 0};
        if (v == nv)
            for (int j = 0; j < tail; ++j) w[j >> 1] |= static_cast<uint32_t>(x[8 * nv + j]) << (16 * (j & 1));
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    const int vecs = nv + (tail ? 1 : 0);
    // largest magnitude as a bit pattern: ordered like the values, infinity
    // and NaN above all of them
    uint4 keep[kVec];
    uint32_t top2 = 0;
    auto take = [&](const uint4& v) {
        top2 = __vmaxu2(top2, v.x & 0x7fff7fffu);
        top2 = __vmaxu2(top2, v.y & 0x7fff7fffu);
        top2 = __vmaxu2(top2, v.z & 0x7fff7fffu);
        top2 = __vmaxu2(top2, v.w & 0x7fff7fffu);
    };
    if constexpr (FITS) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) keep[i] = load(t + i * TPR);
#pragma unroll
        for (int i = 0; i < kVec; ++i) take(keep[i]);
    } else {
        for (int v = t; v < vecs; v += TPR) take(load(v));
    }
    uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (WPR > 1) {
        __shared__ uint32_t part[WPR];               // one row per block here
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
        __syncthreads();
        top = part[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i) top = max(top, part[i]);
    }
    const bool bad = top >= (BF16 ? 0x7f80u : 0x7c00u);
    const float ftop = widen<BF16>(top).x;
    const bool divide = ftop < 0x1p-100f;
    const float inv = divide ? 0.f : __fdiv_rn(127.f, ftop);
    if (t == 0) scales[row] = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(ftop, 127.f);
    int8_t* q = Q + row * ldq;
    auto store = [&](int v, const uint4& val) {
        if (v >= vecs) return;
        const uint2 o = (bad || top == 0) ? make_uint2(0, 0) : round8<BF16>(val, inv, ftop, divide);
        if (v < nv) {
            *reinterpret_cast<uint2*>(q + 8 * v) = o;
        } else {
            for (int j = 0; j < tail; ++j)
                q[8 * v + j] = static_cast<int8_t>((j < 4 ? o.x >> (8 * j) : o.y >> (8 * (j - 4))) & 0xff);
        }
    };
    if constexpr (FITS) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) store(t + i * TPR, keep[i]);
    } else {
        for (int v = t; v < vecs; v += TPR) store(v, load(v));
    }
}

template <bool BF16, int TPR, bool FITS>
void start(int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scales, cudaStream_t s) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    quant_i8_kernel<BF16, TPR, FITS><<<static_cast<unsigned>((M + RPB - 1) / RPB), TPR < 128 ? 128 : TPR, 0, s>>>(
        static_cast<int>(M), static_cast<int>(K), static_cast<const uint16_t*>(X), ldx, Q, ldq, scales);
}

template <bool BF16>
void pick(int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scales, cudaStream_t s) {
    const int64_t vecs = (K + 7) / 8;
    if (vecs <= 32 * kVec) start<BF16, 32, true>(M, K, X, ldx, Q, ldq, scales, s);
    else if (vecs <= 128 * kVec) start<BF16, 128, true>(M, K, X, ldx, Q, ldq, scales, s);
    else if (vecs <= 256 * kVec) start<BF16, 256, true>(M, K, X, ldx, Q, ldq, scales, s);
    else if (vecs <= 512 * kVec) start<BF16, 512, true>(M, K, X, ldx, Q, ldq, scales, s);
    else start<BF16, 512, false>(M, K, X, ldx, Q, ldq, scales, s);
}

}  // namespace

int launch_quant_i8(int64_t M, int64_t K, const void* X, int64_t ldx, int bf16, int8_t* Q,
                    int64_t ldq, float* scales, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (bf16) pick<true>(M, K, X, ldx, Q, ldq, scales, s);
    else pick<false>(M, K, X, ldx, Q, ldq, scales, s);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

}  // namespace tg
