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
// unless r lies within 2^-16 of halfway (127 * 2^-24 is less than 2^-17).
// Those few values, and rows whose 127 / top could overflow, take the
// division, which is off by 2^-24 of the quotient and keeps exact halves exact.
// For bfloat16 it divides x * 127 * 2^-8 by top * 2^-8, since x * 127 alone
// would leave fp32 where x is above 2^128 / 127; both are exact down to the
// smallest subnormal (multiples of 2^-141, of at most 18 bits).
//
// Bound by HBM, 2 bytes in and 1 out per value, and close behind by the issue
// of its instructions (69 % of the slots): 16384 rows of 8192 bf16 values take
// 70 us (5.75 TB/s), 79 with the division asked for eight values at a time.
// One group of threads per row keeps the row in registers between the maximum
// and the rounding; rows longer than that (16384 values) are read twice, the
// second time from L2.
#include "host.cuh"
#include "launch.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tg {

namespace {

constexpr int kVec = 4;                 // 16-byte vectors a thread keeps
template <bool BF16>
constexpr float kDown = BF16 ? 0x1p-8f : 1.f;       // keeps x * 127 finite in the division

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

// Eight values -> eight integers; top is the row's times kDown.  The division is asked for pair by pair: in
// a row of bfloat16 about one value in 600 is the half of its largest (63.5),
// so that 35 % of a warp's 256 values held one, and dividing all eight of each
// lane was a third of the kernel's instructions.
template <bool BF16>
__device__ __forceinline__ uint2 round8(const uint4& v, float inv, float top, bool divide) {
    constexpr float kMagic = 12582912.f;             // 1.5 * 2^23: adding it leaves rint(r) in the low bits
    const uint64_t magic = pair(kMagic, kMagic), inv2 = pair(inv, inv);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t t[4];                                   // two integers each, in the low bytes of its halves
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = widen<BF16>(w[j]);
        const uint64_t x2 = pair(x.x, x.y);
        const uint64_t s2 = fma2(x2, inv2, magic);
        float2 s = unpair(s2);
        const float2 d = unpair(fma2(x2, inv2, sub2(magic, s2)));       // r - rint(r)
        if (divide || fmaxf(fabsf(d.x), fabsf(d.y)) > 0.5f - 0x1p-16f) {
            s.x = __fdiv_rn(x.x * (127.f * kDown<BF16>), top) + kMagic;
            s.y = __fdiv_rn(x.y * (127.f * kDown<BF16>), top) + kMagic;
        }
        t[j] = __byte_perm(__float_as_uint(s.x), __float_as_uint(s.y), 0x0040);
    }
    return make_uint2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[2], t[3], 0x5410));
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
    const uint4* x = reinterpret_cast<const uint4*>(X + row * ldx) + t;
    // whole vectors of this thread (every TPR-th from t), and the values after
    // the row's last whole vector, which the thread next in turn takes
    const int nv = K >> 3;
    const int mine = nv > t ? (nv - t - 1) / TPR + 1 : 0;
    const int tail = nv % TPR == t ? K & 7 : 0;
    // largest magnitude as a bit pattern: ordered like the values, infinity
    // and NaN above all of them
    uint4 keep[kVec];
    uint32_t top2 = 0;
    auto take = [&](const uint4& v) {
        top2 = __vimax3_u16x2(top2, v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
        top2 = __vimax3_u16x2(top2, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
    };
    if constexpr (FITS) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            keep[i] = i < mine ? __ldg(x + i * TPR) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kVec; ++i) take(keep[i]);
    } else {
        for (int i = 0; i < mine; ++i) take(__ldg(x + static_cast<int64_t>(i) * TPR));
    }
    uint4 rest = make_uint4(0, 0, 0, 0);
    if (tail) {
        const uint16_t* end = X + row * ldx + 8ll * nv;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < tail) w[j >> 1] |= static_cast<uint32_t>(end[j]) << (16 * (j & 1));
        rest = make_uint4(w[0], w[1], w[2], w[3]);
        take(rest);
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
    if (t == 0) scales[row] = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(ftop, 127.f);
    int8_t* q8 = Q + row * ldq;
    uint2* q = reinterpret_cast<uint2*>(q8) + t;
    const bool zero = bad || top == 0;
    const bool divide = ftop < 0x1p-100f;
    const float inv = divide ? 0.f : __fdiv_rn(127.f, ftop), low = ftop * kDown<BF16>;
    auto store = [&](int i, const uint4& v) {
        q[static_cast<int64_t>(i) * TPR] = zero ? make_uint2(0, 0) : round8<BF16>(v, inv, low, divide);
    };
    if constexpr (FITS) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < mine) store(i, keep[i]);
    } else {
        for (int i = 0; i < mine; ++i) store(i, __ldg(x + static_cast<int64_t>(i) * TPR));
    }
    if (tail) {
        const uint2 o = zero ? make_uint2(0, 0) : round8<BF16>(rest, inv, low, divide);
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < tail) q8[8ll * nv + j] = static_cast<int8_t>((j < 4 ? o.x >> (8 * j) : o.y >> (8 * (j - 4))) & 0xff);
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
