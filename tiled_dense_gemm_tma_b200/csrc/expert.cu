// expert.cu -- tokens sorted by expert and back: the data movement around the
// experts' products (gemm_group.cuh).
//
// tokens x topk choices, flat index i = token * topk + j, name an expert each;
// a number outside [0, E) is a dropped choice.  The stable sort by expert puts
// choice i at row pos[i], row r holds choice src[r], the rows of expert e are
// [offsets[e], offsets[e + 1]) and the dropped choices follow, in order, from
// offsets[E] on.  Their rows are zero and count for nothing:
//
//   gather        Xs[pos[i]] = X[i / topk]                       (else 0)
//   combine       Y[t] = sum_j w[t][j] * Ys[pos[t, j]]           (kept j, in order, fp32)
//   combine grad  dYs[pos[t, j]] = w[t][j] * dY[t],  dw[t][j] = <Ys[pos[t, j]], dY[t]>
//
// combine without weights is the gradient of gather.  All of them walk the
// tokens, not the sorted rows: a token's row is then read once however many
// experts it goes to, and sums over its choices need no atomics.
#include "host.cuh"
#include "launch.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tg {

namespace {

// ------------------------------------------------------------------- sort
//
// Counting sort with ranks from warp votes.  A warp takes 32 consecutive
// choices at a time; the lanes that hold the same expert find each other with
// a match vote, the lowest adds their number to the warp's own counter of that
// expert, so no counter is shared and the order is the input's.  Counters:
// [warp][E + 1] in shared memory (the last for dropped choices), turned into
// each warp's first row by a sum over the warps before it, the blocks before
// it (several blocks only), and all smaller experts.
//
// Up to kOneBlock choices one block does it all in one launch.  More of them
// are cut among up to kMaxBlocks blocks: a first launch writes each block's
// counts, the second starts from them.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kOneBlock = 8192;
constexpr int kPerBlock = 2048;
constexpr int kMaxBlocks = 148;

struct SortPlan {
    int blocks;
    int64_t chunk;            // choices per block
};

SortPlan sort_plan(int64_t n) {
    SortPlan p;
    p.blocks = 1;
    if (n > kOneBlock) {
        const int64_t b = (n + kPerBlock - 1) / kPerBlock;
        p.blocks = static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
    }
    p.chunk = ((n + p.blocks - 1) / p.blocks + 31) / 32 * 32;
    return p;
}

template <typename Id>
__device__ __forceinline__ int choice(const Id* ids, int64_t i, int64_t end, int E) {
    if (i >= end) return -1;                          // no choice: counted nowhere
    const Id v = ids[i];
    return v >= 0 && v < static_cast<Id>(E) ? static_cast<int>(v) : E;
}

// This warp's counts of its choices [w0, w1) into cnt (E + 1, zeroed).
template <typename Id>
__device__ __forceinline__ void count_choices(const Id* ids, int64_t w0, int64_t w1, int E, int* cnt, int lane) {
    for (int64_t i = w0; i < w1; i += 32) {
        const int e = choice(ids, i + lane, w1, E);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) cnt[e] += __popc(same);
        __syncwarp();
    }
}

// Exclusive prefix sums of v over the block's threads, in thread order; total
// gets their sum.  `part` is kSortWarps + 1 ints of shared memory.
__device__ __forceinline__ int block_exclusive(int v, int* part, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();                                  // part may still be read from an earlier call
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int t = part[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += y;
        }
        part[lane] = t;
    }
    __syncthreads();
    total = part[kSortWarps - 1];
    return (warp ? part[warp - 1] : 0) + s - v;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const Id* __restrict__ ids, int64_t n, int64_t chunk, int E, int* __restrict__ counts) {
    extern __shared__ int cnt[];                      // [warp][E + 1]
    const int W = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kSortWarps * W; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t b0 = blockIdx.x * chunk, b1 = min(n, b0 + chunk);
    const int64_t per = (chunk / 32 + kSortWarps - 1) / kSortWarps * 32;
    const int64_t w0 = min(b1, b0 + warp * per), w1 = min(b1, w0 + per);
    count_choices(ids, w0, w1, E, cnt + warp * W, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < W; e += kSortThreads) {
        int s = 0;
        for (int w = 0; w < kSortWarps; ++w) s += cnt[w * W + e];
        counts[static_cast<int64_t>(blockIdx.x) * W + e] = s;
    }
}

// counts: [gridDim.x][E + 1] of sort_count_kernel, or null for a lone block.
template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const Id* __restrict__ ids, int64_t n, int64_t chunk, int E, const int* __restrict__ counts,
                  int* __restrict__ offsets, int* __restrict__ pos, int* __restrict__ src) {
    extern __shared__ int cnt[];                      // [warp][E + 1], then all [E + 1], before [E + 1]
    __shared__ int part[kSortWarps + 1];
    const int W = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* all = cnt + kSortWarps * W;
    int* before = all + W;
    for (int i = threadIdx.x; i < (kSortWarps + 2) * W; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t b0 = blockIdx.x * chunk, b1 = min(n, b0 + chunk);
    const int64_t per = (chunk / 32 + kSortWarps - 1) / kSortWarps * 32;
    const int64_t w0 = min(b1, b0 + warp * per), w1 = min(b1, w0 + per);
    count_choices(ids, w0, w1, E, cnt + warp * W, lane);
    if (counts) {
        // each expert's count in all blocks and in the blocks before this one:
        // the threads take (block, expert) pairs in memory order
        const int total = gridDim.x * W, mine = blockIdx.x * W;
        for (int i = threadIdx.x; i < total; i += kSortThreads) {
            const int c = counts[i];
            if (c) {
                const int e = i % W;
                atomicAdd(all + e, c);                // integers: any order gives the same sum
                if (i < mine) atomicAdd(before + e, c);
            }
        }
    }
    __syncthreads();
    // first row of each warp's choices of each expert
    int run = 0;
    for (int e0 = 0; e0 < W; e0 += kSortThreads) {
        const int e = e0 + threadIdx.x;
        int mine = 0;
        if (e < W && !counts)
            for (int w = 0; w < kSortWarps; ++w) mine += cnt[w * W + e];
        const int sum = e < W ? (counts ? all[e] : mine) : 0;
        int total;
        int at = run + block_exclusive(sum, part, total);
        run += total;
        if (e < W) {
            if (blockIdx.x == 0) offsets[e] = at;     // W entries: offsets[E] starts the dropped
            at += before[e];
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = cnt[w * W + e];
                cnt[w * W + e] = at;
                at += c;
            }
        }
    }
    __syncthreads();
    int* first = cnt + warp * W;
    for (int64_t i = w0; i < w1; i += 32) {
        const int e = choice(ids, i + lane, w1, E);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        const int r = e >= 0 ? first[e] + rank : 0;
        __syncwarp();
        if (e >= 0 && rank == 0) first[e] += __popc(same);
        __syncwarp();
        if (e >= 0) {
            pos[i + lane] = r;
            src[r] = static_cast<int>(i + lane);
        }
    }
}

template <typename Id>
int run_sort(int64_t n, int E, const Id* ids, int* offsets, int* pos, int* src, int* scratch, cudaStream_t s) {
    const SortPlan pl = sort_plan(n);
    const int W = E + 1;
    const int smem1 = kSortWarps * W * 4, smem2 = (kSortWarps + 2) * W * 4;
    const int slot = sizeof(Id) == 4 ? 82 : 84;
    if (set_smem_attr(reinterpret_cast<const void*>(sort_count_kernel<Id>), (kSortWarps) * 1025 * 4, slot) != cudaSuccess ||
        set_smem_attr(reinterpret_cast<const void*>(sort_place_kernel<Id>), (kSortWarps + 2) * 1025 * 4, slot + 1) != cudaSuccess)
        return kCudaError;
    const bool many = pl.blocks > 1;
    if (many) sort_count_kernel<Id><<<pl.blocks, kSortThreads, smem1, s>>>(ids, n, pl.chunk, E, scratch);
    sort_place_kernel<Id><<<pl.blocks, kSortThreads, smem2, s>>>(ids, n, pl.chunk, E, many ? scratch : nullptr,
                                                                offsets, pos, src);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

// ----------------------------------------------------------------- gather
//
// A warp takes one token's row, or a 2 KB piece of it: the piece stays in
// registers and is written to each of its rows.

__device__ __forceinline__ int kept_rows(const int* kept, int64_t n) {
    const int k = *kept;
    return k < 0 ? 0 : k > n ? static_cast<int>(n) : k;
}

constexpr int kPiece = 128;             // 16-byte vectors a warp takes at a time

__global__ void __launch_bounds__(256)
gather_kernel(int64_t tokens, int topk, int64_t bytes, const uint8_t* __restrict__ X, int64_t ldx,
              const float* __restrict__ scales, const int* __restrict__ pos, const int* __restrict__ kept,
              uint8_t* __restrict__ out, int64_t ldo, float* __restrict__ out_scales, int pieces) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = id / pieces;
    if (t >= tokens) return;
    const int piece = static_cast<int>(id - t * pieces), lane = threadIdx.x & 31;
    const int64_t n = tokens * topk;
    const int live = kept_rows(kept, n);
    const int64_t nv = bytes >> 4;
    const int tail = static_cast<int>(bytes & 15);
    const int64_t v0 = static_cast<int64_t>(piece) * kPiece + lane;
    const uint8_t* x = X + t * ldx;
    uint4 v[kPiece / 32];
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i)
        v[i] = v0 + 32 * i < nv ? __ldg(reinterpret_cast<const uint4*>(x) + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
    const bool last = piece == pieces - 1;
    const uint8_t end = last && lane < tail ? x[nv * 16 + lane] : 0;
    for (int j = 0; j < topk; ++j) {
        const int r = __ldg(pos + t * topk + j);
        if (r < 0 || r >= n) continue;                // not a row
        const bool keep = r < live;
        uint8_t* o = out + r * ldo;
#pragma unroll
        for (int i = 0; i < kPiece / 32; ++i)
            if (v0 + 32 * i < nv)
                *(reinterpret_cast<uint4*>(o) + v0 + 32 * i) = keep ? v[i] : make_uint4(0, 0, 0, 0);
        if (last && lane < tail) o[nv * 16 + lane] = keep ? end : 0;
        if (out_scales && piece == 0 && lane == 0) out_scales[r] = keep ? scales[t] : 0.f;
    }
}

// ---------------------------------------------------------------- combine

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            f[2 * j] = h.x;
            f[2 * j + 1] = h.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            w[j] = *reinterpret_cast<uint32_t*>(&h);
        } else {
            __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
            w[j] = *reinterpret_cast<uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector v of a row of H 16-bit values: whole, or the last H % 8 values.
__device__ __forceinline__ uint4 load_vec(const uint16_t* row, int64_t v, int64_t nv, int tail) {
    if (v < nv) return __ldg(reinterpret_cast<const uint4*>(row) + v);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < tail) w[j >> 1] |= static_cast<uint32_t>(row[8 * nv + j]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_vec(uint16_t* row, int64_t v, int64_t nv, int tail, const uint4& x) {
    if (v < nv) {
        *(reinterpret_cast<uint4*>(row) + v) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < tail) row[8 * nv + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
}

// A warp takes one token's row, or a piece of it, and sums its choices' rows
// in order.
template <bool BF16>
__global__ void __launch_bounds__(256)
combine_kernel(int64_t tokens, int topk, int64_t H, const uint16_t* __restrict__ Y, int64_t ldy,
               const int* __restrict__ pos, const int* __restrict__ kept, const float* __restrict__ weights,
               uint16_t* __restrict__ out, int64_t ldo, int pieces) {
    constexpr int V = 2;                              // vectors a lane sums at a time
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = id / pieces;
    if (t >= tokens) return;
    const int piece = static_cast<int>(id - t * pieces), lane = threadIdx.x & 31;
    const int live = kept_rows(kept, tokens * topk);
    const int64_t nv = H >> 3;
    const int tail = static_cast<int>(H & 7);
    const int64_t vecs = nv + (tail ? 1 : 0);
    const int64_t v0 = static_cast<int64_t>(piece) * (32 * V) + lane;
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
#pragma unroll 4
    for (int j = 0; j < topk; ++j) {
        const int r = __ldg(pos + t * topk + j);
        if (r < 0 || r >= live) continue;             // dropped
        const float w = weights ? __ldg(weights + t * topk + j) : 1.f;
        const uint16_t* y = Y + r * ldy;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (v0 + 32 * i < vecs) {
                float f[8];
                widen8<BF16>(load_vec(y, v0 + 32 * i, nv, tail), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i][e] = fmaf(w, f[e], acc[i][e]);
            }
    }
    uint16_t* o = out + t * ldo;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (v0 + 32 * i < vecs) store_vec(o, v0 + 32 * i, nv, tail, narrow8<BF16>(acc[i]));
}

// A block takes one token: four choices at a time it reads their rows, writes
// the rows' gradient and sums the four dot products, over the threads in a
// fixed order.
constexpr int kGradThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kGradThreads)
combine_grad_kernel(int topk, int64_t n, int64_t H, const uint16_t* __restrict__ Y, int64_t ldy,
                    const uint16_t* __restrict__ dout, int64_t ldd, const int* __restrict__ pos,
                    const int* __restrict__ kept, const float* __restrict__ weights,
                    uint16_t* __restrict__ dY, int64_t lddy, float* __restrict__ dweights) {
    constexpr int J = 4;
    __shared__ float part[kGradThreads / 32][J];
    const int64_t t = blockIdx.x;
    const int live = kept_rows(kept, n);
    const int64_t nv = H >> 3;
    const int tail = static_cast<int>(H & 7);
    const int64_t vecs = nv + (tail ? 1 : 0);
    const uint16_t* g = dout + t * ldd;
    for (int j0 = 0; j0 < topk; j0 += J) {
        int r[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            r[j] = j0 + j < topk ? __ldg(pos + t * topk + j0 + j) : -1;
            if (r[j] >= n) r[j] = -1;                 // not a row
            w[j] = j0 + j < topk ? __ldg(weights + t * topk + j0 + j) : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t v = threadIdx.x; v < vecs; v += kGradThreads) {
            float d[8];
            widen8<BF16>(load_vec(g, v, nv, tail), d);
            uint4 y[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                y[j] = r[j] >= 0 && r[j] < live ? load_vec(Y + r[j] * ldy, v, nv, tail) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (r[j] < 0) continue;
                float f[8], o[8];
                const bool keep = r[j] < live;
                widen8<BF16>(y[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (keep) dot[j] = fmaf(f[e], d[e], dot[j]);
                    o[e] = keep ? w[j] * d[e] : 0.f;
                }
                store_vec(dY + r[j] * lddy, v, nv, tail, narrow8<BF16>(o));
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < J && j0 + threadIdx.x < topk) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kGradThreads / 32; ++i) s += part[i][threadIdx.x];
            dweights[t * topk + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

bool grid_ok(int64_t blocks) { return blocks <= 0x7fffffffll; }

}  // namespace

int64_t expert_sort_scratch(int64_t n, int E) {
    const SortPlan p = sort_plan(n);
    return p.blocks > 1 ? static_cast<int64_t>(p.blocks) * (E + 1) * 4 : 0;
}

int launch_expert_sort(int64_t tokens, int topk, int E, const void* ids, int id_bytes, int* offsets,
                       int* pos, int* src, void* scratch, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t n = tokens * topk;
    if (id_bytes == 4)
        return run_sort(n, E, static_cast<const int32_t*>(ids), offsets, pos, src, static_cast<int*>(scratch), s);
    return run_sort(n, E, static_cast<const long long*>(ids), offsets, pos, src, static_cast<int*>(scratch), s);
}

int launch_expert_gather(int64_t tokens, int topk, int64_t H, int eb, const void* X, int64_t ldx,
                         const float* scales, const int* pos, const int* kept, void* out,
                         int64_t ldo, float* out_scales, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const int64_t bytes = H * eb;
    int64_t pieces = (bytes / 16 + kPiece - 1) / kPiece;
    if (pieces < 1) pieces = 1;
    const int64_t blocks = (tokens * pieces + 7) / 8;
    if (!grid_ok(blocks)) return kUnsupported;
    gather_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        tokens, topk, bytes, static_cast<const uint8_t*>(X), ldx * eb, scales, pos, kept,
        static_cast<uint8_t*>(out), ldo * eb, out_scales, static_cast<int>(pieces));
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

int launch_expert_combine(int64_t tokens, int topk, int64_t H, int bf16, const void* Y, int64_t ldy,
                          const int* pos, const int* kept, const float* weights, void* out,
                          int64_t ldo, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const int64_t pieces = ((H + 7) / 8 + 63) / 64;
    const int64_t blocks = (tokens * pieces + 7) / 8;
    if (!grid_ok(blocks)) return kUnsupported;
    auto k = bf16 ? combine_kernel<true> : combine_kernel<false>;
    k<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        tokens, topk, H, static_cast<const uint16_t*>(Y), ldy, pos, kept, weights, static_cast<uint16_t*>(out),
        ldo, static_cast<int>(pieces));
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

int launch_expert_combine_grad(int64_t tokens, int topk, int64_t H, int bf16, const void* Y,
                               int64_t ldy, const void* dout, int64_t ldd, const int* pos,
                               const int* kept, const float* weights, void* dY, int64_t lddy,
                               float* dweights, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    if (!grid_ok(tokens)) return kUnsupported;
    auto k = bf16 ? combine_grad_kernel<true> : combine_grad_kernel<false>;
    k<<<static_cast<unsigned>(tokens), kGradThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        topk, tokens * topk, H, static_cast<const uint16_t*>(Y), ldy, static_cast<const uint16_t*>(dout), ldd, pos,
        kept, weights, static_cast<uint16_t*>(dY), lddy, dweights);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

}  // namespace tg
