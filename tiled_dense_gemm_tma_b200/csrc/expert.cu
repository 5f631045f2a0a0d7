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
// votes, the lowest adds their number to the warp's own counter of that
// expert, so no counter is shared and the order is the input's.  Counters:
// [warp][E + 1] in shared memory (the last for dropped choices), turned into
// each warp's first row by a sum over the warps before it, the blocks before
// it (several blocks only), and all smaller experts.  A warp keeps the first
// kKeep x 32 of its choices in registers between counting and placing.
//
// Bound by latency, not by its 12 bytes a choice.  Up to kOneBlock choices one
// block does it all in one launch.  More of them are cut among several blocks: a
// first launch writes each block's counts, the second places.  Every block of it
// reads all counts, so that many experts ask for fewer blocks (kMaxCounts).
// One block against several (us, one / several): 2048 choices 6.2 / 10.3 of 8
// experts and 9.3 / 14.4 of 1024; 4096 choices 10.3 / 10.3 and 16.4 / 15.4.
// Blocks of 8 warps, or of 32 where that leaves a warp more than kKeep x 32
// choices.  Measured, us (8 warps / 32): 1024 choices 4.1 / 5.1, 4096 of 128
// experts 10.3 / 12.3, 65536 14.6 / 16.4; 524288 of 256 38.9 / 22.6.

constexpr int kKeep = 8;
constexpr int kOneBlock = 2048;
constexpr int kPerBlock = 1024;
constexpr int kMaxBlocks = 148;
constexpr int kMaxCounts = 40960;

struct SortPlan {
    int blocks, warps;
    int64_t chunk;            // choices per block
};

SortPlan sort_plan(int64_t n, int E) {
    SortPlan p;
    p.blocks = 1;
    if (n > kOneBlock) {
        int64_t b = (n + kPerBlock - 1) / kPerBlock;
        const int most = kMaxCounts / (E + 1);
        if (b > most) b = most;
        p.blocks = static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
    }
    p.chunk = ((n + p.blocks - 1) / p.blocks + 31) / 32 * 32;
    p.warps = p.chunk <= 8 * 32 * kKeep ? 8 : 32;
    return p;
}

// The choices [w0, w1) of one warp.
template <typename Id>
struct WarpChoices {
    const Id* ids;
    int64_t w0, w1;
    int E, lane, bits;
    int e[kKeep];
    uint32_t same[kKeep];     // the lanes that hold the same expert, from count on

    // Lanes whose x (0..E, or -1: none) equals this lane's: one vote a bit.  The
    // match instruction does it at once, but an SM takes one about every 64
    // clocks: with it 8192 choices in one block took 22 us.
    __device__ __forceinline__ uint32_t alike(int x) const {
        uint32_t m = __ballot_sync(0xffffffffu, x >= 0);
#pragma unroll 4
        for (int b = 0; b < bits; ++b) {
            const bool on = (x >> b) & 1;
            const uint32_t v = __ballot_sync(0xffffffffu, on);
            m &= on ? v : ~v;
        }
        return m;
    }
    // expert of this lane's choice from i on: E if dropped, -1 past the end
    __device__ __forceinline__ int fetch(int64_t i) const {
        if (i + lane >= w1) return -1;
        const Id v = ids[i + lane];
        return v >= 0 && v < static_cast<Id>(E) ? static_cast<int>(v) : E;
    }
    __device__ __forceinline__ void start(const Id* p, int64_t n, int64_t chunk, int warps, int experts) {
        ids = p;
        E = experts;
        lane = threadIdx.x & 31;
        bits = 32 - __clz(experts);                   // of the numbers 0..E
        const int64_t b0 = blockIdx.x * chunk, b1 = min(n, b0 + chunk);
        const int64_t per = (chunk / 32 + warps - 1) / warps * 32;
        w0 = min(b1, b0 + static_cast<int64_t>(threadIdx.x >> 5) * per);
        w1 = min(b1, w0 + per);
#pragma unroll
        for (int k = 0; k < kKeep; ++k) e[k] = fetch(w0 + 32 * k);
    }
    // the number of each expert's choices, added to cnt
    __device__ __forceinline__ void count(int* cnt) {
        auto add = [&](int x, uint32_t m) {
            if (x >= 0 && lane == __ffs(m) - 1) cnt[x] += __popc(m);
            __syncwarp();
        };
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (w0 + 32 * k < w1) {
                same[k] = alike(e[k]);
                add(e[k], same[k]);
            }
        for (int64_t i = w0 + 32 * kKeep; i < w1; i += 32) {
            const int x = fetch(i);
            add(x, alike(x));
        }
    }
    // after count: f(expert or -1, lanes that hold it, index of lane 0's choice)
    // for every 32 choices, in order
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (w0 + 32 * k < w1) f(e[k], same[k], w0 + 32 * k);
        for (int64_t i = w0 + 32 * kKeep; i < w1; i += 32) {
            const int x = fetch(i);
            f(x, alike(x), i);
        }
    }
};

// Exclusive prefix sums of v over the block's threads, in thread order; total
// gets their sum.  `part`: WARPS ints of shared memory.
template <int WARPS>
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
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const int x = part[w];
        before += w < warp ? x : 0;
        total += x;
    }
    return before + s - v;
}

template <typename Id, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
sort_count_kernel(const Id* __restrict__ ids, int64_t n, int64_t chunk, int E, int* __restrict__ counts) {
    extern __shared__ int cnt[];                      // [warp][E + 1]
    const int W = E + 1;
    WarpChoices<Id> mine;
    mine.start(ids, n, chunk, WARPS, E);
    for (int i = threadIdx.x; i < WARPS * W; i += 32 * WARPS) cnt[i] = 0;
    __syncthreads();
    mine.count(cnt + (threadIdx.x >> 5) * W);
    __syncthreads();
    for (int e = threadIdx.x; e < W; e += 32 * WARPS) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += cnt[w * W + e];
        counts[static_cast<int64_t>(blockIdx.x) * W + e] = s;
    }
}

// counts: [gridDim.x][E + 1] of sort_count_kernel, or null for a lone block.
template <typename Id, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
sort_place_kernel(const Id* __restrict__ ids, int64_t n, int64_t chunk, int E, const int* __restrict__ counts,
                  int* __restrict__ offsets, int* __restrict__ pos, int* __restrict__ src) {
    constexpr int THREADS = 32 * WARPS;
    extern __shared__ int cnt[];                      // [warp][E + 1], then all [E + 1], before [E + 1]
    __shared__ int part[WARPS];
    const int W = E + 1;
    int* all = cnt + WARPS * W;
    int* before = all + W;
    int* first = cnt + (threadIdx.x >> 5) * W;
    WarpChoices<Id> mine;
    mine.start(ids, n, chunk, WARPS, E);
    for (int i = threadIdx.x; i < (WARPS + 2) * W; i += THREADS) cnt[i] = 0;
    __syncthreads();
    mine.count(first);
    if (counts) {
        // each expert's count in all blocks and in the blocks before this one:
        // the threads take (block, expert) pairs in memory order, eight loads
        // under way at a time
        const int total = gridDim.x * W, own = blockIdx.x * W;
        int e = threadIdx.x % W;
        const int step = THREADS % W;
        for (int i0 = threadIdx.x; i0 < total; i0 += 8 * THREADS) {
            int c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = i0 + j * THREADS;
                c[j] = i < total ? __ldg(counts + i) : 0;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (c[j]) {
                    atomicAdd(all + e, c[j]);         // integers: any order gives the same sum
                    if (i0 + j * THREADS < own) atomicAdd(before + e, c[j]);
                }
                e += step;
                if (e >= W) e -= W;
            }
        }
    }
    __syncthreads();
    // first row of each warp's choices of each expert
    int run = 0;
    for (int e0 = 0; e0 < W; e0 += THREADS) {
        const int e = e0 + threadIdx.x;
        int sum = 0;
        if (e < W) {
            if (counts) {
                sum = all[e];
            } else {
#pragma unroll
                for (int w = 0; w < WARPS; ++w) sum += cnt[w * W + e];
            }
        }
        int total;
        int at = run + block_exclusive<WARPS>(sum, part, total);
        run += total;
        if (e < W) {
            if (blockIdx.x == 0) offsets[e] = at;     // W entries: offsets[E] starts the dropped
            at += before[e];
#pragma unroll
            for (int w0 = 0; w0 < WARPS; w0 += 8) {
                int c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = cnt[(w0 + w) * W + e];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    cnt[(w0 + w) * W + e] = at;
                    at += c[w];
                }
            }
        }
    }
    __syncthreads();
    mine.each([&](int x, uint32_t m, int64_t i) {
        const int rank = __popc(m & ((1u << mine.lane) - 1));
        const int r = x >= 0 ? first[x] + rank : 0;
        __syncwarp();
        if (x >= 0 && rank == 0) first[x] += __popc(m);
        __syncwarp();
        if (x >= 0) {
            pos[i + mine.lane] = r;
            src[r] = static_cast<int>(i + mine.lane);
        }
    });
}

template <typename Id, int WARPS>
int run_sort(const SortPlan& pl, int slot, int64_t n, int E, const Id* ids, int* offsets, int* pos, int* src,
             int* scratch, cudaStream_t s) {
    const int W = E + 1;
    auto count = sort_count_kernel<Id, WARPS>;
    auto place = sort_place_kernel<Id, WARPS>;
    if (set_smem_attr(reinterpret_cast<const void*>(count), WARPS * 1025 * 4, slot) != cudaSuccess ||
        set_smem_attr(reinterpret_cast<const void*>(place), (WARPS + 2) * 1025 * 4, slot + 1) != cudaSuccess)
        return kCudaError;
    if (pl.blocks > 1) {
        count<<<pl.blocks, 32 * WARPS, WARPS * W * 4, s>>>(ids, n, pl.chunk, E, scratch);
        if (cudaGetLastError() != cudaSuccess) return kCudaError;
    }
    place<<<pl.blocks, 32 * WARPS, (WARPS + 2) * W * 4, s>>>(ids, n, pl.chunk, E, pl.blocks > 1 ? scratch : nullptr,
                                                              offsets, pos, src);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

template <typename Id>
int pick_sort(int64_t n, int E, const Id* ids, int* offsets, int* pos, int* src, int* scratch, cudaStream_t s) {
    const SortPlan pl = sort_plan(n, E);
    const int slot = sizeof(Id) == 4 ? 82 : 86;
    return pl.warps == 8 ? run_sort<Id, 8>(pl, slot, n, E, ids, offsets, pos, src, scratch, s)
                         : run_sort<Id, 32>(pl, slot + 2, n, E, ids, offsets, pos, src, scratch, s);
}

// ----------------------------------------------------------------- gather
//
// A warp takes one token's row, or a 2 KB piece of it: the piece stays in
// registers and is written to each of its rows.  Bound by HBM, each row read
// once and its copies written: 8192 tokens of 4 KB to 8 rows each 48 us, 6.3 TB/s
// (gathering row by row would read each token's row eight times).

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

// The rows of up to J of a token's choices from j0 on: row numbers (-1: none
// there) and weights, 0 for what does not count so that 0 * 0 is added.
template <int J>
struct Choices {
    int r[J];
    float w[J];
    __device__ __forceinline__ void load(const int* pos, const float* weights, int64_t at, int j0, int topk,
                                         int64_t n, int live) {
#pragma unroll
        for (int j = 0; j < J; ++j) r[j] = j0 + j < topk ? __ldg(pos + at + j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < J; ++j) w[j] = weights && j0 + j < topk ? __ldg(weights + at + j0 + j) : 1.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (r[j] < 0 || r[j] >= n) r[j] = -1;
            if (r[j] < 0 || r[j] >= live) w[j] = 0.f;
        }
    }
    __device__ __forceinline__ bool kept(int j, int live) const { return r[j] >= 0 && r[j] < live; }
};

// A warp takes one token's row, or a 1 KB piece of it, and sums its choices'
// rows in order, J of them requested before the first is used.  Measured with
// the caches flushed, event times of which about 5 us are the launch: one row
// at a time 80 us for 8 rows of 2048 values each of 8192 tokens, J = 4 61 us
// (floor 46), J = 2 63; 6 rows of 2040 values 55 and 51 (floor 36), 2 rows of
// 4096 53 and 45 (floor 31): what J rounds topk up to counts.
template <bool BF16, int J>
__global__ void __launch_bounds__(256)
combine_kernel(int64_t tokens, int topk, int64_t H, const uint16_t* __restrict__ Y, int64_t ldy,
               const int* __restrict__ pos, const int* __restrict__ kept, const float* __restrict__ weights,
               uint16_t* __restrict__ out, int64_t ldo, int pieces) {
    constexpr int V = 2;                              // vectors a lane sums at a time
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = id / pieces;
    if (t >= tokens) return;
    const int piece = static_cast<int>(id - t * pieces), lane = threadIdx.x & 31;
    const int64_t n = tokens * topk;
    const int live = kept_rows(kept, n);
    const int64_t nv = H >> 3;
    const int tail = static_cast<int>(H & 7);
    const int64_t vecs = nv + (tail ? 1 : 0);
    const int64_t v0 = static_cast<int64_t>(piece) * (32 * V) + lane;
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
    for (int j0 = 0; j0 < topk; j0 += J) {
        Choices<J> c;
        c.load(pos, weights, t * topk, j0, topk, n, live);
        uint4 y[J][V];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                y[j][i] = c.kept(j, live) && v0 + 32 * i < vecs ? load_vec(Y + c.r[j] * ldy, v0 + 32 * i, nv, tail)
                                                                : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[8];
                widen8<BF16>(y[j][i], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i][e] = fmaf(c.w[j], f[e], acc[i][e]);
            }
    }
    uint16_t* o = out + t * ldo;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (v0 + 32 * i < vecs) store_vec(o, v0 + 32 * i, nv, tail, narrow8<BF16>(acc[i]));
}

// A block takes one token: J choices at a time it reads their rows, writes
// the rows' gradient and sums the J dot products, over the threads in a
// fixed order.
template <bool BF16, int J, int V, int THREADS>
__global__ void __launch_bounds__(THREADS)
combine_grad_kernel(int topk, int64_t n, int64_t H, const uint16_t* __restrict__ Y, int64_t ldy,
                    const uint16_t* __restrict__ dout, int64_t ldd, const int* __restrict__ pos,
                    const int* __restrict__ kept, const float* __restrict__ weights,
                    uint16_t* __restrict__ dY, int64_t lddy, float* __restrict__ dweights) {
    __shared__ float part[THREADS / 32][J];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int live = kept_rows(kept, n);
    const int64_t nv = H >> 3;
    const int tail = static_cast<int>(H & 7);
    const int64_t vecs = nv + (tail ? 1 : 0);
    const uint16_t* g = dout + t * ldd;
    for (int j0 = 0; j0 < topk; j0 += J) {
        Choices<J> c;
        c.load(pos, weights, t * topk, j0, topk, n, live);
        float dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) dot[j] = 0.f;
        for (int64_t v0 = threadIdx.x; v0 < vecs; v0 += V * THREADS) {
            uint4 y[V][J], gv[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int64_t v = v0 + i * THREADS;
                gv[i] = v < vecs ? load_vec(g, v, nv, tail) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    y[i][j] = v < vecs && c.kept(j, live) ? load_vec(Y + c.r[j] * ldy, v, nv, tail)
                                                          : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int64_t v = v0 + i * THREADS;
                if (v >= vecs) break;
                float d[8];
                widen8<BF16>(gv[i], d);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (c.r[j] < 0) continue;
                    float f[8], o[8];
                    const bool keep = c.r[j] < live;
                    widen8<BF16>(y[i][j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (keep) dot[j] = fmaf(f[e], d[e], dot[j]);
                        o[e] = keep ? c.w[j] * d[e] : 0.f;
                    }
                    store_vec(dY + c.r[j] * lddy, v, nv, tail, narrow8<BF16>(o));
                }
            }
        }
        // J sums over 32 lanes: halve the lanes' share of the J sums as long
        // as there are several, so that J + log2(32 / J) exchanges do
        int at = 0;                                   // which sum this lane ends up with
#pragma unroll
        for (int m = J / 2, d = 16; m >= 1; m >>= 1, d >>= 1) {
            const bool up = lane & d;
#pragma unroll
            for (int j = 0; j < m; ++j) {
                const float give = up ? dot[j] : dot[j + m], keep = up ? dot[j + m] : dot[j];
                dot[j] = keep + __shfl_xor_sync(0xffffffffu, give, d);
            }
            at += up ? m : 0;
        }
#pragma unroll
        for (int d = 16 / J; d >= 1; d >>= 1) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], d);
        if (lane % (32 / J) == 0) part[warp][at] = dot[0];
        __syncthreads();
        if (threadIdx.x < J && j0 + threadIdx.x < topk) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < THREADS / 32; ++i) s += part[i][threadIdx.x];
            dweights[t * topk + j0 + threadIdx.x] = s;
        }
        if (j0 + J < topk) __syncthreads();
    }
}

template <bool BF16>
void start_combine_grad(unsigned tokens, cudaStream_t s, int topk, int64_t n, int64_t H, const uint16_t* Y,
                        int64_t ldy, const uint16_t* dout, int64_t ldd, const int* pos, const int* kept,
                        const float* weights, uint16_t* dY, int64_t lddy, float* dweights) {
    // Threads a token and what they hold, measured (us; the floors of 2 n H + T H
    // 2-byte values are 66, 87, 51 and 23): with 6 x 2040, 8 x 2048, 2 x 4096 (8192
    // tokens) and 4 x 512 (16384 tokens) values a token, two choices and two
    // vectors at a time take 80, 98, 59, 41 on two warps and 88, 111, 64, 33 on
    // one; eight choices at a time on eight warps 121, 137, 70, 55: small blocks
    // wait for each other less at the dot products' end.  Few tokens leave SMs
    // idle, and then eight warps a token shorten each one's chain of loads.  At the
    // limits (us, rows of launches on inputs beyond L2, one / two / eight warps):
    //   6 choices of   512 values   520 values          1024            2048            4096
    //   256 tokens  7.7  6.5  7.1   9.1  7.8  7.7   12.4 8.3 8.3   18.0 12.0  8.8   32.3 19.0 10.8
    //   512 tokens  8.3  8.3 12.4  10.3  8.3 12.4   12.0 8.6 12.2  19.5 13.1 14.4   32.9 20.8 18.5
    //   1024        8.7  8.2 16.7  10.5 10.0 18.2   13.7 10.3 18.5 21.1 16.4 20.6   36.9 26.7 27.5
    //   8192       22.8 30.0 94.3  28.7 34.9 98.3   39.0 41.0 102  83.4 71.8 121    166  151  164
    if (H <= 512)
        combine_grad_kernel<BF16, 2, 2, 32><<<tokens, 32, 0, s>>>(topk, n, H, Y, ldy, dout, ldd, pos, kept, weights,
                                                                  dY, lddy, dweights);
    else if (tokens > (H > 2048 ? 512 : 256))
        combine_grad_kernel<BF16, 2, 2, 64><<<tokens, 64, 0, s>>>(topk, n, H, Y, ldy, dout, ldd, pos, kept, weights,
                                                                  dY, lddy, dweights);
    else
        combine_grad_kernel<BF16, 2, 2, 256><<<tokens, 256, 0, s>>>(topk, n, H, Y, ldy, dout, ldd, pos, kept, weights,
                                                                    dY, lddy, dweights);
}

bool grid_ok(int64_t blocks) { return blocks <= 0x7fffffffll; }

}  // namespace

int64_t expert_sort_scratch(int64_t n, int E) {
    const SortPlan p = sort_plan(n, E);
    return p.blocks > 1 ? static_cast<int64_t>(p.blocks) * (E + 1) * 4 : 0;
}

int launch_expert_sort(int64_t tokens, int topk, int E, const void* ids, int id_bytes, int* offsets,
                       int* pos, int* src, void* scratch, void* stream) {
    if (!current_device(nullptr)) return kNoDevice;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t n = tokens * topk;
    if (id_bytes == 4)
        return pick_sort(n, E, static_cast<const int32_t*>(ids), offsets, pos, src, static_cast<int*>(scratch), s);
    return pick_sort(n, E, static_cast<const long long*>(ids), offsets, pos, src, static_cast<int*>(scratch), s);
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
    const bool four = (topk + 1) / 2 % 2 == 0;        // whole fours, or all but one of them
    auto k = bf16 ? (four ? combine_kernel<true, 4> : combine_kernel<true, 2>)
                  : (four ? combine_kernel<false, 4> : combine_kernel<false, 2>);
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
    auto start = bf16 ? start_combine_grad<true> : start_combine_grad<false>;
    start(static_cast<unsigned>(tokens), static_cast<cudaStream_t>(stream), topk, tokens * topk, H,
          static_cast<const uint16_t*>(Y), ldy, static_cast<const uint16_t*>(dout), ldd, pos, kept, weights,
          static_cast<uint16_t*>(dY), lddy, dweights);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

}  // namespace tg
