// gemm_group.cuh -- products over groups of rows on CTA pairs: the experts'
// products of a mixture-of-experts layer (16-bit, 8-bit and microscaled 4-bit), their
// weight gradient, and, as one group of all rows, the dense 8-bit and 4-bit products.
//
// The rows of A (R x K) are sorted into groups: group e is the rows
// [offsets[e], offsets[e + 1]), known on the device only.
//
//   product (WG = 0):          C[r][n]    = epi( sum_k A[r][k] * W_e[k][n] )
//   weight gradient (WG = 1):  C_e[k][n]  = sum_{r in group e} A[r][k] * G[r][n]
//
// 4-bit operands (E2M1 in blocks of 32 k with E8M0 scales): the tensor cores
// multiply by the scales (kind::mxf4), which they read from tensor memory; sums
// are fp32.  Three more warps of each CTA bring the scales of its weight columns
// and of all the tile's rows (block_scales.cuh).
//
// 8-bit operands: the sum is an exact 32-bit integer, and
// C[r][n] = epi( (sum * row_scale[r]) * col_scale_e[n] ), in fp32, rounded once.
//
// Two CTAs on neighbouring SMs (cluster of 2, tcgen05 cta_group::2) share a
// 256-lane tile, as in gemm_tc2.cuh; the roles (TMA, MMA, epilogue), the
// barriers and the bounded waits are the same, but two TMA warps take the k
// blocks in turn and up to eight epilogue warps share a tile (four took 26.5 us
// for 2048 x 8192 x 1024 in 8 bits, eight 23.9: its 8 blocks of MMAs a tile are
// shorter than the epilogue).
//
// Product: the operands are swapped, D = C^T.  The 256 lanes are weight
// columns n (each CTA stages its 128), and the rows r are the MMA's N side,
// whose width is a run-time multiple of 32 up to 256 (each CTA stages half).
// A group of a few rows then costs a narrow MMA and few operand bytes where
// rows on the 256-lane side would always pay for 256, and the loads of a
// small group are almost only its weights.  A tile is read from tensor
// memory as MMA fragments (16x256b), rounded, transposed by stmatrix into a
// [32 rows][32 columns] staging tile and written with 16-byte stores, which
// stop at the group's last row; the rows past it belong to the next group
// and were only read.  Row tiles of a group are as even as whole widths
// allow (grp_tile of tile_sched.h).  Rows behind the last group are written
// as zero.
//
// Weight gradient: the 256 lanes are the columns k of A, the MMA's N side
// the columns n of G, the reduction runs over the group's rows.  Both
// operands are read MN-major (a shared-memory row is one row r).  The rows
// of the last 64-row block that lie past the group belong to the next group:
// MMA steps (16 rows) that hold none of the group's are skipped, and where
// the group ends inside a step, a fix-up warp of the leader CTA clears the
// step's other rows in both CTAs' shared memory, in both operands (0 * NaN is
// NaN), before the MMA reads them.  Such a block's loads complete on a barrier
// of their own in the leader, and the fix-up warp arrives on the full barrier
// in the producers' place.  A group of no rows gets zeros.
//
// Every CTA derives the tile list from the offsets itself: no host knows the
// group sizes, and no launch precedes this one.
//
// What bounds it: the MMAs where groups are large (32 groups of 1024 rows,
// 4096 x 2048 bf16: 352 us forward, 1560 TFLOP/s, 521 clocks a block of 512 MMA
// clocks; its weight gradient 354, 374 with groups of 1000 rows; 8-bit 4096 x
// 8192 x 8192 141 to 159 us, 3450 to 3900 TOP/s), the weight stream where they are
// small (64 groups of one row, 1024 x 2048: 47 us, 5.7 TB/s), and in long runs the
// power limit, at 1.1 to 1.7 GHz.  4-bit: a block of 256 k takes 512 clocks of MMAs
// and 600 in all, with five stages (six do not fit beside the scales) and shared memory
// that MMAs, copies and scales contend for; about 900 more a tile pass between
// its last MMA and the next one's first where their accumulators share columns.
// 8192 x 8192 x 8192 190 us (5780 TFLOP/s), 64 groups of 256 rows, 4096 x 4096, 133
// (5.6 TB/s), of 64 rows 110 (5.6 TB/s).  With few blocks (1024 k) the epilogue
// bounds it, some 150 clocks to read, 170 to pack and 300 to store 32 rows of a warp:
// 8192 x 8192 x 1024 47 us.
#pragma once
#include "gemm_tc.cuh"
#include "block_scales.cuh"

namespace tg {

constexpr int kMaxGroups = 1024;

struct GrpParams {
    int M, N, K;              // rows of A, columns of W / G, columns of A
    int E;                    // groups
    const int* offsets;       // E + 1, or null: one group of all rows
    int relu;
    int inject;               // debug: 1 = pair 0's leader skips arming the first slot
    int group_m;              // raster band height in 256-lane tiles
    unsigned long long timeout_ns;
    int* status;
    void* C;
    long long ldc;            // elements
    long long plane;          // WG: elements between the matrices of C
    const float* row_scale;   // 8-bit: one per row of A
    const float* col_scale;   // 8-bit: one per column, scale_plane apart per group
    long long scale_plane;
    // 4-bit (K in bytes, two values each): a row's scale bytes, one per 32 values
    const uint8_t* row_blocks;  // M rows of A, block_lda bytes apart
    const uint8_t* col_blocks;  // N rows of W_e, block_ldb apart, block_plane per group
    long long block_lda, block_ldb, block_plane;
    int blocks;               // scale bytes in a row
    int tiles;                // row tiles where one group holds all rows; 0: as its rows ask for
};

// TYPE: 0 f16, 1 bf16 (idesc formats), 3 signed 8-bit, 4 4-bit floating point
// with block scales (only K-major; k counts bytes, two values each).  W_MN = 1: the weights
// are stored K x N, their tiles MN-major; 0: N x K, K-major.  WG: the weight
// gradient (16-bit; both operands MN-major).  EPI: epilogue warps, one or two
// to each quarter of the lanes.
template <int TYPE_, OutT OUT_, int W_MN_, int WG_ = 0, int EPI_ = 8>
struct GrpCfg {
    static constexpr int TYPE = TYPE_;
    static constexpr OutT OUT = OUT_;
    static constexpr int W_MN = W_MN_;
    static constexpr int WG = WG_;
    static constexpr bool I8 = TYPE_ == 3;
    static constexpr bool MX = TYPE_ == 4;
    static constexpr int EB = I8 || MX ? 1 : 2;         // operand bytes
    static constexpr int BK = 128 / EB;                 // k per stage: one 128-byte swizzle row
    static constexpr int MMA_K = 32 / EB;               // k per MMA: 16 or 32
    static constexpr int STEPS = BK / MMA_K;            // MMAs per stage
    static constexpr int CHUNK = 128 / EB;              // columns per MN-major box row
    static constexpr int STAGES = MX ? 5 : 6;
    // 4-bit: a chunk is 1024 k, 32 scale bytes of every row and four stages, in a
    // slot of 128 lanes' and up to 256 rows' scales.  Three warps take the chunks
    // in turn, each with a slot of its own.
    static constexpr int SF_WARPS = MX ? 3 : 0;
    static constexpr int SF_TILE = 128 * 32;
    static constexpr int SF_SLOT = 3 * SF_TILE;
    static constexpr int SF_COLS = 24;                  // tensor memory of a stage's scales
    static constexpr int A_STAGE = 128 * 128;           // 128 lanes' operand, either major-ness
    static constexpr int B_STAGE = 128 * 128;           // up to 128 of the N side
    static constexpr int EPI_WARPS = EPI_;
    static constexpr int HALVES = EPI_ / 4;             // warps to a quarter of the lanes
    static_assert(EPI_ == 4 || EPI_ == 8, "epilogue warps");
    static constexpr int FIX_WARPS = WG_ ? 1 : 0;
    static constexpr int PRODUCERS = 2;                 // warp 0, and the first behind the epilogue
    static constexpr int THREADS = 32 * (1 + PRODUCERS + EPI_WARPS + FIX_WARPS + SF_WARPS);
    static constexpr int STG_BUF = WG_ ? 4096 : 2048;   // a warp's [32 rows][128 bytes] or [32 rows][32 columns]
    static constexpr int NBUF = WG_ ? 8 / EPI_ : 1;     // staging tiles a warp
    // Two accumulators of up to 256 columns, the first from the left, the second up
    // to ACC_END.  4-bit scales take the last 48 columns, so that two accumulators of
    // together more than 464 rows share some in the middle: the second waits until
    // those have been read.  (Tiles of at most 224 rows never would: 8192 x 8192 x
    // 8192 220 us.)
    static constexpr int TMEM_COLS = 512;
    static constexpr int ACC_END = MX ? TMEM_COLS - 2 * SF_COLS : TMEM_COLS;
    static constexpr int TABLE = WG_ ? 0 : ((MX ? 3 : 4) * (kMaxGroups + 2) * 4 + 15) / 16 * 16;
    static constexpr int ITEMS = MX ? 64 : 0;           // a pair's first items, ready in shared memory
    static constexpr int SMEM_DATA = STAGES * (A_STAGE + B_STAGE) + EPI_WARPS * NBUF * STG_BUF + SF_WARPS * SF_SLOT;
    static constexpr int SMEM_BYTES = SMEM_DATA + 512 + TABLE + ITEMS * 16 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(!(EB == 1 && WG_), "the 8-bit and 4-bit products have no gradient");
    static_assert(!(MX && W_MN_), "4-bit operands are K-major");
};

// First column of an accumulator of `width` columns.
template <class Cfg>
__device__ __forceinline__ uint32_t grp_acc_col(uint32_t acc, int width) {
    return !acc ? 0 : Cfg::MX ? Cfg::ACC_END - width : 256;
}

// 16 bytes of zeros at a shared::cluster address, possibly in the peer CTA.
__device__ __forceinline__ void clear_cluster(uint32_t cl_addr) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(cl_addr), "r"(0) : "memory");
}

// The calling thread's earlier writes to either CTA's shared memory reach the
// tensor cores and the copy engine.
__device__ __forceinline__ void fence_proxy_async_cluster() {
    asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}

// Both arrivals of a phase at once.
__device__ __forceinline__ void mbar_arrive_two(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 2;" ::"r"(smem_u32(bar)) : "memory");
}

// One work item: a 256-lane tile of the weight columns (WG: of A's columns)
// starting at n0, against the rows [m0, m1) (WG: the columns of G from m0).
struct GrpItem {
    int e;                    // group
    int n0, m0, m1;           // m0 >= m1: nothing to do
    int width;                // MMA N
    int kb;                   // k blocks; 0: the tile is zero
    int r0, rows;             // WG: the group's rows
};

// Where a role stands in its pair's items.
struct GrpWalk {
    int i = 0;                // 4-bit: next entry of the table
    int g = 0;                // group
};

// Epilogue of a product tile: this warp's 32 weight columns from nw, its share
// of the tile's rows, 32 at a time (half: which of HALVES warps).
template <class Cfg>
__device__ __forceinline__ void grp_store_rows(const GrpParams& p, const GrpItem& it, uint32_t taddr,
                                               int nw, int half, int lane, uint8_t* stg) {
    if (nw >= p.N) return;                                  // warp-uniform
    float cs[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (Cfg::I8) {
        if (it.kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = nw + 8 * j + (lane >> 2);
                if (n < p.N) cs[j] = __ldg(p.col_scale + it.e * p.scale_plane + n);
            }
        }
    }
    auto finish = [&](uint32_t v, float rs, float c) -> float {
        if constexpr (Cfg::I8) {
            // a NaN (of the row's scale) stays one under ReLU; fmaxf would hide it,
            // and a comparison takes 2048 x 8192 x 1024 from 22.6 to 23.8 us
            const float x = (__int2float_rn(static_cast<int>(v)) * rs) * c;
            return p.relu ? max_nan(x, 0.f) : x;
        } else {
            const float x = __uint_as_float(v);
            return p.relu ? fmaxf(x, 0.f) : x;
        }
    };
    auto pack = [&](float a, float b) -> uint32_t {
        if constexpr (Cfg::OUT == OutT::BF16) {
            __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            return *reinterpret_cast<uint32_t*>(&h);
        } else {
            __half2 h = __floats2half2_rn(a, b);
            return *reinterpret_cast<uint32_t*>(&h);
        }
    };
    const uint32_t stg_a = smem_u32(stg);
    const int mj = lane >> 3, mc = lane & 7;                // stmatrix: this lane's matrix and column
    const int rr = lane >> 2, ch = lane & 3;                // row store: row and 16-byte chunk
#pragma unroll 1
    for (int m = it.m0 + 32 * half; m < it.m1; m += 32 * Cfg::HALVES) {
        uint32_t v0[16], v1[16];
        if (it.kb) {
            tmem_ld_16x256b_x4(taddr + (m - it.m0), v0);
            tmem_ld_16x256b_x4(taddr + (16u << 16) + (m - it.m0), v1);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v0[i] = v1[i] = 0;
        }
        float rs[8];
        if constexpr (Cfg::I8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = m + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                rs[i] = (it.kb && r < it.m1) ? __ldg(p.row_scale + r) : 0.f;
            }
        }
        if (it.kb) tmem_ld_wait();
        __syncwarp();                                       // the last chunk's rows are read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float ra = Cfg::I8 ? rs[2 * i] : 0.f, rb = Cfg::I8 ? rs[2 * i + 1] : 0.f;
            const uint32_t w0 = pack(finish(v0[4 * i], ra, cs[0]), finish(v0[4 * i + 1], rb, cs[0]));
            const uint32_t w1 = pack(finish(v0[4 * i + 2], ra, cs[1]), finish(v0[4 * i + 3], rb, cs[1]));
            const uint32_t w2 = pack(finish(v1[4 * i], ra, cs[2]), finish(v1[4 * i + 1], rb, cs[2]));
            const uint32_t w3 = pack(finish(v1[4 * i + 2], ra, cs[3]), finish(v1[4 * i + 3], rb, cs[3]));
            // row 8i + mc, its 16-byte chunk mj at a place that spreads the
            // eight rows of a matrix over all banks
            stmatrix_x4_trans(stg_a + (8 * i + mc) * 64 + ((mj ^ ((mc >> 1) & 3)) << 4), w0, w1, w2, w3);
        }
        __syncwarp();
        uint16_t* dst0 = static_cast<uint16_t*>(p.C) + nw + ch * 8;
        const int left = p.N - (nw + ch * 8);               // columns from this chunk on
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + rr;
            const uint4 x = *reinterpret_cast<const uint4*>(stg + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
            if (m + r < it.m1) {
                uint16_t* dst = dst0 + static_cast<long long>(m + r) * p.ldc;
                if (left >= 8) {
                    *reinterpret_cast<uint4*>(dst) = x;
                } else {
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 7; ++j)
                        if (j < left) dst[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
                }
            }
        }
    }
}

// The same for a 4-bit product.  (Loading the next 32 rows before these are
// written cost time: 8192 x 8192 x 1024 68 us where it took 55.)  Columns that two
// accumulators may share come first, the last ones of the first accumulator, the
// first of the second; tpart hears when they have been read.
template <class Cfg>
__device__ __forceinline__ void grp_store_values(const GrpParams& p, const GrpItem& it, uint32_t taddr, int nw,
                                                 int half, int lane, uint8_t* stg, uint32_t acc, uint64_t* tpart) {
    auto part = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_leader(tpart);
    };
    const int rows = it.m1 - it.m0 - 32 * half;             // from this warp's first on
    const int chunks = nw < p.N && rows > 0 ? (rows - 1) / (32 * Cfg::HALVES) + 1 : 0;
    if (chunks == 0) {                                      // warp-uniform
        if (it.kb) part();
        return;
    }
    const float floor = p.relu ? 0.f : -__builtin_huge_valf();
    auto pack = [&](uint32_t va, uint32_t vb) -> uint32_t {
        // a NaN (of a scale) stays one
        const float a = max_nan(__uint_as_float(va), floor), b = max_nan(__uint_as_float(vb), floor);
        if constexpr (Cfg::OUT == OutT::BF16) {
            __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            return *reinterpret_cast<uint32_t*>(&h);
        } else {
            __half2 h = __floats2half2_rn(a, b);
            return *reinterpret_cast<uint32_t*>(&h);
        }
    };
    const uint32_t stg_a = smem_u32(stg);
    const int mj = lane >> 3, mc = lane & 7;                // as above
    const int rr = lane >> 2, ch = lane & 3;
    const int left = p.N - (nw + ch * 8);
    uint16_t* dst0 = static_cast<uint16_t*>(p.C) + nw + ch * 8;
    // Short sums wait for their epilogues, which are faster without a branch to each row
    // (8192 x 8192 x 512 47 -> 43 us, x 1024 49 -> 47, x 2048 the same, x 8192 188 -> 190).
    const bool whole = nw + 32 <= p.N;
    const bool down = acc == 0;
    uint32_t v0[16], v1[16];
#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
        const int m = it.m0 + 32 * (half + Cfg::HALVES * (down ? chunks - 1 - i : i));
        if (it.kb) {
            tmem_ld_16x256b_x4(taddr + (m - it.m0), v0);
            tmem_ld_16x256b_x4(taddr + (16u << 16) + (m - it.m0), v1);
            tmem_ld_wait_for(v0, v1);
            if (i == 0) part();
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v0[j] = v1[j] = 0;
        }
        __syncwarp();                                       // the last chunk's rows are read
#pragma unroll
        for (int j = 0; j < 4; ++j)
            stmatrix_x4_trans(stg_a + (8 * j + mc) * 64 + ((mj ^ ((mc >> 1) & 3)) << 4), pack(v0[4 * j], v0[4 * j + 1]),
                              pack(v0[4 * j + 2], v0[4 * j + 3]), pack(v1[4 * j], v1[4 * j + 1]),
                              pack(v1[4 * j + 2], v1[4 * j + 3]));
        __syncwarp();
        if (whole && m + 32 <= it.m1) {                     // as below
            uint16_t* dst = dst0 + static_cast<long long>(m + rr) * p.ldc;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(dst + j * 8 * p.ldc) =
                    *reinterpret_cast<const uint4*>(stg + (8 * j + rr) * 64 + ((ch ^ ((rr >> 1) & 3)) << 4));
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + rr;
            const uint4 x = *reinterpret_cast<const uint4*>(stg + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
            if (m + r < it.m1) {
                uint16_t* dst = dst0 + static_cast<long long>(m + r) * p.ldc;
                if (left >= 8) {
                    *reinterpret_cast<uint4*>(dst) = x;
                } else {
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 7; ++k)
                        if (k < left) dst[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
                }
            }
        }
    }
}

// Epilogue of a weight-gradient tile: this warp's 32 rows k from kr of C_e,
// its share of the columns from it.m0 on, 64 at a time.
template <class Cfg>
__device__ __forceinline__ void grp_store_grad(const CUtensorMap* tmC, const GrpParams& p, const GrpItem& it,
                                               uint32_t taddr, int kr, int half, int lane, uint8_t* stg0,
                                               uint32_t& nstore) {
    if (kr >= p.K) return;                                  // warp-uniform
#pragma unroll 1
    for (int c = 64 * half; it.m0 + c < it.m1; c += 64 * Cfg::HALVES) {
        const int col0 = it.m0 + c;
        uint32_t v[64];
        if (it.kb) {
            tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
            tmem_ld_32x32b_x32(taddr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
            tmem_ld_wait();
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = 0;
        }
        uint4 packed[8];
        pack_row_chunk<Cfg::OUT, false>(v, 0, packed);
        if (col0 + 64 > p.N) {
            if (kr + lane < p.K) {
                uint8_t* dst = reinterpret_cast<uint8_t*>(
                    static_cast<uint16_t*>(p.C) + it.e * p.plane + (kr + lane) * p.ldc + col0);
                store_row_tail<2>(dst, packed, (p.N - col0) * 2);
            }
            continue;
        }
        uint8_t* stg = stg0 + (nstore % Cfg::NBUF) * Cfg::STG_BUF;
        if (lane == 0) bulk_wait_read<Cfg::NBUF - 1>();     // this tile's last store has read it
        __syncwarp();
        uint8_t* row = stg + lane * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) = packed[j];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(tmC, stg, col0, kr, it.e);
            bulk_commit();
        }
        ++nstore;
    }
}

// tmA: the 256-lane operand (product: weights, 3-D; WG: A).  tmB .. tmB16:
// the N-side operand (product: rows of A in boxes of 128, 64, 32 and 16 rows;
// WG: G in tmB).  tmC: C (WG only).
template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
grp_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmB64,
                const __grid_constant__ CUtensorMap tmB32,
                const __grid_constant__ CUtensorMap tmB16,
                const __grid_constant__ CUtensorMap tmC,
                const GrpParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* smA = smem;
    uint8_t* smB = smA + Cfg::STAGES * Cfg::A_STAGE;
    uint8_t* smStg = smB + Cfg::STAGES * Cfg::B_STAGE;
    uint8_t* smSf = smStg + Cfg::EPI_WARPS * Cfg::NBUF * Cfg::STG_BUF;
    uint64_t* full = reinterpret_cast<uint64_t*>(smSf + Cfg::SF_WARPS * Cfg::SF_SLOT);
    uint64_t* empty = full + Cfg::STAGES;
    uint64_t* cut = empty + Cfg::STAGES;        // WG: a block that ends inside an MMA step has landed
    uint64_t* tfull = cut + Cfg::STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* sfull = drain + 1;                // 4-bit: a chunk's scales are there, in both CTAs
    uint64_t* sempty = sfull + Cfg::SF_WARPS;
    uint64_t* tpart = sempty + Cfg::SF_WARPS;    // 4-bit: an accumulator's shared columns have been read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tpart + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* gcount = const_cast<int*>(abort_flag) + 1;
    int* gstart = gcount + 1;                   // product: first item of each group that has rows
    int* gexp = gstart + kMaxGroups + 2;        // product: which group that is
    int* grow = gexp + kMaxGroups + 2;          // product: its first row
    int* gend = grow + kMaxGroups + 2;          // product: the row after its last
    int4* gitem = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(full) + 512 + Cfg::TABLE);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;
    const uint64_t limit = p.timeout_ns;
    // 256-lane tiles: of the weight columns, or of A's columns (WG)
    const int lanes_total = Cfg::WG ? p.K : p.N;
    const int ntl = (lanes_total - 1) / 256 + 1;
    const int ntg = Cfg::WG ? (p.N - 1) / 256 + 1 : 0;      // WG: tiles of G's columns
    auto tiles_of = [&](int rows) { return Cfg::MX && p.tiles ? p.tiles : grp_tiles(rows); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1);
            mbar_init(&cut[s], 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * Cfg::EPI_WARPS);
            if constexpr (Cfg::MX) mbar_init(&tpart[a], 2 * Cfg::EPI_WARPS);
        }
        for (int i = 0; i < Cfg::SF_WARPS; ++i) {
            mbar_init(&sfull[i], 2);
            mbar_init(&sempty[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if constexpr (Cfg::WG) {
            tma_prefetch_desc(&tmC);
        } else {
            tma_prefetch_desc(&tmB64);
            tma_prefetch_desc(&tmB32);
            tma_prefetch_desc(&tmB16);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    if constexpr (!Cfg::WG) {
        if (warp == 2) {
            // the groups that have rows, their rows and first items, the rows behind
            // the last group as one more.  A group starts at the largest offset so
            // far (its own, where they do not decrease): whatever the offsets hold,
            // no row belongs to two groups, and the items are no more than the host
            // counted.
            int base = 0, n = 0, reached = 0;
            for (int e0 = 0; e0 <= p.E; e0 += 32) {
                const int e = e0 + lane;
                int r0 = p.M, r1 = p.M, cnt = 0;
                if (e <= p.E) grp_rows(p.offsets, e, p.E, p.M, r0, r1);
                int low = max(r0, reached);
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, low, d);
                    if (lane >= d) low = max(low, y);
                }
                reached = __shfl_sync(0xffffffffu, low, 31);
                r0 = low;
                r1 = max(r1, r0);
                if (r1 > r0) cnt = tiles_of(r1 - r0) * ntl;
                int sum = cnt;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += y;
                }
                const uint32_t live = __ballot_sync(0xffffffffu, cnt > 0);
                if (cnt > 0) {
                    const int i = n + __popc(live & ((1u << lane) - 1));
                    gstart[i] = base + sum - cnt;
                    gexp[i] = e;
                    grow[i] = r0;
                    if constexpr (!Cfg::MX) gend[i] = r1;
                }
                n += __popc(live);
                base += __shfl_sync(0xffffffffu, sum, 31);
            }
            if (lane == 0) {
                if constexpr (Cfg::MX) grow[n] = p.M;
                gstart[n] = base;
                *gcount = n;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();          // peer barriers initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the tiles of a thin last wave in narrower pieces
    const int num_tiles = Cfg::WG ? p.E * ntl * ntg : gstart[*gcount];
    const int pieces = grp_pieces(num_tiles, npairs, Cfg::WG ? 2 : 4);
    const int dp = tail_dp(num_tiles, npairs, pieces);
    const int num_items = tail_items(num_tiles, dp, pieces);

    // item w; g walks forward through the product's groups
    auto item = [&](int i, int& g) -> GrpItem {
        GrpItem it;
        const int w = i < dp ? i : dp + (i - dp) / pieces;
        const int piece = i < dp ? -1 : (i - dp) % pieces;
        if constexpr (Cfg::WG) {
            const int per = ntl * ntg;
            it.e = w / per;
            int tl, tt;
            tile_coords(w - it.e * per, ntl, ntg, p.group_m, tl, tt);
            it.n0 = tl * 256;
            it.m0 = tt * 256;
            it.m1 = min(p.N, it.m0 + 256);
            it.width = 256;
            int r1;
            grp_rows(p.offsets, it.e, p.E, p.M, it.r0, r1);
            it.rows = r1 - it.r0;
            it.kb = (it.rows + Cfg::BK - 1) / Cfg::BK;
        } else {
            while (w >= gstart[g + 1]) ++g;
            it.e = gexp[g];
            const int r1 = Cfg::MX ? grow[g + 1] : gend[g];     // groups lie one behind the other
            it.r0 = grow[g];
            it.rows = r1 - it.r0;
            int tl, tt, at;
            tile_coords(w - gstart[g], ntl, tiles_of(it.rows), p.group_m, tl, tt);
            grp_tile(it.rows, tt, at, it.width, tiles_of(it.rows));
            it.n0 = tl * 256;
            it.m0 = it.r0 + at;
            it.m1 = min(r1, it.m0 + it.width);
            it.kb = it.e < p.E ? (p.K - 1) / Cfg::BK + 1 : 0;
        }
        if (piece >= 0) {
            it.width = grp_piece_width(it.width, pieces);
            it.m0 += piece * it.width;
            it.m1 = min(it.m1, it.m0 + it.width);
            if (it.m0 >= it.m1) it.kb = 0;              // no rows left for this piece
        }
        return it;
    };
    // The next item.  Its six divisions take 900 clocks: of 4-bit products, whose tiles can
    // be nearly as short, a thread each works out the pair's first ITEMS, before the
    // roles part (8192 x 8192 x 1024 51 -> 47 us, x 512 47 -> 43, x 8192 191 -> 190).
    if constexpr (Cfg::ITEMS > 0) {
        const long long w = pair + static_cast<long long>(threadIdx.x) * npairs;
        if (threadIdx.x < Cfg::ITEMS && w < num_items) {
            const int i = static_cast<int>(w), t = i < dp ? i : dp + (i - dp) / pieces;
            int g = 0, after = *gcount;                     // gstart[g] <= t < gstart[after]
            while (after - g > 1) {
                const int mid = (g + after) >> 1;
                if (gstart[mid] <= t) g = mid;
                else after = mid;
            }
            const GrpItem it = item(i, g);
            gitem[threadIdx.x] = make_int4(it.m0, it.n0, it.width | max(it.m1 - it.m0, 0) << 16,
                                           it.kb ? it.e : it.e | 1 << 16);
        }
        __syncthreads();
    }
    auto next = [&](int w, GrpWalk& at) -> GrpItem {
        if constexpr (Cfg::ITEMS > 0) {
            if (at.i < Cfg::ITEMS) {
                const int4 v = gitem[at.i++];
                GrpItem it;
                it.m0 = v.x;
                it.n0 = v.y;
                it.width = v.z & 0xffff;
                it.m1 = v.x + (v.z >> 16);
                it.e = v.w & 0xffff;
                it.kb = v.w >> 16 ? 0 : (p.K - 1) / Cfg::BK + 1;
                it.r0 = it.rows = 0;                        // WG's
                return it;
            }
        }
        return item(w, at.g);
    };
    // WG: rows of the group in its last block, and whether they end inside an
    // MMA step
    auto last_rows = [&](const GrpItem& it) { return it.rows - (it.kb - 1) * Cfg::BK; };
    auto is_cut = [&](const GrpItem& it) { return it.kb > 0 && last_rows(it) % Cfg::MMA_K != 0; };

    if (warp == 0 || warp == 2 + Cfg::EPI_WARPS) {
        // ----------------------------------------------- TMA producers (both)
        // Two warps take the blocks in turn.  A thread issues a copy about
        // every 95 clocks and needs some 240 more for a block's wait and
        // arrival: with 3 to 5 copies a block that is more than the 512 (for
        // a 256-row tile) or 448 clocks of its MMAs, and one warp alone paced
        // the kernel (148 groups of 224 rows, K = 4096, weights K x N: 790
        // clocks a block).
        const uint32_t turn = warp == 0 ? 0 : 1;
        if (elect_one()) {
            uint32_t armed = 0, armed_par = 0, ld = 0;
            bool ok = true;
            GrpWalk at;
            for (int w = pair; w < num_items && ok; w += npairs) {
                const GrpItem it = next(w, at);
                const int n0 = it.n0 + static_cast<int>(rank) * 128;     // this CTA's lanes
                const int left = lanes_total - n0;
                const int hn = it.width >> 1;
                const int b0 = it.m0 + static_cast<int>(rank) * hn;      // this CTA's half of the N side
                // boxes entirely past the matrix edge are not loaded: they only
                // feed lanes and columns that are never stored
                const int a_live = left <= 0 ? 0 : (Cfg::CHUNK >= 128 || left > 64) ? 128 / Cfg::CHUNK : 1;
                const int b_left = p.N - b0;
                const int b_live = b_left <= 0 ? 0 : min(hn / 64, b_left > 64 ? 2 : 1);   // WG
                constexpr bool A_MN = Cfg::WG || Cfg::W_MN;
                const uint32_t a_bytes = A_MN ? a_live * (Cfg::BK * 128) : (a_live ? Cfg::A_STAGE : 0);
                // product: hn rows are whole boxes of 128, 64, 32 and 16; those that
                // start past the last row are not loaded either
                uint32_t b_boxes = 0;
                if constexpr (!Cfg::WG)
                    for (int box = 128; box >= 16; box >>= 1)
                        if ((hn & box) && b0 + (hn & -2 * box) < p.M) b_boxes |= box;
                const uint32_t b_bytes = Cfg::WG ? b_live * (Cfg::BK * 128) : b_boxes * 128;
                const bool cut_last = Cfg::WG && is_cut(it);
                for (int kb = 0; kb < it.kb; ++kb, ++ld) {
                    if (ld % Cfg::PRODUCERS != turn) continue;
                    const uint32_t s = ld % Cfg::STAGES;
                    const uint32_t ph = (ld / Cfg::STAGES) & 1;
                    if (!bounded_wait(&empty[s], ph ^ 1, abort_flag, limit, p.status)) { ok = false; break; }
                    if (p.inject == 1 && ld == 0 && pair == 0 && rank == 0) continue;   // debug
                    // a block that needs the fix-up completes on a barrier of its own
                    const bool fix = cut_last && kb == it.kb - 1;
                    const uint32_t fbar = mapa_shared(smem_u32(fix ? &cut[s] : &full[s]), 0);
                    mbar_arrive_expect_tx_cluster(fbar, a_bytes + b_bytes);
                    if (!fix) {
                        armed |= 1u << s;
                        armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    }
                    uint8_t* a_dst = smA + s * Cfg::A_STAGE;
                    uint8_t* b_dst = smB + s * Cfg::B_STAGE;
                    if constexpr (Cfg::WG) {
                        const int r = it.r0 + kb * Cfg::BK;
                        for (int j = 0; j < a_live; ++j)
                            tma_load_2d_pair(a_dst + j * (Cfg::BK * 128), &tmA, fbar, n0 + Cfg::CHUNK * j, r);
                        for (int j = 0; j < b_live; ++j)
                            tma_load_2d_pair(b_dst + j * (Cfg::BK * 128), &tmB, fbar, b0 + Cfg::CHUNK * j, r);
                    } else {
                        if constexpr (Cfg::W_MN) {
                            for (int j = 0; j < a_live; ++j)
                                tma_load_3d_pair(a_dst + j * (Cfg::BK * 128), &tmA, fbar, n0 + Cfg::CHUNK * j,
                                                 kb * Cfg::BK, it.e);
                        } else if (a_live) {
                            tma_load_3d_pair(a_dst, &tmA, fbar, kb * Cfg::BK, n0, it.e);
                        }
                        auto rows = [&](const CUtensorMap* map, int box) {
                            const int at = hn & -2 * box;
                            if (b_boxes & box) tma_load_2d_pair(b_dst + at * 128, map, fbar, kb * Cfg::BK, b0 + at);
                        };
                        rows(&tmB, 128);
                        rows(&tmB64, 64);
                        rows(&tmB32, 32);
                        rows(&tmB16, 16);
                    }
                }
            }
            if (!ok) {
                if (rank == 0)
                    for (int s = 0; s < Cfg::STAGES; ++s)
                        if (armed & (1u << s)) {
                            volatile int never = 0;
                            bounded_wait(&full[s], (armed_par >> s) & 1, &never, limit, p.status);
                        }
                // copies that complete on barriers this thread cannot wait on (the
                // leader's; a block under fix-up): a fixed 1 ms to land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(10000);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------ MMA issuer (leader only)
        if (rank == 0 && elect_one()) {
            if constexpr (Cfg::MX) {
                // A stage's MMAs take 512 clocks, and this thread not much less to issue
                // them: positions in the rings are counted, descriptors added to, and one
                // commit reaches both CTAs (8192 x 8192 x 8192 197 -> 189 us).
                uint32_t tl = 0;
                uint32_t s = 0, ph = 0;                              // this stage's slot and parity
                uint32_t old = Cfg::STAGES - 2, old_ph = 1;          // of the stage before the last
                uint32_t slot = 0, slot_ph = 0, set = 0;             // of the chunk; columns of its scales
                const uint64_t a0 = sw128_desc(smem_u32(smA), 16, 1024), b0 = sw128_desc(smem_u32(smB), 16, 1024);
                const uint64_t sf0 = scale_desc(smem_u32(smSf));
                int last_width = 0;
                bool ok = true;
                GrpWalk at;
                for (int w = pair; w < num_items && ok; w += npairs) {
                    const GrpItem it = next(w, at);
                    if (it.kb == 0) continue;
                    const uint32_t acc = tl & 1;
                    if (!bounded_wait(&tempty[acc], ((tl >> 1) & 1) ^ 1, abort_flag, limit, p.status)) { ok = false; break; }
                    // (tl - 1) / 2: the last tile's use of the other accumulator
                    if (last_width + it.width > Cfg::ACC_END &&
                        !bounded_wait(&tpart[acc ^ 1], ((tl - 1) >> 1) & 1, abort_flag, limit, p.status)) {
                        ok = false;
                        break;
                    }
                    last_width = it.width;
                    ++tl;
                    const uint32_t d_tmem = tmem_base + grp_acc_col<Cfg>(acc, it.width);
                    const uint32_t idesc = make_idesc_mx4(256, 0) | (static_cast<uint32_t>(it.width >> 3) << 17);
                    for (int kb = 0; kb < it.kb; ++kb) {
                        if (!(kb & 3) && !bounded_wait_cluster(&sfull[slot], slot_ph, abort_flag, limit, p.status)) {
                            ok = false;
                            break;
                        }
                        // two sets of columns in turn.  A copy runs before the MMAs issued
                        // after it, but its definition does not put it behind those issued
                        // before: the MMAs that read the set, of the stage before the last,
                        // have to be done.  (The wait took 8192 x 8192 x 8192 from 189
                        // to 202 us; sets of half a stage, four of them, 226: MMAs wait for
                        // copies in between.)
                        if (!bounded_wait(&empty[old], old_ph, abort_flag, limit, p.status)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sf = tmem_base + Cfg::ACC_END + set;
                        const uint64_t src = sf0 + ((slot * Cfg::SF_SLOT + (kb & 3) * 1024) >> 4);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            tmem_cp_scales_pair(sf + 4 * j, src + 32 * j);
                            tmem_cp_scales_pair(sf + 8 + 8 * j, src + (Cfg::SF_TILE >> 4) + 32 * j);
                            if (it.width > 128)
                                tmem_cp_scales_pair(sf + 12 + 8 * j, src + (Cfg::SF_TILE >> 3) + 32 * j);
                        }
                        if (!bounded_wait(&full[s], ph, abort_flag, limit, p.status)) { ok = false; break; }
                        tc_fence_after();
                        const uint64_t ad = a0 + s * (Cfg::A_STAGE >> 4), bd = b0 + s * (Cfg::B_STAGE >> 4);
#pragma unroll
                        for (int k = 0; k < Cfg::STEPS; ++k)         // 32 bytes of k along the 128-byte rows
                            mma_mx4_pair(d_tmem, ad + 2 * k, bd + 2 * k, idesc | mx4_scale_id(k & 1), kb != 0 || k != 0,
                                         sf + 4 * (k >> 1), sf + 8 + 8 * (k >> 1));
                        mma_commit_both(&empty[s]);                  // both CTAs' slots
                        if ((kb & 3) == 3 || kb == it.kb - 1) {
                            mma_commit_both(&sempty[slot]);
                            if (++slot == Cfg::SF_WARPS) slot = 0, slot_ph ^= 1;
                        }
                        if (++s == Cfg::STAGES) s = 0, ph ^= 1;
                        if (++old == Cfg::STAGES) old = 0, old_ph ^= 1;
                        set = Cfg::SF_COLS - set;
                    }
                    if (ok) mma_commit_both(&tfull[acc]);            // both CTAs' accumulators
                }
            } else {
                constexpr int A_MN = Cfg::WG || Cfg::W_MN;
                constexpr uint32_t idesc0 = Cfg::I8 ? make_idesc_i8(256, 0, A_MN, 0)
                                          : make_idesc(Cfg::TYPE, 256, 0, A_MN, Cfg::WG);
                uint32_t ld = 0, tl = 0;
                bool ok = true;
                GrpWalk at;
                for (int w = pair; w < num_items && ok; w += npairs) {
                    const GrpItem it = next(w, at);
                    if (it.kb == 0) continue;
                    const uint32_t acc = tl & 1;
                    const uint32_t aph = (tl >> 1) & 1;
                    if (!bounded_wait(&tempty[acc], aph ^ 1, abort_flag, limit, p.status)) { ok = false; break; }
                    ++tl;
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + grp_acc_col<Cfg>(acc, it.width);
                    const uint32_t idesc = idesc0 | (static_cast<uint32_t>(it.width >> 3) << 17);
                    for (int kb = 0; kb < it.kb; ++kb, ++ld) {
                        const uint32_t s = ld % Cfg::STAGES;
                        const uint32_t ph = (ld / Cfg::STAGES) & 1;
                        if (!bounded_wait(&full[s], ph, abort_flag, limit, p.status)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t a_addr = smem_u32(smA + s * Cfg::A_STAGE);
                        const uint32_t b_addr = smem_u32(smB + s * Cfg::B_STAGE);
                        const int steps = Cfg::WG && kb == it.kb - 1
                            ? (last_rows(it) + Cfg::MMA_K - 1) / Cfg::MMA_K : Cfg::STEPS;
#pragma unroll
                        for (int k = 0; k < Cfg::STEPS; ++k) {
                            if (Cfg::WG && k >= steps) break;
                            // K-major: 32 bytes of k along the 128-byte rows; MN-major:
                            // MMA_K rows of 128 bytes, 128-byte wide chunks LBO apart
                            const uint64_t ad = A_MN
                                ? sw128_desc(a_addr + k * Cfg::MMA_K * 128, Cfg::BK * 128, 1024)
                                : sw128_desc(a_addr + k * 32, 16, 1024);
                            const uint64_t bd = Cfg::WG
                                ? sw128_desc(b_addr + k * Cfg::MMA_K * 128, Cfg::BK * 128, 1024)
                                : sw128_desc(b_addr + k * 32, 16, 1024);
                            if constexpr (Cfg::I8) mma_i8_pair(d_tmem, ad, bd, idesc, kb != 0 || k != 0);
                            else mma_f16_pair(d_tmem, ad, bd, idesc, kb != 0 || k != 0);
                        }
                        const uint32_t e_loc = smem_u32(&empty[s]);
                        mma_commit_pair(mapa_shared(e_loc, 0));      // both CTAs' slots
                        mma_commit_pair(mapa_shared(e_loc, 1));
                    }
                    if (!ok) break;
                    const uint32_t f_loc = smem_u32(&tfull[acc]);
                    mma_commit_pair(mapa_shared(f_loc, 0));          // both CTAs' accumulators
                    mma_commit_pair(mapa_shared(f_loc, 1));
                }
            }
            mma_commit_pair(mapa_shared(smem_u32(drain), 0));
            volatile int never = 0;
            bounded_wait(drain, 0, &never, limit, p.status);
        }
        __syncwarp();
    } else if (warp >= 2 && warp < 2 + Cfg::EPI_WARPS) {
        // --------------------------------------------------- epilogue (both)
        const int q = warp & 3;
        const int half = (warp - 2) >> 2;
        uint8_t* stg = smStg + (warp - 2) * Cfg::NBUF * Cfg::STG_BUF;
        uint32_t tl = 0, nstore = 0;
        GrpWalk at;
        for (int w = pair; w < num_items; w += npairs) {
            const GrpItem it = next(w, at);
            const uint32_t acc = tl & 1;
            const uint32_t aph = (tl >> 1) & 1;
            if (it.kb) {
                ++tl;
                // the only wait that lasts a whole tile, however long its sum: 4 us
                // more for each block, of which 8 columns of 2^24 k take 0.3 us each
                if (!bounded_wait(&tfull[acc], aph, abort_flag, limit + it.kb * 4096ull, p.status)) break;
                tc_fence_after();
            }
            const uint32_t taddr = tmem_base + grp_acc_col<Cfg>(acc, it.width) + (static_cast<uint32_t>(q * 32) << 16);
            const int l0 = it.n0 + static_cast<int>(rank) * 128 + q * 32;
            if constexpr (Cfg::WG) grp_store_grad<Cfg>(&tmC, p, it, taddr, l0, half, lane, stg, nstore);
            else if constexpr (Cfg::MX) grp_store_values<Cfg>(p, it, taddr, l0, half, lane, stg, acc, &tpart[acc]);
            else grp_store_rows<Cfg>(p, it, taddr, l0, half, lane, stg);
            if (it.kb) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
            }
        }
        if constexpr (Cfg::WG) {
            if (lane == 0) bulk_wait<0>();
            __syncwarp();
        }
    } else {
        if constexpr (Cfg::MX) {
            // ---------------------------------------- block scales (4-bit, both)
            // Each CTA brings the scales of its own lanes and of all the tile's rows,
            // which may start anywhere, in asynchronous 16-byte copies: two lanes to a
            // row, a sector.  (8192 x 8192 x 8192: plain loads 376 us with 16 bytes of a
            // row at a time, their lines thrash what shared memory leaves of L1; boxes
            // of the copy engine 220, of 32 bytes 191: a chunk's 384 rows land late.)
            const int turn = warp - (3 + Cfg::EPI_WARPS);
            const uint32_t slot = smem_u32(smSf + turn * Cfg::SF_SLOT);
            uint32_t chunk = 0, uses = 0;
            bool ok = true;
            GrpWalk at;
            for (int w = pair; w < num_items && ok; w += npairs) {
                const GrpItem it = next(w, at);
                const int n0 = it.n0 + static_cast<int>(rank) * 128;
                const uint8_t* cols = p.col_blocks + it.e * p.block_plane;
                const int tiles = it.width > 128 ? 3 : 2;
                for (int c = 0; c < (it.kb + 3) / 4; ++c, ++chunk) {
                    if (static_cast<int>(chunk % Cfg::SF_WARPS) != turn) continue;
                    if (!bounded_wait(&sempty[turn], (uses & 1) ^ 1, abort_flag, limit, p.status)) { ok = false; break; }
                    ++uses;
                    load_scales(slot, cols, n0, p.N, p.block_ldb, 32 * c, p.blocks, lane);
                    load_scales(slot + Cfg::SF_TILE, p.row_blocks, it.m0, p.M, p.block_lda, 32 * c, p.blocks, lane);
                    if (tiles > 2)
                        load_scales(slot + 2 * Cfg::SF_TILE, p.row_blocks, it.m0 + 128, p.M, p.block_lda, 32 * c, p.blocks, lane);
                    cp_async_wait();
                    __syncwarp();
                    for (int i = 0; i < tiles; ++i) order_scales<2>(slot + i * Cfg::SF_TILE, lane);
                    // the copies into both CTAs' tensor memory are issued by the leader
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_release_cluster(mapa_shared(smem_u32(&sfull[turn]), 0));
                }
            }
        }
        // ------------------------------------------ fix-up (WG, leader only)
        if constexpr (Cfg::WG) {
            uint32_t ld = 0, seen = 0;                  // seen: parity of each slot's cut barrier
            GrpWalk at;
            for (int w = pair; w < num_items && rank == 0; w += npairs) {
                const GrpItem it = next(w, at);
                ld += it.kb;
                if (!is_cut(it)) continue;
                const uint32_t s = (ld - 1) % Cfg::STAGES;
                if (!bounded_wait(&cut[s], (seen >> s) & 1, abort_flag, limit, p.status)) break;
                seen ^= 1u << s;
                // rows [first, end of its MMA step) of both operands, both
                // 64-column chunks: a row is 128 bytes of each chunk
                const int first = last_rows(it);
                const int count = (first + Cfg::MMA_K - 1) / Cfg::MMA_K * Cfg::MMA_K - first;
                const uint32_t a = smem_u32(smA + s * Cfg::A_STAGE + first * 128);
                const uint32_t b = smem_u32(smB + s * Cfg::B_STAGE + first * 128);
                for (int r = 0; r < 2; ++r) {
                    const uint32_t ar = mapa_shared(a, r), br = mapa_shared(b, r);
                    for (int i = lane; i < count * 8; i += 32) {
                        clear_cluster(ar + i * 16);
                        clear_cluster(ar + Cfg::BK * 128 + i * 16);
                        clear_cluster(br + i * 16);
                        clear_cluster(br + Cfg::BK * 128 + i * 16);
                    }
                }
                // The zeros, the peer's too, come from the CTA whose thread issues
                // the MMA over both CTAs' shared memory: the proxy fence and an
                // arrival within the CTA order them.  Where each CTA clears its
                // own, the peer's arrival has to release at cluster scope, which
                // waits for a memory barrier: 32 groups of 1001 and 1047 rows then
                // take 444 us, so 415.
                fence_proxy_async_cluster();
                __syncwarp();
                if (lane == 0) mbar_arrive_two(&full[s]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();          // the pair is done with each other's barriers and TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace tg
