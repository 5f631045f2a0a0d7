// launch.h -- internal interface between the C ABI shim and the launchers.
// Arguments arrive here already validated (sizes, pointers, alignment).
#pragma once
#include <cstdint>

#include "tune.h"

namespace tg {

// Internal status values; identical to the tg_status codes.
enum : int { kOk = 0, kInvalidArg = 1, kAlignment = 2, kUnsupported = 3, kCudaError = 4,
             kTimeout = 5, kNoDevice = 6 };

struct GemmArgs {
    int64_t M, N, K;
    const void* A; int64_t lda;      // elements
    const void* B; int64_t ldb;      // elements (bytes for packed 4-bit weights)
    void* C; int64_t ldc;            // elements
    const void* scales; int64_t lds; // 4-bit paths only (lds: elements, bytes for E8M0 scales)
    int group;                       // 4-bit paths only
    int relu;
    void* stream;
    // launch shape from the tuning table (tune.h); 0 = the launcher's default
    int path;                        // TunePath: kernel family
    int ctas;                        // persistent CTAs (CTA pairs), stream-K ranges
    int group_m;                     // raster band height in tiles
    int splits;                      // fp32 FFMA split-K ranges
    int stages;                      // 16-bit CTA-pair ring depth (4 or 6)
};

// The arguments with a tuning rule's launch-shape fields.
inline GemmArgs with_rule(GemmArgs a, const TuneRule& r) {
    a.path = r.path;
    a.ctas = r.ctas;
    a.group_m = r.group_m;
    a.splits = r.splits;
    a.stages = r.stages;
    return a;
}

// Persistent grid size: `units` of work over at most `cap` CTAs (the rule's
// CTA count when set, else all of `cap`).
inline long long persistent_grid(long long units, int cap, int ctas) {
    const long long c = ctas > 0 && ctas < cap ? ctas : cap;
    return units < c ? units : c;
}

// Products over groups of rows (gemm_group.cuh): g.M rows of A, K columns,
// weights (or, for the weight gradient, the rows' gradient) in g.B.
struct GroupArgs {
    GemmArgs g;
    int E;                           // groups
    const int* offsets;              // device, E + 1; null: one group of all rows (E = 1)
    int trans_b;                     // weights stored N x K
    int64_t plane_b;                 // elements between the weights of two groups
    int64_t plane;                   // weight gradient: elements between two matrices of C
    const float* row_scale;          // 8-bit only: g.M
    const float* col_scale;          // 8-bit only: N per group, scale_plane apart
    int64_t scale_plane;
};
int launch_group(const GroupArgs& a, int bf16);
int launch_group_grad(const GroupArgs& a, int bf16);
int launch_group_i8(const GroupArgs& a, int bf16);
// One group of all rows: the weight-streaming or the CTA-pair kernel.
int launch_w8a8(const GroupArgs& a, int bf16);

// Rows of 16-bit values to 8-bit integers with one scale per row.
int launch_quant_i8(int64_t M, int64_t K, const void* X, int64_t ldx, int bf16, int8_t* Q,
                    int64_t ldq, float* scales, void* stream);
// Tokens sorted by expert, and back (expert.cu).
int64_t expert_sort_scratch(int64_t n, int E);
int launch_expert_sort(int64_t tokens, int topk, int E, const void* ids, int id_bytes, int* offsets,
                       int* pos, int* src, void* scratch, void* stream);
int launch_expert_gather(int64_t tokens, int topk, int64_t H, int eb, const void* X, int64_t ldx,
                         const float* scales, const int* pos, const int* kept, void* out,
                         int64_t ldo, float* out_scales, void* stream);
int launch_expert_combine(int64_t tokens, int topk, int64_t H, int bf16, const void* Y, int64_t ldy,
                          const int* pos, const int* kept, const float* weights, void* out,
                          int64_t ldo, void* stream);
int launch_expert_combine_grad(int64_t tokens, int topk, int64_t H, int bf16, const void* Y,
                               int64_t ldy, const void* dout, int64_t ldd, const int* pos,
                               const int* kept, const float* weights, void* dY, int64_t lddy,
                               float* dweights, void* stream);

int launch_tc_bf16(const GemmArgs& a);
int launch_tc_f16(const GemmArgs& a);
int launch_tc_tf32(const GemmArgs& a);
int launch_tc_trans(const GemmArgs& a, int bf16, int trans_a, int trans_b);
int launch_ffma_f32(const GemmArgs& a);
int launch_w4a16(const GemmArgs& a);
int launch_w4a16_large(const GemmArgs& a);
int launch_w4a16_pair(const GemmArgs& a);
// FP4 (E2M1 + E8M0) weights, bf16 activations: scales / lds in bytes.
int launch_wfp4(const GemmArgs& a);
int launch_wfp4_large(const GemmArgs& a);
int launch_wfp4_pair(const GemmArgs& a);
int launch_skinny_wfp4(const GemmArgs& a);
// 2:4 sparse A: a.A / a.lda are the compressed values, E / lde the codes.
int launch_sp24(const GemmArgs& a, const void* E, int64_t lde, int bf16);
int launch_skinny_bf16(const GemmArgs& a);
int launch_skinny_f16(const GemmArgs& a);
int launch_skinny_w4a16(const GemmArgs& a);
// 16-bit weights stored transposed (B is N x K): the weight-streaming kernel
// reading K-major weight tiles.
int launch_skinny_trans_b(const GemmArgs& a, int bf16);
int launch_gemv_bf16(const GemmArgs& a);
int launch_gemv_f16(const GemmArgs& a);
int launch_gemv_w4a16(const GemmArgs& a);
int launch_gemv_wfp4(const GemmArgs& a);
void mark_workspaces_dirty(int dev);
// The argument checks every 16-bit and fp32 entry point runs before any CUDA
// call (sizes, pointers, leading dimensions, the row-pitch bound, alignment)
// for elements of `eb` bytes; returns a tg_status value.
int check_gemm_args(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                    int64_t ldb, const void* C, int64_t ldc, int epilogue, int eb);
// Per-(device, stream) scratch of the split-K paths: `tickets` ints (zero
// between calls) and `partial_bytes` of fp32 partials.
bool stream_workspace(int dev, void* stream, long long tickets, long long partial_bytes,
                      int** tk, float** part);

// Activation rows up to which the CUDA-core kernel is used.
constexpr long long kGemvMaxM = 4;
// Activation rows up to which the weight-streaming kernel is used.
constexpr long long kSkinnyMaxM = 128;

}  // namespace tg
