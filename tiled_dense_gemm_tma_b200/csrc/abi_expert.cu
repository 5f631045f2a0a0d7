// abi_expert.cu -- the C ABI of the 8-bit and microscaled 4-bit linear layers and
// the experts' operators: argument validation and dispatch.  As in abi.cu every check runs
// before any CUDA call.
#include "../../include/tg_gemm.h"
#include "launch.h"
#include "host.cuh"

#include <cuda_runtime.h>

#include <initializer_list>

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1;      // kernel indices and TMA coords are int32
constexpr int64_t kMaxTiled = kMaxDim - 1024;     // a tile past the last row stays inside 32 bits
constexpr int64_t kMaxK8 = 131071;                // 128 * 128 * K stays inside 32 bits
constexpr int kMaxExperts = 1024;                 // the kernels' tables in shared memory

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A matrix of `rows` x `cols` elements of eb bytes: what is wrong with its
// pointer and pitch, in the order of the header's codes.
tg_status check_matrix(const void* p, int64_t ld, int64_t cols, int eb) {
    if (!p || ld < cols) return TG_ERR_INVALID_ARG;
    if (ld >= (1ll << 40) / eb) return TG_ERR_UNSUPPORTED;       // TMA stride limit
    if (!aligned(p, 16) || (ld * eb) % 16 != 0) return TG_ERR_ALIGNMENT;
    return TG_OK;
}

// The distance between the matrices of E groups.
tg_status check_plane(int64_t plane, int E, int eb) {
    if (E == 1) return TG_OK;
    if (plane <= 0) return TG_ERR_INVALID_ARG;
    if (plane >= (1ll << 40) / eb) return TG_ERR_UNSUPPORTED;
    return (plane * eb) % 16 != 0 ? TG_ERR_ALIGNMENT : TG_OK;
}

// The first status that is not TG_OK, invalid arguments before limits before
// alignment.
tg_status worst(std::initializer_list<tg_status> all) {
    for (tg_status want : {TG_ERR_INVALID_ARG, TG_ERR_UNSUPPORTED, TG_ERR_ALIGNMENT})
        for (tg_status s : all)
            if (s == want) return s;
    return TG_OK;
}

tg_status float_ptr(const void* p) {
    return !p ? TG_ERR_INVALID_ARG : aligned(p, 4) ? TG_OK : TG_ERR_ALIGNMENT;
}

bool bad_type(int type) { return type != TG_TYPE_F16 && type != TG_TYPE_BF16; }

tg::GroupArgs group_args(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda,
                         const int32_t* offsets, const void* B, int64_t ldb, int64_t plane_b,
                         int trans_b, void* C, int64_t ldc, int epilogue, void* stream) {
    tg::GroupArgs a = {};
    a.g.M = M; a.g.N = N; a.g.K = K;
    a.g.A = A; a.g.lda = lda; a.g.B = B; a.g.ldb = ldb; a.g.C = C; a.g.ldc = ldc;
    a.g.relu = epilogue == TG_EPI_RELU;
    a.g.stream = stream;
    a.E = E;
    a.offsets = offsets;
    a.trans_b = trans_b;
    a.plane_b = plane_b;
    return a;
}

tg_status zero_rows(void* C, int64_t ldc, int64_t M, int64_t N, void* stream) {
    if (!tg::current_device(nullptr)) return TG_ERR_NO_DEVICE;
    return cudaMemset2DAsync(C, static_cast<size_t>(ldc * 2), 0, static_cast<size_t>(N * 2), static_cast<size_t>(M),
                             static_cast<cudaStream_t>(stream)) == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}

// The checks that every product over groups shares; *done: nothing to launch.
tg_status check_product(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda,
                        const void* B, int64_t ldb, int64_t plane_b, int trans_b, void* C, int64_t ldc,
                        int epilogue, int eb, void* stream, bool* done) {
    *done = true;
    if (M < 0 || N < 0 || K < 0 || E < 1) return TG_ERR_INVALID_ARG;
    if (epilogue != TG_EPI_NONE && epilogue != TG_EPI_RELU) return TG_ERR_INVALID_ARG;
    if (trans_b != 0 && trans_b != 1) return TG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TG_OK;
    tg_status s = worst({check_matrix(C, ldc, N, 2), K > 0 ? check_matrix(A, lda, K, eb) : TG_OK,
                         K > 0 ? check_matrix(B, ldb, trans_b ? K : N, eb) : TG_OK,
                         K > 0 ? check_plane(plane_b, E, eb) : TG_OK,
                         (M > kMaxTiled || N > kMaxTiled || K > kMaxTiled || E > kMaxExperts) ? TG_ERR_UNSUPPORTED : TG_OK,
                         (eb == 1 && K > kMaxK8) ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    if (K == 0) return zero_rows(C, ldc, M, N, stream);
    *done = false;
    return TG_OK;
}

tg_status grouped16(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda, const int32_t* offsets,
                    const void* B, int64_t ldb, int64_t plane_b, int trans_b, void* C, int64_t ldc,
                    int epilogue, void* stream, int bf16) {
    if (M > 0 && N > 0 && float_ptr(offsets) != TG_OK) return float_ptr(offsets);
    bool done;
    const tg_status s = check_product(M, N, K, E, A, lda, B, ldb, plane_b, trans_b, C, ldc, epilogue, 2, stream, &done);
    if (s != TG_OK || done) return s;
    return static_cast<tg_status>(tg::launch_group(
        group_args(M, N, K, E, A, lda, offsets, B, ldb, plane_b, trans_b, C, ldc, epilogue, stream), bf16));
}

tg_status wgrad16(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda, const void* G, int64_t ldg,
                  const int32_t* offsets, void* C, int64_t ldc, int64_t plane_c, void* stream, int bf16) {
    if (M < 0 || N < 0 || K < 0 || E < 1) return TG_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return TG_OK;
    const bool overlap = E > 1 && plane_c < static_cast<__int128>(K - 1) * ldc + N;
    tg_status s = worst({check_matrix(C, ldc, N, 2), M > 0 ? check_matrix(A, lda, K, 2) : TG_OK,
                         M > 0 ? check_matrix(G, ldg, N, 2) : TG_OK, check_plane(plane_c, E, 2),
                         M > 0 ? float_ptr(offsets) : TG_OK, overlap ? TG_ERR_INVALID_ARG : TG_OK,
                         (M > kMaxTiled || N > kMaxTiled || K > kMaxTiled || E > kMaxExperts) ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    if (M == 0) {
        for (int e = 0; e < E && s == TG_OK; ++e)
            s = zero_rows(static_cast<char*>(C) + (E > 1 ? e * plane_c * 2 : 0), ldc, K, N, stream);
        return s;
    }
    tg::GroupArgs a = group_args(M, N, K, E, A, lda, offsets, G, ldg, 0, 0, C, ldc, TG_EPI_NONE, stream);
    a.plane = plane_c;
    return static_cast<tg_status>(tg::launch_group_grad(a, bf16));
}

}  // namespace

extern "C" {

tg_status tg_quant_i8(int64_t M, int64_t K, const void* X, int64_t ldx, int type, int8_t* Q, int64_t ldq,
                      float* scales, void* stream) {
    if (M < 0 || K < 0 || bad_type(type)) return TG_ERR_INVALID_ARG;
    if (M == 0) return TG_OK;
    const tg_status s = worst({K > 0 ? check_matrix(X, ldx, K, 2) : TG_OK, K > 0 ? check_matrix(Q, ldq, K, 1) : TG_OK,
                               float_ptr(scales), (M > kMaxDim || K > kMaxDim) ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_quant_i8(M, K, X, ldx, type == TG_TYPE_BF16, Q, ldq, scales, stream));
}

tg_status tg_gemm_w8a8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* row_scales,
                       const int8_t* B, int64_t ldb, int trans_b, const float* col_scales, void* C, int64_t ldc,
                       int type, int epilogue, void* stream) {
    if (bad_type(type)) return TG_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && K > 0) {
        const tg_status s = worst({float_ptr(row_scales), float_ptr(col_scales)});
        if (s != TG_OK) return s;
    }
    bool done;
    const tg_status s = check_product(M, N, K, 1, A, lda, B, ldb, 0, trans_b, C, ldc, epilogue, 1, stream, &done);
    if (s != TG_OK || done) return s;
    tg::GroupArgs a = group_args(M, N, K, 1, A, lda, nullptr, B, ldb, 0, trans_b, C, ldc, epilogue, stream);
    a.row_scale = row_scales;
    a.col_scale = col_scales;
    return static_cast<tg_status>(tg::launch_w8a8(a, type == TG_TYPE_BF16));
}

tg_status tg_gemm_grouped_f16(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda,
                              const int32_t* offsets, const void* B, int64_t ldb, int64_t plane_b, int trans_b,
                              void* C, int64_t ldc, int epilogue, void* stream) {
    return grouped16(M, N, K, E, A, lda, offsets, B, ldb, plane_b, trans_b, C, ldc, epilogue, stream, 0);
}

tg_status tg_gemm_grouped_bf16(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda,
                               const int32_t* offsets, const void* B, int64_t ldb, int64_t plane_b, int trans_b,
                               void* C, int64_t ldc, int epilogue, void* stream) {
    return grouped16(M, N, K, E, A, lda, offsets, B, ldb, plane_b, trans_b, C, ldc, epilogue, stream, 1);
}

tg_status tg_gemm_grouped_wgrad_f16(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda,
                                    const void* G, int64_t ldg, const int32_t* offsets, void* C, int64_t ldc,
                                    int64_t plane_c, void* stream) {
    return wgrad16(M, N, K, E, A, lda, G, ldg, offsets, C, ldc, plane_c, stream, 0);
}

tg_status tg_gemm_grouped_wgrad_bf16(int64_t M, int64_t N, int64_t K, int E, const void* A, int64_t lda,
                                     const void* G, int64_t ldg, const int32_t* offsets, void* C, int64_t ldc,
                                     int64_t plane_c, void* stream) {
    return wgrad16(M, N, K, E, A, lda, G, ldg, offsets, C, ldc, plane_c, stream, 1);
}

tg_status tg_gemm_grouped_w8a8(int64_t M, int64_t N, int64_t K, int E, const int8_t* A, int64_t lda,
                               const float* row_scales, const int32_t* offsets, const int8_t* B, int64_t ldb,
                               int64_t plane_b, int trans_b, const float* col_scales, int64_t plane_s, void* C,
                               int64_t ldc, int type, int epilogue, void* stream) {
    if (bad_type(type)) return TG_ERR_INVALID_ARG;
    if (M > 0 && N > 0) {
        const tg_status s = worst({float_ptr(offsets), K > 0 ? float_ptr(row_scales) : TG_OK,
                                   K > 0 ? float_ptr(col_scales) : TG_OK,
                                   (K > 0 && E > 1 && plane_s < 0) ? TG_ERR_INVALID_ARG : TG_OK});
        if (s != TG_OK) return s;
    }
    bool done;
    const tg_status s = check_product(M, N, K, E, A, lda, B, ldb, plane_b, trans_b, C, ldc, epilogue, 1, stream, &done);
    if (s != TG_OK || done) return s;
    tg::GroupArgs a = group_args(M, N, K, E, A, lda, offsets, B, ldb, plane_b, trans_b, C, ldc, epilogue, stream);
    a.row_scale = row_scales;
    a.col_scale = col_scales;
    a.scale_plane = plane_s;
    return static_cast<tg_status>(tg::launch_group_i8(a, type == TG_TYPE_BF16));
}

namespace {

tg_status check_choices(int64_t tokens, int topk) {
    if (tokens < 0 || topk < 1) return TG_ERR_INVALID_ARG;
    return tokens > kMaxDim / topk ? TG_ERR_UNSUPPORTED : TG_OK;
}

}  // namespace

int64_t tg_expert_sort_scratch(int64_t choices, int E) {
    if (choices < 0 || choices > kMaxDim || E < 1 || E > kMaxExperts) return -1;
    return tg::expert_sort_scratch(choices, E);
}

tg_status tg_expert_sort(int64_t tokens, int topk, int E, const void* ids, int id_bytes, int32_t* offsets,
                         int32_t* pos, int32_t* src, void* scratch, void* stream) {
    if (E < 1 || (id_bytes != 4 && id_bytes != 8)) return TG_ERR_INVALID_ARG;
    tg_status s = check_choices(tokens, topk);
    if (s != TG_OK) return s;
    const bool any = tokens > 0;
    s = worst({float_ptr(offsets), any ? float_ptr(pos) : TG_OK, any ? float_ptr(src) : TG_OK,
               !any ? TG_OK : !ids ? TG_ERR_INVALID_ARG : aligned(ids, id_bytes) ? TG_OK : TG_ERR_ALIGNMENT,
               E > kMaxExperts ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    if (tg::expert_sort_scratch(tokens * topk, E) > 0 && float_ptr(scratch) != TG_OK) return float_ptr(scratch);
    return static_cast<tg_status>(tg::launch_expert_sort(tokens, topk, E, ids, id_bytes, offsets, pos, src, scratch, stream));
}

tg_status tg_expert_gather(int64_t tokens, int topk, int64_t H, int elem_bytes, const void* X, int64_t ldx,
                           const float* scales, const int32_t* pos, const int32_t* kept, void* out, int64_t ldo,
                           float* out_scales, void* stream) {
    if (H < 0 || (elem_bytes != 1 && elem_bytes != 2) || (scales == nullptr) != (out_scales == nullptr))
        return TG_ERR_INVALID_ARG;
    tg_status s = check_choices(tokens, topk);
    if (s != TG_OK) return s;
    if (tokens == 0 || (H == 0 && !scales)) return TG_OK;
    s = worst({H > 0 ? check_matrix(X, ldx, H, elem_bytes) : TG_OK, H > 0 ? check_matrix(out, ldo, H, elem_bytes) : TG_OK,
               float_ptr(pos), float_ptr(kept), scales ? float_ptr(scales) : TG_OK,
               scales ? float_ptr(out_scales) : TG_OK, H > kMaxDim ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_expert_gather(tokens, topk, H, elem_bytes, X, ldx, scales, pos, kept,
                                                           out, ldo, out_scales, stream));
}

tg_status tg_expert_combine(int64_t tokens, int topk, int64_t H, int type, const void* Y, int64_t ldy,
                            const int32_t* pos, const int32_t* kept, const float* weights, void* out,
                            int64_t ldo, void* stream) {
    if (H < 0 || bad_type(type)) return TG_ERR_INVALID_ARG;
    tg_status s = check_choices(tokens, topk);
    if (s != TG_OK || tokens == 0 || H == 0) return s;
    s = worst({check_matrix(Y, ldy, H, 2), check_matrix(out, ldo, H, 2), float_ptr(pos), float_ptr(kept),
               weights ? float_ptr(weights) : TG_OK, H > kMaxDim ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_expert_combine(tokens, topk, H, type == TG_TYPE_BF16, Y, ldy, pos, kept,
                                                            weights, out, ldo, stream));
}

tg_status tg_expert_combine_grad(int64_t tokens, int topk, int64_t H, int type, const void* Y, int64_t ldy,
                                 const void* dout, int64_t ldd, const int32_t* pos, const int32_t* kept,
                                 const float* weights, void* dY, int64_t lddy, float* dweights, void* stream) {
    if (H < 0 || bad_type(type)) return TG_ERR_INVALID_ARG;
    tg_status s = check_choices(tokens, topk);
    if (s != TG_OK || tokens == 0) return s;
    s = worst({H > 0 ? check_matrix(Y, ldy, H, 2) : TG_OK, H > 0 ? check_matrix(dout, ldd, H, 2) : TG_OK,
               H > 0 ? check_matrix(dY, lddy, H, 2) : TG_OK, float_ptr(pos), float_ptr(kept), float_ptr(weights),
               float_ptr(dweights), H > kMaxDim ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_expert_combine_grad(tokens, topk, H, type == TG_TYPE_BF16, Y, ldy, dout,
                                                                 ldd, pos, kept, weights, dY, lddy, dweights, stream));
}

namespace {

// Codes and scales of `rows` rows of K values.
tg_status check_blocks(const void* q, int64_t ldq, const void* scales, int64_t lds, int64_t K) {
    return worst({check_matrix(q, ldq, (K + 1) / 2, 1), check_matrix(scales, lds, (K + 31) / 32, 1)});
}

tg_status mxfp4(int64_t M, int64_t N, int64_t K, int E, const uint8_t* A, int64_t lda, const uint8_t* a_scales,
                int64_t ldas, const int32_t* offsets, const uint8_t* B, int64_t ldb, int64_t plane_b,
                const uint8_t* b_scales, int64_t ldbs, int64_t plane_s, void* C, int64_t ldc, int type,
                int epilogue, void* stream) {
    if (M < 0 || N < 0 || K < 0 || E < 1 || bad_type(type)) return TG_ERR_INVALID_ARG;
    if (epilogue != TG_EPI_NONE && epilogue != TG_EPI_RELU) return TG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TG_OK;
    const tg_status s = worst({check_matrix(C, ldc, N, 2), K > 0 ? check_blocks(A, lda, a_scales, ldas, K) : TG_OK,
                               K > 0 ? check_blocks(B, ldb, b_scales, ldbs, K) : TG_OK,
                               K > 0 ? check_plane(plane_b, E, 1) : TG_OK, K > 0 ? check_plane(plane_s, E, 1) : TG_OK,
                               (M > kMaxTiled || N > kMaxTiled || K > kMaxTiled || E > kMaxExperts) ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    if (K == 0) return zero_rows(C, ldc, M, N, stream);
    tg::GroupArgs a = group_args(M, N, (K + 1) / 2, E, A, lda, offsets, B, ldb, plane_b, 1, C, ldc, epilogue, stream);
    a.row_blocks = a_scales;
    a.block_lda = ldas;
    a.col_blocks = b_scales;
    a.block_ldb = ldbs;
    a.block_plane = plane_s;
    a.blocks = (K + 31) / 32;
    const int bf16 = type == TG_TYPE_BF16;
    return static_cast<tg_status>(offsets ? tg::launch_group_mx4(a, bf16) : tg::launch_mx4(a, bf16));
}

// Logits or their gradient: any pitch, the elements' own alignment.
tg_status check_logits(const void* p, int64_t ld, int E, int type) {
    const int eb = type == TG_TYPE_F32 ? 4 : 2;
    if (!p || ld < E) return TG_ERR_INVALID_ARG;
    if (ld >= (1ll << 40) / eb) return TG_ERR_UNSUPPORTED;
    return aligned(p, eb) ? TG_OK : TG_ERR_ALIGNMENT;
}

// What both directions of the routing check.
tg_status check_route(int64_t tokens, int E, const void* logits, int64_t ldl, int type, int score, int topk, int renorm,
                      const void* ids, const void* weights) {
    if (tokens < 0 || E < 1 || topk < 1 || topk > E) return TG_ERR_INVALID_ARG;
    if (type != TG_TYPE_F16 && type != TG_TYPE_BF16 && type != TG_TYPE_F32) return TG_ERR_INVALID_ARG;
    if ((score != TG_SCORE_SOFTMAX && score != TG_SCORE_SIGMOID) || (renorm != 0 && renorm != 1)) return TG_ERR_INVALID_ARG;
    if (tokens == 0) return E > kMaxExperts || topk > 32 ? TG_ERR_UNSUPPORTED : TG_OK;
    return worst({check_logits(logits, ldl, E, type), float_ptr(ids), float_ptr(weights),
                  (tokens > kMaxDim || E > kMaxExperts || topk > 32) ? TG_ERR_UNSUPPORTED : TG_OK});
}

}  // namespace

tg_status tg_quant_mxfp4(int64_t M, int64_t K, const void* X, int64_t ldx, int type, uint8_t* Q, int64_t ldq,
                         uint8_t* scales, int64_t lds, void* stream) {
    if (M < 0 || K < 0 || bad_type(type)) return TG_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return TG_OK;
    const tg_status s = worst({check_matrix(X, ldx, K, 2), check_blocks(Q, ldq, scales, lds, K),
                               (M > kMaxDim || K > kMaxTiled) ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_quant_mxfp4(M, K, X, ldx, type == TG_TYPE_BF16, 1, nullptr, nullptr, Q, ldq,
                                                         scales, lds, stream));
}

tg_status tg_dequant_mxfp4(int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* scales, int64_t lds,
                           void* Y, int64_t ldy, int type, void* stream) {
    if (M < 0 || K < 0 || bad_type(type)) return TG_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return TG_OK;
    const tg_status s = worst({check_matrix(Y, ldy, K, 2), check_blocks(Q, ldq, scales, lds, K),
                               (M > kMaxDim || K > kMaxTiled) ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_dequant_mxfp4(M, K, Q, ldq, scales, lds, Y, ldy, type == TG_TYPE_BF16, stream));
}

tg_status tg_expert_quant_mxfp4(int64_t tokens, int topk, int64_t K, const void* X, int64_t ldx, int type,
                                const int32_t* pos, const int32_t* kept, uint8_t* Q, int64_t ldq, uint8_t* scales,
                                int64_t lds, void* stream) {
    if (K < 0 || bad_type(type)) return TG_ERR_INVALID_ARG;
    tg_status s = check_choices(tokens, topk);
    if (s != TG_OK || tokens == 0 || K == 0) return s;
    s = worst({check_matrix(X, ldx, K, 2), check_blocks(Q, ldq, scales, lds, K), float_ptr(pos), float_ptr(kept),
               K > kMaxTiled ? TG_ERR_UNSUPPORTED : TG_OK});
    if (s != TG_OK) return s;
    return static_cast<tg_status>(tg::launch_quant_mxfp4(tokens, K, X, ldx, type == TG_TYPE_BF16, topk, pos, kept, Q, ldq,
                                                         scales, lds, stream));
}

tg_status tg_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const uint8_t* a_scales,
                        int64_t ldas, const uint8_t* B, int64_t ldb, const uint8_t* b_scales, int64_t ldbs, void* C,
                        int64_t ldc, int type, int epilogue, void* stream) {
    return mxfp4(M, N, K, 1, A, lda, a_scales, ldas, nullptr, B, ldb, 0, b_scales, ldbs, 0, C, ldc, type, epilogue, stream);
}

tg_status tg_gemm_grouped_mxfp4(int64_t M, int64_t N, int64_t K, int E, const uint8_t* A, int64_t lda,
                                const uint8_t* a_scales, int64_t ldas, const int32_t* offsets, const uint8_t* B,
                                int64_t ldb, int64_t plane_b, const uint8_t* b_scales, int64_t ldbs, int64_t plane_s,
                                void* C, int64_t ldc, int type, int epilogue, void* stream) {
    if (M > 0 && N > 0 && float_ptr(offsets) != TG_OK) return float_ptr(offsets);
    return mxfp4(M, N, K, E, A, lda, a_scales, ldas, offsets, B, ldb, plane_b, b_scales, ldbs, plane_s, C, ldc, type,
                 epilogue, stream);
}

tg_status tg_expert_route(int64_t tokens, int E, const void* logits, int64_t ldl, int type, const float* bias, int score,
                          int groups, int keep_groups, int topk, int renorm, float scale, int32_t* ids, float* weights,
                          void* stream) {
    if (groups < 1 || E < 1 || groups > E || E % groups != 0 || keep_groups < 1 || keep_groups > groups) return TG_ERR_INVALID_ARG;
    if (topk > keep_groups * static_cast<int64_t>(E / groups)) return TG_ERR_INVALID_ARG;
    tg_status s = check_route(tokens, E, logits, ldl, type, score, topk, renorm, ids, weights);
    if (s == TG_ERR_INVALID_ARG) return s;
    s = worst({s, groups > 32 ? TG_ERR_UNSUPPORTED : TG_OK,
               bias && tokens > 0 ? float_ptr(bias) : TG_OK});
    if (s != TG_OK || tokens == 0) return s;
    tg::RouteArgs a = {};
    a.tokens = tokens; a.E = E; a.groups = groups; a.keep = keep_groups; a.topk = topk;
    a.type = type; a.sigmoid = score == TG_SCORE_SIGMOID; a.renorm = renorm; a.scale = scale;
    a.logits = logits; a.ldl = ldl; a.bias = bias; a.ids = ids; a.weights = weights;
    a.stream = stream;
    return static_cast<tg_status>(tg::launch_route(a));
}

tg_status tg_expert_route_grad(int64_t tokens, int E, const void* logits, int64_t ldl, int type, int score, int topk,
                               int renorm, float scale, const int32_t* ids, const float* dweights, void* dlogits,
                               int64_t ldd, void* stream) {
    tg_status s = check_route(tokens, E, logits, ldl, type, score, topk, renorm, ids, dweights);
    if (s == TG_ERR_INVALID_ARG || tokens == 0) return s;
    s = worst({s, check_logits(dlogits, ldd, E, type)});
    if (s != TG_OK) return s;
    tg::RouteArgs a = {};
    a.tokens = tokens; a.E = E; a.groups = 1; a.keep = 1; a.topk = topk;
    a.type = type; a.sigmoid = score == TG_SCORE_SIGMOID; a.renorm = renorm; a.scale = scale;
    a.logits = logits; a.ldl = ldl; a.ids = const_cast<int32_t*>(ids); a.dweights = dweights;
    a.dlogits = dlogits; a.ldd = ldd;
    a.stream = stream;
    return static_cast<tg_status>(tg::launch_route_grad(a));
}

}  // extern "C"
