// gemm_skinny_i8.cu -- launcher of the weight-streaming kernel for 8-bit
// weights and activations with at most 128 rows.
#include "gemm_skinny.cuh"
#include "host.cuh"
#include "launch.h"

namespace tg {

namespace {

// CTAs a 128-column group is split over: the most of 4, 2, 1 that leave every
// CTA k-units of its own and all groups on the device at once; 1 where the
// groups alone fill it.  Unlike skinny_cluster_split it never asks for
// stream-K, whose partials would need a workspace: 8192 x 8192 weights take
// 64 x 2 CTAs either way.
template <class Cfg>
int split(long long T, long long KB, int num_sms, int slot) {
    static_assert(Cfg::CL_OK, "partials fit the ring");
    for (int S = 4; S > 1; S >>= 1) {
        if (S > KB || T * S > num_sms) continue;
        if (max_active_clusters(reinterpret_cast<const void*>(skinny_kernel<Cfg>), slot, S, Cfg::THREADS,
                                Cfg::SMEM_BYTES) >= T)
            return S;
    }
    return 1;
}

template <int MPAD, int WK>
int run(const GroupArgs& a, int bf16, int slot) {
    using Cfg = SkCfg<WKind::I8, MPAD, WK>;
    const DeviceInfo* di = current_device(nullptr);
    if (!di) return kNoDevice;
    const GemmArgs& g = a.g;
    const long long T = (g.N + Cfg::GN - 1) / Cfg::GN, KB = (g.K + Cfg::BK - 1) / Cfg::BK;
    if (T * KB > 0x7fffffffll) return kUnsupported;
    auto kern = skinny_kernel<Cfg>;
    if (set_smem_attr(reinterpret_cast<const void*>(kern), Cfg::SMEM_BYTES, slot) != cudaSuccess) return kCudaError;
    const int S = split<Cfg>(T, KB, di->num_sms, slot);
    CUtensorMap tW, tX;
    constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (WK ? !tensor_map_2d(&tW, g.B, dt, 1, g.K, g.N, g.ldb, 128, Cfg::TN, SWZ_128)
           : !tensor_map_2d(&tW, g.B, dt, 1, g.N, g.K, g.ldb, 128, Cfg::BK, SWZ_128))
        return kCudaError;
    if (!tensor_map_2d(&tX, g.A, dt, 1, g.K, g.M, g.lda, 128, MPAD, SWZ_128)) return kCudaError;
    SkParams p = {};
    p.M = static_cast<int>(g.M);
    p.N = static_cast<int>(g.N);
    p.K = static_cast<int>(g.K);
    p.relu = g.relu;
    p.T = static_cast<int>(T);
    p.KB = static_cast<int>(KB);
    p.U = static_cast<int>(T * KB);
    p.J = 1;
    p.S = S;
    p.inject = inject_mode();
    p.timeout_ns = wait_limit_ns();
    p.status = device_status_ptr();
    p.C = g.C;
    p.ldc = g.ldc;
    p.row_scale = a.row_scale;
    p.col_scale = a.col_scale;
    p.out_bf16 = bf16;
    if (!p.status) return kCudaError;
    return skinny_launch<Cfg>(T * S, S, static_cast<cudaStream_t>(g.stream), tW, tW, tX, p) == cudaSuccess
               ? kOk : kCudaError;
}

template <int WK>
int dispatch(const GroupArgs& a, int bf16, int slot) {
    if (a.g.M <= 16) return run<16, WK>(a, bf16, slot);
    if (a.g.M <= 32) return run<32, WK>(a, bf16, slot + 1);
    if (a.g.M <= 64) return run<64, WK>(a, bf16, slot + 2);
    return run<128, WK>(a, bf16, slot + 3);
}

}  // namespace

// The dense 8-bit product.  With at most 128 rows it streams the weights, where
// their 128-column groups can be split over the SMs (at least two CTAs a
// group) or the rows are so few that the row side does not matter.  Measured
// (us by events, L2 flushed, an empty kernel reads 6; weight-streaming / CTA
// pairs): 8192 x 8192 weights 20.6 / 26.8 with 16 rows, 28.3 / 28.7 with 128;
// 1024 x 8192 12.6 / 26.8 and 18.7 / 28.3; unsplit 14336 x 4096 18.5 / 20.5
// with 16 rows but 22.7 / 20.5 with 64 and 30.6 / 20.8 with 128.
int launch_w8a8(const GroupArgs& a, int bf16) {
    const DeviceInfo* di = current_device(nullptr);
    if (!di) return kNoDevice;
    const bool splits = (a.g.N + 127) / 128 * 2 <= di->num_sms;
    if (a.g.M <= 16 || (a.g.M <= kSkinnyMaxM && splits))
        return a.trans_b ? dispatch<1>(a, bf16, 90) : dispatch<0>(a, bf16, 94);
    return launch_group_i8(a, bf16);
}

}  // namespace tg
