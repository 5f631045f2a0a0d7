// gemm_skinny_mx4.cu -- launcher of the weight-streaming kernel for microscaled
// 4-bit weights and activations with at most 128 rows.
#include "gemm_skinny.cuh"
#include "host.cuh"
#include "launch.h"

namespace tg {

namespace {

template <int MPAD>
int run(const GroupArgs& a, int bf16, int slot) {
    using Cfg = SkCfg<WKind::MX4, MPAD, 1>;
    const DeviceInfo* di = current_device(nullptr);
    if (!di) return kNoDevice;
    const GemmArgs& g = a.g;
    const long long T = (g.N + Cfg::GN - 1) / Cfg::GN, KB = (g.K + Cfg::BK - 1) / Cfg::BK;
    if (T * KB > 0x7fffffffll) return kUnsupported;
    auto kern = skinny_kernel<Cfg>;
    if (set_smem_attr(reinterpret_cast<const void*>(kern), Cfg::SMEM_BYTES, slot) != cudaSuccess) return kCudaError;
    const int S = skinny_whole_split<Cfg>(T, KB, di->num_sms, slot);
    CUtensorMap tW, tX, tS, tSX;
    constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!tensor_map_2d(&tW, g.B, dt, 1, g.K, g.N, g.ldb, 128, Cfg::TN, SWZ_128) ||
        !tensor_map_2d(&tX, g.A, dt, 1, g.K, g.M, g.lda, 128, MPAD, SWZ_128) ||
        !tensor_map_2d(&tS, a.col_blocks, dt, 1, a.blocks, g.N, a.block_ldb, 16, Cfg::TN, SWZ_NONE) ||
        !tensor_map_2d(&tSX, a.row_blocks, dt, 1, a.blocks, g.M, a.block_lda, 16, MPAD, SWZ_NONE))
        return kCudaError;
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
    p.out_bf16 = bf16;
    if (!p.status) return kCudaError;
    return skinny_launch<Cfg>(T * S, S, static_cast<cudaStream_t>(g.stream), tW, tS, tX, tSX, p) == cudaSuccess
               ? kOk : kCudaError;
}

}  // namespace

// The dense 4-bit product: the choice of the 8-bit one (launch_w8a8).  This kernel
// against that on CTA pairs, us in a graph: K = 8192, N = 8192, 1 row 12.0 / 16.8, 17
// 12.4 / 16.9, 64 14.1 / 16.7, 128 17.3 / 17.5; N = 14336, 16 rows 15.8 / 19.2, 17 16.1 /
// 19.3, 64 18.5 / 19.3, 128 22.9 / 20.4; K = 2048, N = 8192, 17 rows 7.8 / 9.4, 64 9.4
// both, 128 12.0 / 10.1.  (So of 17 to 64 rows with more than 9472 columns the slower
// one is taken, and of 65 to 128 with few k.)
int launch_mx4(const GroupArgs& a, int bf16) {
    const DeviceInfo* di = current_device(nullptr);
    if (!di) return kNoDevice;
    const bool splits = (a.g.N + 127) / 128 * 2 <= di->num_sms;
    if (a.g.M > 16 && !(a.g.M <= kSkinnyMaxM && splits)) return launch_group_mx4(a, bf16);
    if (a.g.M <= 16) return run<16>(a, bf16, 100);
    if (a.g.M <= 32) return run<32>(a, bf16, 101);
    if (a.g.M <= 64) return run<64>(a, bf16, 102);
    return run<128>(a, bf16, 103);
}

}  // namespace tg
