// gemm_group.cu -- launchers of the products over groups of rows: 16-bit
// experts' products and their weight gradient, 8-bit experts' products and
// the dense 8-bit product.
#include "gemm_group.cuh"
#include "host.cuh"
#include "launch.h"

namespace tg {

namespace {

GrpParams params(const GroupArgs& a) {
    GrpParams p = {};
    p.M = static_cast<int>(a.g.M);
    p.N = static_cast<int>(a.g.N);
    p.K = static_cast<int>(a.g.K);
    p.E = a.E;
    p.offsets = a.offsets;
    p.relu = a.g.relu;
    p.inject = inject_mode();
    p.group_m = 8;
    p.timeout_ns = wait_limit_ns();
    p.status = device_status_ptr();
    p.C = a.g.C;
    p.ldc = a.g.ldc;
    p.plane = a.plane;
    p.row_scale = a.row_scale;
    p.col_scale = a.col_scale;
    p.scale_plane = a.scale_plane;
    p.row_blocks = a.row_blocks;
    p.col_blocks = a.col_blocks;
    p.block_lda = a.block_lda;
    p.block_ldb = a.block_ldb;
    p.block_plane = a.block_plane;
    p.blocks = static_cast<int>(a.blocks);
    return p;
}

// At most one item per 256 rows and one more per group with rows (the rows
// behind the last group included), times the 256-column tiles.
long long max_items(const GroupArgs& a) {
    const long long groups = a.offsets ? (a.E + 1 < a.g.M ? a.E + 1 : a.g.M) : 1;
    return (a.g.M / 256 + groups) * ((a.g.N - 1) / 256 + 1);
}

template <class Cfg>
int launch(const GroupArgs& a, long long items, int tiles, const CUtensorMap& tA, const CUtensorMap (&tB)[4],
           const CUtensorMap& tC, int num_sms) {
    GrpParams p = params(a);
    p.tiles = tiles;
    if (!p.status) return kCudaError;
    // a tile of a thin wave runs as up to four pieces (WG: two)
    const long long npairs = persistent_grid(items * (Cfg::WG ? 2 : 4), num_sms / 2, 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * npairs), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = static_cast<cudaStream_t>(a.g.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, grp_gemm_kernel<Cfg>, tA, tB[0], tB[1], tB[2], tB[3], tC, p);
    if (e != cudaSuccess) {
        cudaGetLastError();                       // clear
        return kUnsupported;
    }
    return kOk;
}

template <class Cfg>
int run_product(const GroupArgs& a, CUtensorMapDataType dt, int slot) {
    if (pair_kernels_disabled()) return kUnsupported;
    const DeviceInfo* di = current_device(nullptr);
    if (!di) return kNoDevice;
    long long items = max_items(a);
    int tiles = 0;
    if (Cfg::MX && !a.offsets) {
        const long long ntl = (a.g.N - 1) / 256 + 1;
        tiles = mx4_even_tiles(a.g.M, ntl, di->num_sms / 2);
        items = tiles * ntl;
    }
    if (items > 0x7fffffffll) return kUnsupported;
    constexpr int eb = Cfg::EB;
    const GemmArgs& g = a.g;
    const uint64_t plane = static_cast<uint64_t>(a.E > 1 ? a.plane_b : g.ldb) * eb;   // one group: any legal stride
    CUtensorMap tA, tB[4];
    // weights: K x N -> boxes of 128 bytes of columns x BK rows; N x K ->
    // boxes of BK x 128 columns
    if (Cfg::W_MN ? !tensor_map_3d(&tA, g.B, dt, g.N, g.K, g.ldb * eb, a.E, plane, Cfg::CHUNK, Cfg::BK, SWZ_128)
                  : !tensor_map_3d(&tA, g.B, dt, g.K, g.N, g.ldb * eb, a.E, plane, Cfg::BK, 128, SWZ_128))
        return kCudaError;
    for (int i = 0; i < 4; ++i)
        if (!tensor_map_2d(&tB[i], g.A, dt, eb, g.K, g.M, g.lda * eb, Cfg::BK, 128 >> i, SWZ_128))
            return kCudaError;
    if (set_smem_attr(reinterpret_cast<const void*>(grp_gemm_kernel<Cfg>), Cfg::SMEM_BYTES, slot) != cudaSuccess)
        return kCudaError;
    return launch<Cfg>(a, items, tiles, tA, tB, tA, di->num_sms);
}

template <class Cfg>
int run_grad(const GroupArgs& a, CUtensorMapDataType dt, int slot) {
    if (pair_kernels_disabled()) return kUnsupported;
    const DeviceInfo* di = current_device(nullptr);
    if (!di) return kNoDevice;
    const GemmArgs& g = a.g;
    const long long per = ((g.K - 1) / 256 + 1) * ((g.N - 1) / 256 + 1);
    if (per > 0x7fffffffll / a.E) return kUnsupported;
    CUtensorMap tA, tB[4], tC;
    if (!tensor_map_2d(&tA, g.A, dt, 2, g.K, g.M, g.lda * 2, 64, 64, SWZ_128) ||
        !tensor_map_2d(&tB[0], g.B, dt, 2, g.N, g.M, g.ldb * 2, 64, 64, SWZ_128) ||
        !tensor_map_3d(&tC, g.C, dt, g.N, g.K, g.ldc * 2, a.E,
                       static_cast<uint64_t>(a.E > 1 ? a.plane : g.ldc) * 2, 64, 32, SWZ_128))
        return kCudaError;
    tB[1] = tB[2] = tB[3] = tB[0];
    if (set_smem_attr(reinterpret_cast<const void*>(grp_gemm_kernel<Cfg>), Cfg::SMEM_BYTES, slot) != cudaSuccess)
        return kCudaError;
    return launch<Cfg>(a, per * a.E, 0, tA, tB, tC, di->num_sms);
}

}  // namespace

int launch_group(const GroupArgs& a, int bf16) {
    constexpr CUtensorMapDataType tb = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, th = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (bf16)
        return a.trans_b ? run_product<GrpCfg<1, OutT::BF16, 0>>(a, tb, 70) : run_product<GrpCfg<1, OutT::BF16, 1>>(a, tb, 71);
    return a.trans_b ? run_product<GrpCfg<0, OutT::F16, 0>>(a, th, 72) : run_product<GrpCfg<0, OutT::F16, 1>>(a, th, 73);
}

// Eight epilogue warps where groups have few rows and writing their gradients
// takes longer than their MMAs, else four with two staging tiles each.  Measured
// (us, four / eight) on 32 groups of 4096 x 2048 with 64 rows 116 / 114, 100 rows
// 122 / 109, 128 rows 121 / 111, 200 rows 143 / 147, 256 rows 133 / 135, 384 rows
// 163 / 168, 1000 rows 374 / 379.
int launch_group_grad(const GroupArgs& a, int bf16) {
    constexpr CUtensorMapDataType tb = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, th = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (a.g.M < 256ll * a.E)
        return bf16 ? run_grad<GrpCfg<1, OutT::BF16, 1, 1, 8>>(a, tb, 74) : run_grad<GrpCfg<0, OutT::F16, 1, 1, 8>>(a, th, 75);
    return bf16 ? run_grad<GrpCfg<1, OutT::BF16, 1, 1, 4>>(a, tb, 80) : run_grad<GrpCfg<0, OutT::F16, 1, 1, 4>>(a, th, 81);
}

int launch_group_mx4(const GroupArgs& a, int bf16) {
    constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return bf16 ? run_product<GrpCfg<4, OutT::BF16, 0>>(a, dt, 98) : run_product<GrpCfg<4, OutT::F16, 0>>(a, dt, 99);
}

int launch_group_i8(const GroupArgs& a, int bf16) {
    constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (bf16)
        return a.trans_b ? run_product<GrpCfg<3, OutT::BF16, 0>>(a, dt, 76) : run_product<GrpCfg<3, OutT::BF16, 1>>(a, dt, 77);
    return a.trans_b ? run_product<GrpCfg<3, OutT::F16, 0>>(a, dt, 78) : run_product<GrpCfg<3, OutT::F16, 1>>(a, dt, 79);
}

}  // namespace tg
