// moe_gemm.cu -- host side of the matrix product grouped by expert: workspace, tensor map,
// choice of the kernel (moe_gemm_few.cuh, moe_gemm_many.cuh) and its tile, launches.
#include <algorithm>

#include "moe_gemm_few.cuh"
#include "moe_gemm_many.cuh"

namespace q4 {

unsigned int *gemm_status_word();

namespace {

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: prepared x, its scales, arrival counters, partial sums.
struct Layout {
    int64_t xscale, arrived, partial, total;
    int counters;
};

// Tile: weight tiles and rows of x per item.
//   bfloat16: up to 24 rows per expert on average, 32 rows of the kernel for few rows; above,
//   the kernel for many.
//   binary32: always the kernel for few rows, whose sums per group of weights leave room for
//   16, 32 or 64 rows with groups of 32, 64 or 128; no more than the average expert fills.
struct Tile {
    int rt, nt;
};
Tile tile_of(int64_t R, int E, int group, bool bf16) {
    if (bf16) return R <= 24 * static_cast<int64_t>(E) ? Tile{1, 32} : Tile{2, 128};
    if (group == 32 || R <= 8 * static_cast<int64_t>(E)) return Tile{1, 16};
    return group == 64 || R <= 24 * static_cast<int64_t>(E) ? Tile{1, 32} : Tile{1, 64};
}

Layout layout_of(int64_t R, int64_t Tx, int64_t K, const Tile &t, bool bf16) {
    const int64_t ctas = device_info().sms;
    Layout l;
    l.counters = static_cast<int>(ctas) * t.rt;
    l.xscale = round256((Tx + 1) * K * (bf16 ? 2 : 4));
    l.arrived = l.xscale + round256(4 * (Tx + 1));
    l.partial = l.arrived + round256(4 * ctas * t.rt);
    l.total = l.partial + 2 * ctas * 4 * t.rt * 128 * t.nt;
    return l;
}

bool encode_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner, int64_t rows,
               int64_t stride, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
    const cuuint32_t box[2] = {box_inner, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One CTA per SM, overlapped with the kernel that prepares x.
int launch_product(void (*kern)(CUtensorMap, MoeKernelArgs), int threads, size_t smem, size_t most,
                   std::atomic<bool> *configured, const CUtensorMap &codes, const MoeKernelArgs &g,
                   cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(most));
        if (e != cudaSuccess) {
            cudaGetLastError();
            set_cuda_error(e);
            return Q4_ERR_CUDA;
        }
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return launch_overlappable(kern, dim3(static_cast<unsigned>(device_info().sms)),
                               dim3(static_cast<unsigned>(threads)), smem, stream, true, codes, g);
}
template <int PARTS, int NT>
int launch_few(const CUtensorMap &codes, const MoeKernelArgs &g, cudaStream_t stream) {
    using S = FewShape<PARTS, NT>;
    static std::atomic<bool> configured[64];
    return launch_product(moe_gemm_few_kernel<PARTS, NT>, S::kThreads, S::smem(g.E), S::smem(kMaxExperts), configured,
                          codes, g, stream);
}
int launch_many(const CUtensorMap &codes, const MoeKernelArgs &g, cudaStream_t stream) {
    using S = ManyShape;
    static std::atomic<bool> configured[64];
    return launch_product(moe_gemm_many_kernel, S::kThreads, S::smem(g.E), S::smem(kMaxExperts), configured, codes, g,
                          stream);
}

}  // namespace

// Items are counted in 32 bits (and so are units while the K of items is shared).
bool moe_gemm_countable(int64_t R, int E, int64_t N, int group, bool bf16) {
    const Tile t = tile_of(R, E, group, bf16);
    return R / t.nt + std::min<int64_t>(R, E) <= 0x7fffffffLL / ((N + 128 * t.rt - 1) / (128 * t.rt) + 1);
}

int64_t moe_gemm_workspace_bytes(int64_t R, int64_t Tx, int64_t, int64_t K, int E, bool bf16) {
    int64_t most = 0;   // whatever the group
    for (int group : {32, 64, 128})
        most = std::max(most, layout_of(R, Tx, K, tile_of(R, E, group, bf16), bf16).total);
    return most;
}

int launch_moe_gemm(const MoeGemmArgs &a, cudaStream_t stream) {
    const bool bf16 = a.bf16 != 0;
    const Tile t = tile_of(a.R, a.E, a.group, bf16);
    const Layout l = layout_of(a.R, a.Tx, a.K, t, bf16);
    unsigned char *w = static_cast<unsigned char *>(a.workspace);
    MoeKernelArgs g;
    g.scales = a.scales;
    g.zeros = a.zeros;
    g.rows = a.rows;
    g.offsets = a.offsets;
    g.xscale = reinterpret_cast<float *>(w + l.xscale);
    g.y = a.y;
    g.partial = reinterpret_cast<float *>(w + l.partial);
    g.arrived = reinterpret_cast<unsigned int *>(w + l.arrived);
    g.E = a.E;
    g.R = a.R;
    g.Tx = a.Tx;
    g.N = a.N;
    g.K = a.K;
    g.nb = a.K / a.group;
    g.zrow = (g.nb + 1) / 2;
    g.gshift = a.group == 32 ? 5 : (a.group == 64 ? 6 : 7);
    g.swiglu = a.swiglu;
    g.wide_scales = g.nb % 8 == 0 && aligned(a.scales, 16);
    g.wide_zeros = g.zrow % 8 == 0 && aligned(a.zeros, 8);
    g.copy_scales = g.nb % 4 == 0 && aligned(a.scales, 8) && (a.zeros == nullptr || g.wide_zeros);
    g.timeout_ns = call_options().wait_ns;
    g.status = gemm_status_word();
    g.bounds = bounds_counter();
    if (g.status == nullptr) return Q4_ERR_CUDA;
    CUtensorMap codes;
    if (!encode_2d(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.K / 2, static_cast<int64_t>(a.E) * a.N, a.K / 2,
                   kUnit / 2, 128, CU_TENSOR_MAP_SWIZZLE_64B))
        return Q4_ERR_UNSUPPORTED;
    __half *xp = reinterpret_cast<__half *>(w);
    g.xparts = xp;
    float *xscale = reinterpret_cast<float *>(w + l.xscale);
    const dim3 grid(static_cast<unsigned>(a.Tx + 1));
    const bool overlap = call_options().overlap;
    int st = bf16 ? launch_overlappable(moe_prepare_kernel<true>, grid, dim3(256), 0, stream, overlap, a.x, a.Tx, a.K,
                                        xp, xscale, g.arrived, l.counters)
                  : launch_overlappable(moe_prepare_kernel<false>, grid, dim3(256), 0, stream, overlap, a.x, a.Tx, a.K,
                                        xp, xscale, g.arrived, l.counters);
    if (st != Q4_OK) return st;
    if (bf16) return t.rt == 1 ? launch_few<1, 32>(codes, g, stream) : launch_many(codes, g, stream);
    if (t.nt == 16) return launch_few<2, 16>(codes, g, stream);
    return t.nt == 32 ? launch_few<2, 32>(codes, g, stream) : launch_few<2, 64>(codes, g, stream);
}

}  // namespace q4
