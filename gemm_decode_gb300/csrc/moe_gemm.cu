// moe_gemm.cu -- host side of the matrix product grouped by expert (moe_gemm_kernel.cuh):
// workspace, tensor maps, choice of the tile, launches.
#include <algorithm>

#include "moe_gemm_kernel.cuh"

namespace q4 {

unsigned int *gemm_status_word();

namespace {

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: prepared x, its scales, arrival counters, partial sums.
struct Layout {
    int64_t xscale, arrived, partial, total;
    int counters;
};

// Tile: rows of x per item.  One weight tile with 32 rows of x streams the weights with the
// most copies in flight; 256 weight rows by 128 rows of x read each row of x for twice as
// many products.
struct Tile {
    int rt, nt;
};
Tile tile_of(int64_t R, int E, bool bf16) {
    if (R <= 24 * static_cast<int64_t>(E)) return Tile{1, 32};
    return bf16 ? Tile{2, 128} : Tile{1, 64};
}

Layout layout_of(int64_t R, int64_t Tx, int64_t K, int E, bool bf16) {
    const Tile t = tile_of(R, E, bf16);
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

template <int PARTS, int RT, int NT>
int launch_tile(const CUtensorMap &codes, const MoeKernelArgs &g, cudaStream_t stream) {
    using S = MoeShape<PARTS, RT, NT>;
    auto kern = moe_gemm_kernel<PARTS, RT, NT>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(S::smem(kMaxExperts)));
        if (e != cudaSuccess) {
            cudaGetLastError();
            set_cuda_error(e);
            return Q4_ERR_CUDA;
        }
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return launch_overlappable(kern, dim3(static_cast<unsigned>(device_info().sms)), dim3(S::kThreads), S::smem(g.E),
                               stream, true, codes, g);
}

}  // namespace

int64_t moe_gemm_workspace_bytes(int64_t R, int64_t Tx, int64_t, int64_t K, int E, bool bf16) {
    return layout_of(R, Tx, K, E, bf16).total;
}

int launch_moe_gemm(const MoeGemmArgs &a, cudaStream_t stream) {
    const bool bf16 = a.bf16 != 0;
    const Tile t = tile_of(a.R, a.E, bf16);
    // items are counted in 32 bits, and so are units while the K of items is shared
    const int64_t most = (a.R / t.nt + std::min<int64_t>(a.R, a.E)) * ((a.N + 128 * t.rt - 1) / (128 * t.rt));
    if (most > 0x7fffffffLL || a.K > (1 << 26)) return Q4_ERR_UNSUPPORTED;
    const Layout l = layout_of(a.R, a.Tx, a.K, a.E, bf16);
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
    if (t.nt == 32)
        return bf16 ? launch_tile<1, 1, 32>(codes, g, stream) : launch_tile<2, 1, 32>(codes, g, stream);
    return bf16 ? launch_tile<1, 2, 128>(codes, g, stream) : launch_tile<2, 1, 64>(codes, g, stream);
}

}  // namespace q4
