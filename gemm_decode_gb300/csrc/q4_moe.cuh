// q4_moe.cuh -- launchers of the mixture-of-experts kernels (internal, not part of the
// public ABI).
#pragma once

#include "q4_common.cuh"

namespace q4 {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxNormH = 16384;
constexpr int64_t kMaxMoeK = 1 << 26;   // units of 128 k are counted in 32 bits

struct RouteArgs {
    const float *logits, *bias;
    const uint8_t *mask;
    int T, E, k;
    int sigmoid, renorm, score_bias;   // score_bias: the bias is added to the score, not to the logit
    float scale;
    int *ids;
    float *weights;
    int *offsets, *rows, *pos;
    int *hist;   // [blocks][E] choices of each block of tokens (several blocks only), [E] totals (many)
    unsigned int *bounds;   // counter of bounds-checking builds
};
int64_t route_workspace_bytes(int T, int E, int k);
int launch_route(const RouteArgs &a, cudaStream_t stream);

struct MoeGemmArgs {
    const uint8_t *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
    const void *x;
    const int *rows, *offsets;
    void *y;
    int E;
    int R, Tx;
    int N, K, group;
    int bf16, swiglu;
    void *workspace;
};
bool moe_gemm_countable(int64_t R, int E, int64_t N, int group, bool bf16);
int64_t moe_gemm_workspace_bytes(int64_t R, int64_t Tx, int64_t N, int64_t K, int E, bool bf16);
int launch_moe_gemm(const MoeGemmArgs &a, cudaStream_t stream);

int launch_block_norm(const q4_block_norm_t &a, cudaStream_t stream);

// cudaLaunchKernelEx with the call's overlapped-launch attribute when asked for.
template <typename... P, typename... A>
int launch_overlappable(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool overlap,
                        A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (overlap) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error(e);
        return Q4_ERR_CUDA;
    }
    return Q4_OK;
}

}  // namespace q4
