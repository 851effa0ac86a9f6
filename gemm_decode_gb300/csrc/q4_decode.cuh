// q4_decode.cuh -- launchers of the kernels for several continuations of one prompt
// (internal, not part of the public ABI).
#pragma once

#include <atomic>

#include "q4_moe.cuh"

namespace q4 {

constexpr int kMaxHeadD = 256;      // rotary call
constexpr int kMaxBeams = 32;       // beams of a group, and continuations chosen
constexpr int kMaxReorderW = 1024;
constexpr int kMaxQueries = 1 << 20;
constexpr int kMaxShare = 128;      // query heads of a kv head

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The dynamic shared memory that a kernel may be launched with, set once per device.
template <typename... P>
int allow_smem(void (*kernel)(P...), size_t bytes, std::atomic<bool> *configured) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && configured[dev]) return Q4_OK;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error(e);
        return Q4_ERR_CUDA;
    }
    if (dev >= 0 && dev < 64) configured[dev] = true;
    return Q4_OK;
}

int launch_rope_append(const q4_rope_append_t &a, cudaStream_t stream);

int64_t prefix_attn_workspace_bytes(int S, int groups, int Hq, int Hkv, int D);
int launch_prefix_attn(const q4_prefix_attn_t &a, cudaStream_t stream);

struct BeamArgs {
    const float *logits;
    int64_t row_stride;
    const float *scores;
    const uint8_t *finished;
    int groups, W, K;
    int64_t V;
    int eos;
    int *tokens, *parents;
    float *out_scores;
    uint8_t *out_finished;
    void *workspace;
    unsigned int *bounds;   // counter of bounds-checking builds
};
int64_t beam_workspace_bytes(int groups, int W, int K, int64_t V);
int launch_beam_step(const BeamArgs &a, cudaStream_t stream);

int launch_beam_reorder(const q4_beam_reorder_t &a, cudaStream_t stream);

}  // namespace q4
