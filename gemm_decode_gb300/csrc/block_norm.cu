// block_norm.cu -- what follows a block's output, in one pass: the weighted sum of a
// token's expert rows, the norm after the block, its gate, the scaled residual, and the
// norm before the next block.
//
//   b = sum_j w_j y[pos_j];  p = b / sqrt(mean b^2 + eps) * post;  x' = alpha x + gate p;
//   a = x' / sqrt(mean x'^2 + eps) * pre
//
// One CTA per token; each thread keeps its NI vectors of the row in registers from the
// first load to the last store, so every array is read or written once and the two means
// are block sums of registers (binary32, in a fixed order: warps by shuffles, then the
// warps' sums by every thread).  Loads are 16 bytes per thread (8 bf16 or 4 floats); rows
// whose length is no multiple of that, or whose gate is unaligned, take single elements.
//
// Bound: the bytes of the rows of y, x and the outputs for prompts; latency for decoding.
#include <cuda_bf16.h>

#include "q4_moe.cuh"

namespace q4 {

namespace {

template <typename T>
__device__ __forceinline__ float to_float(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
    else return v;
}

// V consecutive elements in one access (V * sizeof(T) is 16 bytes, or V is 1).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_pack(const T *p, float *out) {
    const Pack<T, V> a = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = to_float(a.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const float *in) {
    Pack<T, V> a;
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] = from_float<T>(in[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = a;
}

__device__ __forceinline__ float block_sum(float v, float *warp_sums) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += warp_sums[w];
    return s;
}

}  // namespace

template <typename T, int V, int NI>
__global__ void __launch_bounds__(1024) block_norm_kernel(const q4_block_norm_t g) {
    __shared__ float sums[64];
    __shared__ float w_s[kMaxTopK];
    __shared__ int pos_s[kMaxTopK];
    const int t = blockIdx.x;
    const int H = g.H;
    const T *y = static_cast<const T *>(g.y);
    const T *x = static_cast<const T *>(g.x) + static_cast<int64_t>(t) * H;
    wait_prior_grid();
    allow_next_grid();
    if (threadIdx.x < g.top_k) {
        const int64_t at = static_cast<int64_t>(t) * g.top_k + threadIdx.x;
        const int p = g.pos[at];
        pos_s[threadIdx.x] = p >= 0 && p < g.R ? p : -1;
        w_s[threadIdx.x] = g.weights[at];
    }
    float b[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) b[i][v] = 0.0f;
    if (g.top_k > 0) __syncthreads();
    for (int j = 0; j < (g.top_k > 0 ? g.top_k : 1); ++j) {
        const int64_t row = g.top_k > 0 ? pos_s[j] : t;
        if (row < 0) continue;
        const float w = g.top_k > 0 ? w_s[j] : 1.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < H) {
                float in[V];
                load_pack<T, V>(y + row * H + c, in);
#pragma unroll
                for (int v = 0; v < V; ++v) b[i][v] = fmaf(w, in[v], b[i][v]);
            }
        }
    }
    if (g.post_gamma != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(b[i][v], b[i][v], ss);
        const float r = 1.0f / sqrtf(block_sum(ss, sums) / static_cast<float>(H) + g.eps);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < H) {
#pragma unroll
                for (int v = 0; v < V; ++v) b[i][v] = b[i][v] * r * g.post_gamma[c + v];
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < H) {
            float in[V];
            if (g.gate != nullptr) {
                load_pack<T, V>(static_cast<const T *>(g.gate) + static_cast<int64_t>(t) * g.gate_stride + c, in);
#pragma unroll
                for (int v = 0; v < V; ++v) b[i][v] *= in[v];
            }
            load_pack<T, V>(x + c, in);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                b[i][v] = fmaf(g.residual_scale, in[v], b[i][v]);
                ss = fmaf(b[i][v], b[i][v], ss);
            }
            store_pack<T, V>(static_cast<T *>(g.out) + static_cast<int64_t>(t) * H + c, b[i]);
        }
    }
    if (g.pre_gamma == nullptr) return;
    const float r = 1.0f / sqrtf(block_sum(ss, sums + 32) / static_cast<float>(H) + g.eps);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < H) {
#pragma unroll
            for (int v = 0; v < V; ++v) b[i][v] = b[i][v] * r * g.pre_gamma[c + v];
            store_pack<T, V>(static_cast<T *>(g.out_norm) + static_cast<int64_t>(t) * H + c, b[i]);
        }
    }
}

template <typename T, int V>
static int launch_norm(const q4_block_norm_t &a, cudaStream_t stream) {
    const bool overlap = call_options().overlap;
    const int vecs = (a.H + V - 1) / V;
    auto threads = [&](int ni) { return dim3(static_cast<unsigned>((((vecs + ni - 1) / ni) + 31) / 32 * 32)); };
    const dim3 grid(static_cast<unsigned>(a.T));
    if (vecs <= 1024) return launch_overlappable(block_norm_kernel<T, V, 1>, grid, threads(1), 0, stream, overlap, a);
    if (vecs <= 4096) return launch_overlappable(block_norm_kernel<T, V, 4>, grid, threads(4), 0, stream, overlap, a);
    return launch_overlappable(block_norm_kernel<T, V, 16>, grid, threads(16), 0, stream, overlap, a);
}

int launch_block_norm(const q4_block_norm_t &a, cudaStream_t stream) {
    if (a.dtype == Q4_F32)
        return a.H % 4 == 0 && aligned(a.gate, 16) ? launch_norm<float, 4>(a, stream)
                                                   : launch_norm<float, 1>(a, stream);
    return a.H % 8 == 0 && aligned(a.gate, 16) ? launch_norm<__nv_bfloat16, 8>(a, stream)
                                               : launch_norm<__nv_bfloat16, 1>(a, stream);
}

}  // namespace q4
