// block_norm.cu -- what follows a block's output, in one pass: the weighted sum of a
// token's expert rows, the norm after the block, its gate, the scaled residual, and the
// norm before the next block.
//
//   b = sum_j w_j y[pos_j];  p = b / sqrt(mean b^2 + eps) * post;  x' = alpha x + gate p;
//   a = x' / sqrt(mean x'^2 + eps) * pre
//
// One CTA per token; each thread keeps its NI vectors of the row in registers from the
// first load to the last store (beyond 8192 features, 4096 with accesses of two elements or
// 2048 of one, part of them is spilled), so every array is read or written once and the two means
// are block sums of registers (binary32, in a fixed order: warps by shuffles, then the
// warps' sums by every thread).  Loads are up to 16 bytes per thread, four of
// the token's rows of y at a time in flight together, and those of x and the gate before
// them, so that no load waits for a sum; rows whose length is no multiple of 16 bytes, or
// whose gate or norm weights are unaligned, take accesses of 8, 4 or 2 bytes.
//
// Bound: the bytes of the rows of y, x and the outputs for prompts (4.4 TB/s, 0.65 of
// measured, at the size below); latency for decoding (4.1 us for one token).
#include <cuda_bf16.h>

#include "q4_moe.cuh"

namespace q4 {

namespace {

// Threads of a CTA at most; two CTAs per SM at least (64 registers a thread).  4096 tokens of
// 4096 features, eight rows each (376 MB): 512 threads of one vector 86 us (4.4 TB/s), 256
// threads of two 99 us, 128 of four 131 us; four CTAs of 512 threads 83 us, but 1 us more for
// one token.
constexpr int kNormThreads = 512;

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

// V consecutive elements in one access of up to 16 bytes.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
// V consecutive norm weights (aligned to the smaller of 4 V and 16 bytes).
template <int V>
__device__ __forceinline__ void load_floats(const float *p, float *out) {
    if constexpr (V == 1) {
        out[0] = *p;
    } else if constexpr (V == 2) {
        const float2 a = *reinterpret_cast<const float2 *>(p);
        out[0] = a.x, out[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + i);
            out[i] = a.x, out[i + 1] = a.y, out[i + 2] = a.z, out[i + 3] = a.w;
        }
    }
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
__global__ void __launch_bounds__(kNormThreads, 2) block_norm_kernel(const q4_block_norm_t g, unsigned int *bounds) {
    __shared__ float sums[64];
    __shared__ float w_s[kMaxTopK];
    __shared__ int pos_s[kMaxTopK];
    const int t = blockIdx.x;
    const int H = g.H;
    // (bounds-checking builds) columns [c, c + V) of row r of an array of `rows` rows, aligned as accessed
    auto ib = [&](int64_t r, int64_t rows, int c, const void *p) {
        return q4_in_bounds(r >= 0 && r < rows && c + V <= H && reinterpret_cast<uintptr_t>(p) % (V * sizeof(T)) == 0,
                            bounds);
    };
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
    // the residual and the gate are on their way while the rows of y are summed
    Pack<T, V> xv[NI], gv[NI];
    float b[NI][V];
    const T *gate = g.gate != nullptr ? static_cast<const T *>(g.gate) + static_cast<int64_t>(t) * g.gate_stride : nullptr;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < H && ib(t, g.T, c, x + c)) {
            xv[i] = load_pack<T, V>(x + c);
            if (gate != nullptr && ib(t, g.T, c, gate + c)) gv[i] = load_pack<T, V>(gate + c);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) b[i][v] = 0.0f;
    }
    if (g.top_k > 0) {
        __syncthreads();
        for (int j0 = 0; j0 < g.top_k; j0 += 4) {
            const T *row[4];
            float w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int p = j0 + q < g.top_k ? pos_s[j0 + q] : -1;
                row[q] = p >= 0 ? y + static_cast<int64_t>(p) * H : nullptr;
                w[q] = p >= 0 ? w_s[j0 + q] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int c = (i * blockDim.x + threadIdx.x) * V;
                if (c < H) {
                    Pack<T, V> in[4] = {};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (row[q] != nullptr && ib(pos_s[j0 + q], g.R, c, row[q] + c)) in[q] = load_pack<T, V>(row[q] + c);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int v = 0; v < V; ++v) b[i][v] = fmaf(w[q], to_float(in[q].v[v]), b[i][v]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < H && ib(t, g.R, c, y + static_cast<int64_t>(t) * H + c)) {
                const Pack<T, V> in = load_pack<T, V>(y + static_cast<int64_t>(t) * H + c);
#pragma unroll
                for (int v = 0; v < V; ++v) b[i][v] = to_float(in.v[v]);
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
                float w[V];
                load_floats<V>(g.post_gamma + c, w);
#pragma unroll
                for (int v = 0; v < V; ++v) b[i][v] = b[i][v] * r * w[v];
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < H) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (gate != nullptr) b[i][v] *= to_float(gv[i].v[v]);
                b[i][v] = fmaf(g.residual_scale, to_float(xv[i].v[v]), b[i][v]);
                ss = fmaf(b[i][v], b[i][v], ss);
            }
            T *to = static_cast<T *>(g.out) + static_cast<int64_t>(t) * H + c;
            if (ib(t, g.T, c, to)) store_pack<T, V>(to, b[i]);
        }
    }
    if (g.pre_gamma == nullptr) return;
    const float r = 1.0f / sqrtf(block_sum(ss, sums + 32) / static_cast<float>(H) + g.eps);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < H) {
            float w[V];
            load_floats<V>(g.pre_gamma + c, w);
#pragma unroll
            for (int v = 0; v < V; ++v) b[i][v] = b[i][v] * r * w[v];
            T *to = static_cast<T *>(g.out_norm) + static_cast<int64_t>(t) * H + c;
            if (ib(t, g.T, c, to)) store_pack<T, V>(to, b[i]);
        }
    }
}

template <typename T, int V>
static int launch_norm(const q4_block_norm_t &a, cudaStream_t stream) {
    const bool overlap = call_options().overlap;
    const int vecs = a.H / V;
    auto launch = [&](auto kernel, int ni) {
        const unsigned threads = static_cast<unsigned>(((vecs + ni - 1) / ni + 31) / 32 * 32);
        return launch_overlappable(kernel, dim3(static_cast<unsigned>(a.T)), dim3(threads), 0, stream, overlap, a,
                                   bounds_counter());
    };
    // vectors per thread; H is at most kMaxNormH
    constexpr int kMost = kMaxNormH / V / kNormThreads;
    if (vecs <= kNormThreads) return launch(block_norm_kernel<T, V, 1>, 1);
    if (vecs <= 2 * kNormThreads) return launch(block_norm_kernel<T, V, 2>, 2);
    if constexpr (kMost > 4)
        if (vecs <= 4 * kNormThreads) return launch(block_norm_kernel<T, V, 4>, 4);
    return launch(block_norm_kernel<T, V, kMost>, kMost);
}

// The widest access that the row's length and the alignment of the gate and of the norm
// weights allow.
template <typename T>
static int launch_norm_of(const q4_block_norm_t &a, cudaStream_t stream) {
    auto fits = [&](int v) {
        const uintptr_t w = v >= 4 ? 16 : 4 * v;
        return a.H % v == 0 && aligned(a.gate, v * sizeof(T)) && aligned(a.post_gamma, w) && aligned(a.pre_gamma, w);
    };
    if constexpr (sizeof(T) == 2)
        if (fits(8)) return launch_norm<T, 8>(a, stream);
    if (fits(4)) return launch_norm<T, 4>(a, stream);
    return fits(2) ? launch_norm<T, 2>(a, stream) : launch_norm<T, 1>(a, stream);
}

int launch_block_norm(const q4_block_norm_t &a, cudaStream_t stream) {
    return a.dtype == Q4_F32 ? launch_norm_of<float>(a, stream) : launch_norm_of<__nv_bfloat16>(a, stream);
}

}  // namespace q4
