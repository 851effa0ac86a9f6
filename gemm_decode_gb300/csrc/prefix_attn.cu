// prefix_attn.cu -- attention of single queries over a shared and an own segment of the paged
// cache.  One warp per query and query head walks the keys with a running maximum and sum.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "q4_decode.cuh"

namespace q4 {

namespace {

template <typename C>
__device__ __forceinline__ float widen(C v) {
    if constexpr (std::is_same<C, __half>::value) return __half2float(v);
    else return __bfloat162float(v);
}

}  // namespace

template <typename C, int D>
__global__ void __launch_bounds__(128) prefix_attn_simple_kernel(const q4_prefix_attn_t g) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t at = blockIdx.x * 4ll + (threadIdx.x >> 5);
    wait_prior_grid();
    if (at >= static_cast<int64_t>(g.S) * g.Hq) return;
    const int s = static_cast<int>(at / g.Hq), h = static_cast<int>(at - static_cast<int64_t>(s) * g.Hq);
    const int kvh = h / (g.Hq / g.cache.heads);
    float q[N], o[N];
    for (int i = 0; i < N; ++i) {
        q[i] = widen(static_cast<const C *>(g.q)[s * g.q_stride + h * D + i * 32 + lane]) * g.scale;
        o[i] = 0.0f;
    }
    float m = -__int_as_float(0x7f800000), l = 0.0f;
    auto walk = [&](const int *pages, int most, int64_t n) {
        const int64_t all = static_cast<int64_t>(most) * g.cache.page;
        n = n < 0 ? 0 : n > all ? all : n;
        for (int64_t j = 0; j < n; ++j) {
            const int64_t p = pages[j / g.cache.page];
            const bool have = p >= 0 && p < g.cache.pages;
            const int64_t row = (have ? p : 0) * g.cache.page_stride + kvh * g.cache.head_stride +
                                (j % g.cache.page) * g.cache.row_stride;
            float x = 0.0f;
            for (int i = 0; i < N; ++i)
                if (have) x = fmaf(q[i], widen(static_cast<const C *>(g.cache.k)[row + i * 32 + lane]), x);
            for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
            const float nm = fmaxf(m, x), f = expf(m - nm), e = expf(x - nm);
            m = nm;
            l = l * f + e;
            for (int i = 0; i < N; ++i)
                o[i] = fmaf(e, have ? widen(static_cast<const C *>(g.cache.v)[row + i * 32 + lane]) : 0.0f, o[i] * f);
        }
    };
    for (int e = 0, first = 0; e < g.groups; ++e) {
        const int a = g.group_offsets != nullptr ? max(first, min(max(g.group_offsets[e], 0), g.S)) : 0;
        const int b = g.group_offsets != nullptr ? max(a, min(max(g.group_offsets[e + 1], 0), g.S)) : g.S;
        first = b;
        if (s < a || s >= b) continue;
        int64_t n = g.shared_lens[e];
        if (g.limits != nullptr) n = min(n, static_cast<int64_t>(g.limits[s]));
        walk(g.shared_pages + static_cast<int64_t>(e) * g.max_shared_pages, g.max_shared_pages, n);
    }
    if (g.own_pages != nullptr)
        walk(g.own_pages + static_cast<int64_t>(s) * g.max_own_pages, g.max_own_pages, g.own_lens[s]);
    const float r = l != 0.0f ? 1.0f / l : 0.0f;   // (no key: 0; NaN stays)
    for (int i = 0; i < N; ++i) {
        const int64_t to = at * D + i * 32 + lane;
        const float v = l != 0.0f ? o[i] * r : 0.0f;
        if (g.out_dtype == Q4_F32) static_cast<float *>(g.out)[to] = v;
        else if constexpr (std::is_same<C, __half>::value) static_cast<__half *>(g.out)[to] = __float2half_rn(v);
        else static_cast<__nv_bfloat16 *>(g.out)[to] = __float2bfloat16_rn(v);
    }
    if (g.lse != nullptr && lane == 0) g.lse[at] = l != 0.0f ? m + logf(l) : -__int_as_float(0x7f800000);
}

int64_t prefix_attn_workspace_bytes(int, int, int, int, int) { return 256; }

template <typename C>
static int launch_simple(const q4_prefix_attn_t &a, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(a.S) * a.Hq;
    const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
    const bool overlap = call_options().overlap;
    return a.cache.D == 64
               ? launch_overlappable(prefix_attn_simple_kernel<C, 64>, grid, dim3(128), 0, stream, overlap, a)
               : launch_overlappable(prefix_attn_simple_kernel<C, 128>, grid, dim3(128), 0, stream, overlap, a);
}

int launch_prefix_attn(const q4_prefix_attn_t &a, cudaStream_t stream) {
    return a.cache.dtype == Q4_F16 ? launch_simple<__half>(a, stream) : launch_simple<__nv_bfloat16>(a, stream);
}

}  // namespace q4
