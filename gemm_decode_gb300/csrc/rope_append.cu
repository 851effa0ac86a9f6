// rope_append.cu -- norm of each head, rotary positions, and the new tokens' keys and values
// into the paged cache, in one pass over the rows that a q/k/v product leaves.
//
//   u = x / sqrt(mean x^2 + eps) * gamma;   (u_a, u_b) -> (c u_a - s u_b, s u_a + c u_b)
//
// The angle of a pair is positions[t] * inv_freq[i].  In binary32 that product is off by
// 2^-24 of itself, 0.008 radians at position 131072; here it is reduced before it is rounded:
// inv_freq / 2 pi is held as a 64-bit fraction of a turn, its product with the position modulo
// 2^64 is the exact fraction of a turn of that frequency, and the cosine and sine are taken of
// that fraction.  The frequency's own rounding, half a unit of 2^-64 turns times |inv_freq|
// plus one for the shift, times a position below 2^31, stays below 2^-28 turns.
//
// One CTA per token: its first rot / 2 threads compute the cosines and sines once for all
// heads, while the loads of the heads are in flight.  A head belongs to L lanes; a lane's
// jobs are pairs of vectors of V features that rotate together (for the half layout V
// features and the V that lie rot / 2 further; for interleaved pairs both vectors side by
// side), so a rotation never leaves a lane, or, beyond rot, single vectors.  The mean is a
// sum over the L lanes by shuffles.
//
// Bound: the bytes of the rows and of the outputs for prompts; latency for decoding.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "q4_decode.cuh"

namespace q4 {

namespace {

// floor(2^64 / (2 pi))
constexpr uint64_t kTurnsPerRadian = 0x28BE60DB9391054Aull;

// inv_freq / 2 pi modulo one turn, as a fraction of 2^64.
__device__ __forceinline__ uint64_t turns_of(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int e = static_cast<int>((bits >> 23) & 255u);
    const uint64_t m = e != 0 ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int k = 150 - (e != 0 ? e : 1);   // |f| = m 2^-k
    const uint64_t lo = m * kTurnsPerRadian, hi = __umul64hi(m, kTurnsPerRadian);
    uint64_t r;
    if (k <= 0) r = k > -64 ? lo << -k : 0;
    else if (k < 64) r = (lo >> k) | (hi << (64 - k));
    else r = k < 128 ? hi >> (k - 64) : 0;
    return (bits >> 31) != 0 ? 0 - r : r;
}

__device__ __forceinline__ void cos_sin(int position, float f, float scale, float &c, float &s) {
    const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns_of(f);
    // the upper half, rounded, as a signed fraction of half a turn
    const float x = static_cast<float>(static_cast<int32_t>((turns + 0x80000000ull) >> 32)) * 0x1p-31f;
    sincospif(x, &s, &c);
    if (!(fabsf(f) <= 3.4e38f)) c = s = __int_as_float(0x7fc00000);
    c *= scale;
    s *= scale;
}

template <typename T>
__device__ __forceinline__ float widen(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T narrow(float v) {
    if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// V features in accesses of up to 16 bytes.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float *out) {
    if constexpr (V == 1) {
        out[0] = widen(*p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + i);
            out[i] = a.x, out[i + 1] = a.y, out[i + 2] = a.z, out[i + 3] = a.w;
        }
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[2 * i] = __uint_as_float(w[i] << 16);
            out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <typename C, int V>
__device__ __forceinline__ void store_vec(C *p, const float *in) {
    if constexpr (V == 1) {
        *p = narrow<C>(in[0]);
    } else {
        C v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = narrow<C>(in[i]);
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v);
    }
}

constexpr int kRopeThreads = 384;

}  // namespace

// T: type of q, k, v; C: of the cache and q_out; V features an access, L lanes a head, NJ jobs
// a lane at most.
template <typename T, typename C, int V, int L, int NJ>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const q4_rope_append_t g, unsigned int *bounds) {
    __shared__ float cs[kMaxHeadD / 2], sn[kMaxHeadD / 2];
    const int t = blockIdx.x;
    const int D = g.cache.D, half = g.rot / 2;
    const bool pairs_apart = g.layout == Q4_ROPE_HALF;
    const int pairs = g.rot / (2 * V), jobs = pairs + (D - g.rot) / V;
    const int heads = g.Hq + (g.k != nullptr ? 2 * g.cache.heads : 0);
    const int sub = threadIdx.x / L, lane = threadIdx.x % L, per = blockDim.x / L;
    auto ib = [&](int64_t r, int64_t rows, int c, const void *p, int esize) {
        return q4_in_bounds(r >= 0 && r < rows && c >= 0 && c + V <= D &&
                                reinterpret_cast<uintptr_t>(p) % (V == 1 ? esize : 16) == 0, bounds);
    };
    wait_prior_grid();
    allow_next_grid();
    bool turned = false;   // the cosines and sines are in shared memory
    for (int h0 = 0; h0 < heads; h0 += per) {
        const int h = h0 + sub;
        const bool have = h < heads;
        // head `at` of kind 0 (query), 1 (key) or 2 (value)
        int kind = 0, at = h;
        if (h >= g.Hq) kind = 1, at = h - g.Hq;
        if (kind == 1 && at >= g.cache.heads) kind = 2, at -= g.cache.heads;
        const T *src = static_cast<const T *>(kind == 0 ? g.q : kind == 1 ? g.k : g.v) +
                       static_cast<int64_t>(t) * (kind == 0 ? g.q_stride : kind == 1 ? g.k_stride : g.v_stride) +
                       static_cast<int64_t>(at) * D;
        float a[NJ][V], b[NJ][V];
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
            const int j = n * L + lane;
#pragma unroll
            for (int v = 0; v < V; ++v) a[n][v] = b[n][v] = 0.0f;
            if (have && j < jobs) {
                const bool pair = j < pairs;
                const int c = pair ? (pairs_apart ? j * V : 2 * j * V) : g.rot + (j - pairs) * V;
                if (ib(t, g.T, c, src + c, sizeof(T))) load_vec<T, V>(src + c, a[n]);
                const int c2 = c + (pairs_apart ? half : V);
                if (pair && ib(t, g.T, c2, src + c2, sizeof(T))) load_vec<T, V>(src + c2, b[n]);
            }
        }
        if (!turned) {
            for (int i = threadIdx.x; i < half; i += blockDim.x)
                cos_sin(g.positions[t], g.inv_freq[i], g.scale, cs[i], sn[i]);
            __syncthreads();
            turned = true;
        }
        const float *gamma = kind == 0 ? g.q_gamma : kind == 1 ? g.k_gamma : nullptr;
        float ss = 0.0f;
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(a[n][v], a[n][v], fmaf(b[n][v], b[n][v], ss));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float r = 1.0f / sqrtf(ss / static_cast<float>(D) + g.eps);
        if (!have) continue;   // (lanes that skip the stores meet the others at the next turn's sums)
        C *dst;
        if (kind == 0) {
            dst = static_cast<C *>(g.q_out) + (static_cast<int64_t>(t) * g.Hq + at) * D;
        } else {
            const int64_t slot = g.slots != nullptr ? g.slots[t] : t;
            const int64_t page = slot >= 0 ? slot / g.cache.page : -1;
            if (page < 0 || page >= g.cache.pages) continue;
            dst = static_cast<C *>(kind == 1 ? g.cache.k : g.cache.v) + page * g.cache.page_stride +
                  at * g.cache.head_stride + (slot - page * g.cache.page) * g.cache.row_stride;
        }
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
            const int j = n * L + lane;
            if (j >= jobs) continue;
            const bool pair = j < pairs;
            const int c = pair ? (pairs_apart ? j * V : 2 * j * V) : g.rot + (j - pairs) * V;
            const int c2 = c + (pairs_apart ? half : V);
            if (gamma != nullptr) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    a[n][v] = a[n][v] * r * gamma[c + v];
                    if (pair) b[n][v] = b[n][v] * r * gamma[c2 + v];
                }
            }
            if (pair && kind != 2) {
                if (pairs_apart) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float x = a[n][v], y = b[n][v], cc = cs[c + v], s = sn[c + v];
                        a[n][v] = cc * x - s * y;
                        b[n][v] = s * x + cc * y;
                    }
                } else if constexpr (V > 1) {
#pragma unroll
                    for (int v = 0; v < V; v += 2) {
                        float x = a[n][v], y = a[n][v + 1], cc = cs[(c + v) / 2], s = sn[(c + v) / 2];
                        a[n][v] = cc * x - s * y;
                        a[n][v + 1] = s * x + cc * y;
                        x = b[n][v], y = b[n][v + 1], cc = cs[(c2 + v) / 2], s = sn[(c2 + v) / 2];
                        b[n][v] = cc * x - s * y;
                        b[n][v + 1] = s * x + cc * y;
                    }
                } else {
                    const float x = a[n][0], y = b[n][0], cc = cs[c / 2], s = sn[c / 2];
                    a[n][0] = cc * x - s * y;
                    b[n][0] = s * x + cc * y;
                }
            }
            if (ib(t, g.T, c, dst + c, sizeof(C))) store_vec<C, V>(dst + c, a[n]);
            if (pair && ib(t, g.T, c2, dst + c2, sizeof(C))) store_vec<C, V>(dst + c2, b[n]);
        }
    }
}

template <typename T, typename C>
static int launch_rope_of(const q4_rope_append_t &a, cudaStream_t stream) {
    const int D = a.cache.D, half = a.rot / 2;
    const int heads = a.Hq + (a.k != nullptr ? 2 * a.cache.heads : 0);
    // vectors of 8 features where every row, head, pair and page starts on 16 bytes
    auto rows = [&](const void *p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; };
    const bool wide = D % 8 == 0 && a.rot % 16 == 0 && (a.layout != Q4_ROPE_HALF || half % 8 == 0) &&
                      rows(a.q, a.q_stride) && rows(a.k, a.k_stride) && rows(a.v, a.v_stride) && aligned(a.q_out, 16) &&
                      rows(a.cache.k, a.cache.page_stride) && rows(a.cache.v, a.cache.head_stride) &&
                      a.cache.row_stride % 8 == 0;
    auto launch = [&](auto kernel, int L) {
        const int need = (heads * L + 31) / 32 * 32;
        // as few turns as the largest block allows, and no more threads than those turns need
        const int turns = (need + kRopeThreads - 1) / kRopeThreads;
        const unsigned threads = static_cast<unsigned>((need / turns + 31) / 32 * 32);
        return launch_overlappable(kernel, dim3(static_cast<unsigned>(a.T)), dim3(threads), 0, stream,
                                   call_options().overlap, a, bounds_counter());
    };
    if (!wide) return launch(rope_append_kernel<T, C, 1, 32, kMaxHeadD / 32>, 32);
    const int jobs = a.rot / 16 + (D - a.rot) / 8;
    if (jobs <= 4) return launch(rope_append_kernel<T, C, 8, 4, 1>, 4);
    if (jobs <= 8) return launch(rope_append_kernel<T, C, 8, 8, 1>, 8);
    return jobs <= 16 ? launch(rope_append_kernel<T, C, 8, 16, 1>, 16)
                      : launch(rope_append_kernel<T, C, 8, 32, 1>, 32);
}

int launch_rope_append(const q4_rope_append_t &a, cudaStream_t stream) {
    const bool half_type = a.cache.dtype == Q4_F16;
    if (a.dtype == Q4_F32)
        return half_type ? launch_rope_of<float, __half>(a, stream) : launch_rope_of<float, __nv_bfloat16>(a, stream);
    return half_type ? launch_rope_of<__nv_bfloat16, __half>(a, stream)
                     : launch_rope_of<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace q4
