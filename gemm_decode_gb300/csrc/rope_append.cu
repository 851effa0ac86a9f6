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
// Bound: latency for decoding (4.0 us for 4 tokens); for prompts the chain from a row's load to
// its store with what an SM's CTAs have in flight: 25.4 us for the 101 MB of 4096 tokens, 4.0
// TB/s, 0.59 of measured.  Heads in a loop with the cosines and weights in registers (27 us),
// and four tokens to a CTA with the next one's rows on their way (32 us), gained nothing.
#include <cuda_bf16.h>

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
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<C, __half>::value)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(in[2 * i + 1]), "f"(in[2 * i]));
            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(in[2 * i + 1]), "f"(in[2 * i]));
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// v * r * gamma
template <int V>
__device__ __forceinline__ void scale_vec(float *v, float r, const float *gamma) {
    if constexpr (V == 1) {
        v[0] = v[0] * r * gamma[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(gamma + i));
            const float2 rr = make_float2(r, r);
            const float2 f = __fmul2_rn(__fmul2_rn(make_float2(v[i], v[i + 1]), rr), make_float2(w.x, w.y));
            const float2 h = __fmul2_rn(__fmul2_rn(make_float2(v[i + 2], v[i + 3]), rr), make_float2(w.z, w.w));
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = h.x, v[i + 3] = h.y;
        }
    }
}

// Two pairs (x, y) turned, the first and the second of each.
__device__ __forceinline__ void turn2(float &x0, float &x1, float &y0, float &y1, const float *c, const float *s) {
    const float2 cc = *reinterpret_cast<const float2 *>(c), ss = *reinterpret_cast<const float2 *>(s);
    const float2 x = make_float2(x0, x1), y = make_float2(y0, y1);
    const float2 nx = __ffma2_rn(x, cc, __fmul2_rn(y, make_float2(-ss.x, -ss.y)));
    const float2 ny = __ffma2_rn(x, ss, __fmul2_rn(y, cc));
    x0 = nx.x, x1 = nx.y;
    y0 = ny.x, y1 = ny.y;
}

// Threads of a CTA at most; of a call of many tokens (kManyTokens to an SM) fewer, which have
// their heads in turn: 4096 tokens of 32 + 2 x 8 heads (101 MB) 28.2 us with 384, 25.4 with 128;
// 4 tokens 4.0 and 5.5.
constexpr int kRopeThreads = 384, kPromptThreads = 128, kManyTokens = 8;

}  // namespace

// T: type of q, k, v; C: of the cache and q_out; V features an access, L lanes a head, NJ jobs
// a lane at most.
template <typename T, typename C, int V, int L, int NJ>
__global__ void __launch_bounds__(kRopeThreads, V == 1 ? 2 : 4) rope_append_kernel(const q4_rope_append_t g, unsigned int *bounds) {
    __shared__ __align__(16) float cs[kMaxHeadD / 2], sn[kMaxHeadD / 2];
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
    const int position = g.rot > 0 ? g.positions[t] : 0;
    const int slot = g.slots != nullptr ? g.slots[t] : t;   // (on its way with the heads)
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
                cos_sin(position, g.inv_freq[i], g.scale, cs[i], sn[i]);
            __syncthreads();
            turned = true;
        }
        const float *gamma = kind == 0 ? g.q_gamma : kind == 1 ? g.k_gamma : nullptr;
        float r = 1.0f;
        if (g.q_gamma != nullptr || g.k_gamma != nullptr) {   // (the sums are of all lanes)
            float ss = 0.0f;
            float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int v = 0; v < V; v += V == 1 ? 1 : 2) {
                    if constexpr (V == 1) {
                        ss = fmaf(a[n][v], a[n][v], fmaf(b[n][v], b[n][v], ss));
                    } else {
                        const float2 x = make_float2(a[n][v], a[n][v + 1]), y = make_float2(b[n][v], b[n][v + 1]);
                        sq = __ffma2_rn(x, x, __ffma2_rn(y, y, sq));
                    }
                }
            ss += sq.x + sq.y;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
            r = rsqrtf(ss / static_cast<float>(D) + g.eps);   // (off by 2^-22, the rounding to come by 2^-11)
        }
        if (!have) continue;   // (lanes that skip the stores meet the others at the next turn's sums)
        C *dst;
        if (kind == 0) {
            dst = static_cast<C *>(g.q_out) + (static_cast<int64_t>(t) * g.Hq + at) * D;
        } else {
            const int page = slot >= 0 ? slot / g.cache.page : -1;
            if (page < 0 || page >= g.cache.pages) continue;
            dst = static_cast<C *>(kind == 1 ? g.cache.k : g.cache.v) + static_cast<int64_t>(page) * g.cache.page_stride +
                  at * g.cache.head_stride + static_cast<int64_t>(slot - page * g.cache.page) * g.cache.row_stride;
        }
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
            const int j = n * L + lane;
            if (j >= jobs) continue;
            const bool pair = j < pairs;
            const int c = pair ? (pairs_apart ? j * V : 2 * j * V) : g.rot + (j - pairs) * V;
            const int c2 = c + (pairs_apart ? half : V);
            if (gamma != nullptr) {
                scale_vec<V>(a[n], r, gamma + c);
                if (pair) scale_vec<V>(b[n], r, gamma + c2);
            }
            if (pair && kind != 2) {
                if constexpr (V == 1) {
                    const int at = pairs_apart ? c : c / 2;
                    const float x = a[n][0], y = b[n][0];
                    a[n][0] = cs[at] * x - sn[at] * y;
                    b[n][0] = sn[at] * x + cs[at] * y;
                } else if (pairs_apart) {
#pragma unroll
                    for (int v = 0; v < V; v += 2)
                        turn2(a[n][v], a[n][v + 1], b[n][v], b[n][v + 1], cs + j * V + v, sn + j * V + v);
                } else {
#pragma unroll
                    for (int v = 0; v < V; v += 4) {
                        turn2(a[n][v], a[n][v + 2], a[n][v + 1], a[n][v + 3], cs + j * V + v / 2, sn + j * V + v / 2);
                        turn2(b[n][v], b[n][v + 2], b[n][v + 1], b[n][v + 3], cs + j * V + (V + v) / 2, sn + j * V + (V + v) / 2);
                    }
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
    // vectors of 8 features where every row, head, pair and page and the norm weights start on 16 bytes
    auto rows = [&](const void *p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; };
    const bool wide = D % 8 == 0 && a.rot % 16 == 0 && (a.layout != Q4_ROPE_HALF || half % 8 == 0) &&
                      rows(a.q, a.q_stride) && rows(a.k, a.k_stride) && rows(a.v, a.v_stride) && aligned(a.q_out, 16) &&
                      rows(a.cache.k, a.cache.page_stride) && rows(a.cache.v, a.cache.head_stride) &&
                      a.cache.row_stride % 8 == 0 && aligned(a.q_gamma, 16) && aligned(a.k_gamma, 16);
    auto launch = [&](auto kernel, int L) {
        const int need = (heads * L + 31) / 32 * 32;
        // as few turns as the block allows, and no more threads than those turns need
        const int most = a.T >= kManyTokens * device_info().sms ? kPromptThreads : kRopeThreads;
        const int turns = (need + most - 1) / most;
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
