// beam_step.cu -- one step of a beam search: the K best of score_w + l_wv - log sum exp l_w over
// a group's beams and the vocabulary.
//
// Within a beam the order of the continuations is that of its logits, so the first kernel
// needs no sums: a CTA reads a chunk of one beam's logits once, into registers, and keeps the
// K largest as 64-bit keys (the logit's bits in an order that compares as an integer, then the
// token, lower first), together with the chunk's maximum and sum of exponentials.
// Of 32 lanes whose own maxima are sorted, the K-th largest is no larger than the K-th largest
// logit of the warp; the largest of these over the warps is a bound that K logits or more
// reach, and few more than K do.  Those are collected and the K largest of them taken out one
// by one.  The second kernel joins the chunks of each beam, forms the scores (binary64: the
// order of continuations of different beams whose scores are close hangs on it) and takes
// the K best of the group.
//
// Bound: the bytes of the logits.
#include <atomic>

#include "q4_decode.cuh"

namespace q4 {

namespace {

constexpr int kBeamThreads = 256;
constexpr int kPerThread = 16;
constexpr int kBlock = kBeamThreads * kPerThread;   // logits in registers at a time
constexpr int kMaxChunks = 64;                      // of one beam

// What a chunk leaves: maximum, sum of exponentials, and keys.
struct BeamLayout {
    int chunks;
    int64_t chunk;   // logits, a multiple of kBlock
};
BeamLayout beam_layout(int64_t V) {
    const int64_t blocks = (V + kBlock - 1) / kBlock, each = (blocks + kMaxChunks - 1) / kMaxChunks;
    return BeamLayout{static_cast<int>((blocks + each - 1) / each), each * kBlock};
}

// Larger logit first, then lower token; 0: no logit.  (l + 0: both zeros are one value.)
__device__ __forceinline__ uint64_t key_of(float l, uint32_t token) {
    if (!(fabsf(l) <= 3.402823466e38f)) return 0;
    const uint32_t b = __float_as_uint(l + 0.0f);
    const uint32_t u = (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
    return static_cast<uint64_t>(u) << 32 | (0xffffffffu - token);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((u & 0x80000000u) != 0 ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint32_t token_of(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t n = __shfl_xor_sync(~0u, k, o);
        k = n > k ? n : k;
    }
    return k;
}

// The K largest of n distinct keys (zeros: none) by one warp, in descending order, into out
// (zeros where there are fewer).  The list is used up.
__device__ __forceinline__ void warp_top(uint64_t *list, int n, int K, uint64_t *out, int lane) {
    uint64_t best = 0;
    int at = lane;
    auto look = [&]() {
        best = 0;
        for (int i = lane; i < n; i += 32)
            if (list[i] > best) best = list[i], at = i;
    };
    look();
    for (int j = 0; j < K; ++j) {
        const uint64_t top = warp_max(best);
        if (lane == 0) out[j] = top;
        if (top != 0 && best == top) {
            list[at] = 0;
            look();
        }
    }
    __syncwarp();
}

}  // namespace

__global__ void __launch_bounds__(kBeamThreads) beam_chunk_kernel(const BeamArgs g, int64_t chunk, int wide,
                                                                  float2 *stats, uint64_t *keys) {
    // candidates: the K best so far, and at most every logit of a block
    extern __shared__ uint64_t list[];   // [kMaxBeams + kBlock]
    __shared__ uint64_t bound[kBeamThreads / 32], kept[kMaxBeams];
    __shared__ float warp_m[kBeamThreads / 32], warp_s[kBeamThreads / 32];
    __shared__ int count;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.y, K = g.K;
    wait_prior_grid();
    allow_next_grid();
    const float cum = g.scores[row];
    if (!(fabsf(cum) <= 3.402823466e38f) || (g.finished != nullptr && g.finished[row] != 0)) return;
    const float *l = g.logits + row * g.row_stride;
    const int64_t v0 = blockIdx.x * chunk, v1 = v0 + chunk < g.V ? v0 + chunk : g.V;
    float m = -__int_as_float(0x7f800000), s = 0.0f;
    if (threadIdx.x < kMaxBeams) kept[threadIdx.x] = 0;
    for (int64_t b0 = v0; b0 < v1; b0 += kBlock) {
        if (threadIdx.x == 0) count = 0;
        float x[kPerThread];
        // 16 logits a thread, four side by side where rows are aligned for it
        auto place = [&](int i) {
            return wide ? b0 + (i / 4 * kBeamThreads + threadIdx.x) * 4 + i % 4 : b0 + i * kBeamThreads + threadIdx.x;
        };
        auto ib = [&](int64_t v, int n) {
            return q4_in_bounds(v >= 0 && v + n <= g.V && row < g.groups * g.W, g.bounds);
        };
        if (wide) {
#pragma unroll
            for (int i = 0; i < kPerThread; i += 4) {
                const int64_t v = place(i);
                float4 f = make_float4(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000),
                                       __int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
                if (v + 4 <= v1) {
                    if (ib(v, 4)) f = __ldcs(reinterpret_cast<const float4 *>(l + v));
                } else {
                    if (v < v1 && ib(v, 1)) f.x = l[v];
                    if (v + 1 < v1 && ib(v + 1, 1)) f.y = l[v + 1];
                    if (v + 2 < v1 && ib(v + 2, 1)) f.z = l[v + 2];
                }
                x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const int64_t v = place(i);
                x[i] = v < v1 && ib(v, 1) ? __ldcs(l + v) : __int_as_float(0x7fc00000);
            }
        }
        uint64_t best = 0;
        float top = -__int_as_float(0x7f800000);
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const uint64_t k = key_of(x[i], static_cast<uint32_t>(place(i)));
            best = k > best ? k : best;
        }
        if (best != 0) top = logit_of(best);
        // running maximum and sum of this thread
        if (best != 0) {
            const float nm = fmaxf(m, top);
            s *= expf(m - nm);   // m = -inf at first: 0
            m = nm;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
                if (fabsf(x[i]) <= 3.402823466e38f) s += expf(x[i] - m);
        }
        // the K-th largest of the lanes' maxima: lane i holds the i-th largest after the sort
        uint64_t o = best;
#pragma unroll
        for (int w = 2; w <= 32; w <<= 1) {
#pragma unroll
            for (int d = w >> 1; d > 0; d >>= 1) {
                const uint64_t n = __shfl_xor_sync(~0u, o, d);
                const bool down = (lane & w) == 0 || w == 32;   // descending half
                const bool first = (lane & d) == 0;
                o = (first == down) == (o > n) ? o : n;
            }
        }
        const uint64_t kth = __shfl_sync(~0u, o, K - 1);
        if (lane == 0) bound[warp] = kth;
        __syncthreads();
        uint64_t least = kept[K - 1];
#pragma unroll
        for (int w = 0; w < kBeamThreads / 32; ++w) least = bound[w] > least ? bound[w] : least;
        if (best != 0 && best >= least) {
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const uint64_t k = key_of(x[i], static_cast<uint32_t>(place(i)));
                if (k != 0 && k >= least) list[kMaxBeams + atomicAdd(&count, 1)] = k;
            }
        }
        __syncthreads();
        if (warp == 0) {
            // the order of the list is that of the atomics; the keys are distinct, so what is chosen is not
            for (int i = lane; i < kMaxBeams; i += 32) list[i] = i < K ? kept[i] : 0;
            __syncwarp();
            warp_top(list, kMaxBeams + count, K, kept, lane);
        }
        __syncthreads();
    }
    // the chunk's maximum and sum, in a fixed order
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(~0u, wm, o));
    float ws = m > -__int_as_float(0x7f800000) ? s * expf(m - wm) : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(~0u, ws, o);
    if (lane == 0) warp_m[warp] = wm, warp_s[warp] = ws;
    __syncthreads();
    const int64_t slot = static_cast<int64_t>(row) * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) {
        float am = warp_m[0], as = 0.0f;
        for (int w = 1; w < kBeamThreads / 32; ++w) am = fmaxf(am, warp_m[w]);
        for (int w = 0; w < kBeamThreads / 32; ++w)
            if (warp_s[w] > 0.0f) as += warp_s[w] * expf(warp_m[w] - am);
        stats[slot] = make_float2(am, as);
    }
    if (threadIdx.x < K) keys[slot * K + threadIdx.x] = kept[threadIdx.x];
}

// One CTA per group: warps take its beams in turn, then the first warp chooses.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps) beam_join_kernel(const BeamArgs g, int chunks, const float2 *stats,
                                                                    const uint64_t *keys) {
    extern __shared__ uint64_t lists[];   // [kJoinWarps][chunks * K]
    __shared__ uint64_t best[kMaxBeams * kMaxBeams];
    __shared__ double score[kMaxBeams * kMaxBeams];
    __shared__ uint64_t taken[kJoinWarps][kMaxBeams];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = g.K;
    const int group = blockIdx.x;
    const double none = -__longlong_as_double(0x7ff0000000000000ll);
    wait_prior_grid();
    allow_next_grid();
    for (int w = warp; w < g.W; w += kJoinWarps) {
        const int64_t row = static_cast<int64_t>(group) * g.W + w;
        const float cum = g.scores[row];
        const bool live = fabsf(cum) <= 3.402823466e38f, done = g.finished != nullptr && g.finished[row] != 0;
        if (!live || done) {
            for (int j = lane; j < K; j += 32) {
                const bool end = live && j == 0;
                best[w * K + j] = end ? 0xffffffffu - static_cast<uint32_t>(g.eos) : 0;
                score[w * K + j] = end ? static_cast<double>(cum) : none;
            }
            continue;
        }
        uint64_t *list = lists + static_cast<size_t>(warp) * chunks * K;
        for (int i = lane; i < chunks * K; i += 32) list[i] = __ldcg(keys + row * chunks * K + i);
        float m = -__int_as_float(0x7f800000);
        for (int c = lane; c < chunks; c += 32) m = fmaxf(m, __ldcg(&stats[row * chunks + c].x));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        double s = 0.0;
        for (int c = lane; c < chunks; c += 32) {
            const float2 p = __ldcg(stats + row * chunks + c);
            if (p.y > 0.0f) s += static_cast<double>(p.y * expf(p.x - m));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        const double lse = static_cast<double>(m) + log(s);
        __syncwarp();
        warp_top(list, chunks * K, K, taken[warp], lane);
        for (int j = lane; j < K; j += 32) {
            const uint64_t k = taken[warp][j];
            best[w * K + j] = k;
            score[w * K + j] = k != 0 ? static_cast<double>(cum) + (static_cast<double>(logit_of(k)) - lse) : none;
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp != 0) return;
    // The places are in the order of beams, and within a beam of scores, then tokens: of equal
    // scores the lower place is the one with the lower beam, then the lower token.
    const int n = g.W * K;
    double top = none;
    int at = n;
    auto look = [&]() {
        top = none;
        at = n;
        for (int i = lane; i < n; i += 32)
            if (score[i] > top) top = score[i], at = i;
    };
    look();
    for (int j = 0; j < K; ++j) {
        double t = top;
        int a = at;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double t2 = __shfl_xor_sync(~0u, t, o);
            const int a2 = __shfl_xor_sync(~0u, a, o);
            if (t2 > t || (t2 == t && a2 < a)) t = t2, a = a2;
        }
        if (lane == 0) {
            const int64_t to = static_cast<int64_t>(group) * K + j;
            const bool found = a < n;
            const int token = found ? static_cast<int>(token_of(best[a])) : -1;
            g.tokens[to] = token;
            g.parents[to] = found ? a / K : -1;
            g.out_scores[to] = static_cast<float>(t);
            if (g.out_finished != nullptr) g.out_finished[to] = found && token == g.eos;
        }
        if (a < n && a == at) {
            score[a] = none;
            look();
        }
    }
}

int64_t beam_workspace_bytes(int groups, int W, int K, int64_t V) {
    const BeamLayout b = beam_layout(V);
    return static_cast<int64_t>(groups) * W * b.chunks * (8 + 8 * static_cast<int64_t>(K));
}

int launch_beam_step(const BeamArgs &a, cudaStream_t stream) {
    const BeamLayout b = beam_layout(a.V);
    const int rows = a.groups * a.W;
    uint64_t *keys = static_cast<uint64_t *>(a.workspace);
    float2 *stats = reinterpret_cast<float2 *>(keys + static_cast<int64_t>(rows) * b.chunks * a.K);
    const int wide = aligned(a.logits, 16) && a.row_stride % 4 == 0;
    const size_t list = (kMaxBeams + kBlock) * sizeof(uint64_t);
    const bool overlap = call_options().overlap;
    // the grid's second dimension has 65535 places
    for (int r0 = 0; r0 < rows; r0 += 65535 / a.W * a.W) {
        BeamArgs p = a;
        const int part = rows - r0 < 65535 / a.W * a.W ? rows - r0 : 65535 / a.W * a.W;
        p.logits += static_cast<int64_t>(r0) * a.row_stride;
        p.scores += r0;
        if (p.finished != nullptr) p.finished += r0;
        const int st = launch_overlappable(beam_chunk_kernel, dim3(static_cast<unsigned>(b.chunks), static_cast<unsigned>(part)),
                                           dim3(kBeamThreads), list, stream, overlap, p, b.chunk, wide,
                                           stats + static_cast<int64_t>(r0) * b.chunks,
                                           keys + static_cast<int64_t>(r0) * b.chunks * a.K);
        if (st != Q4_OK) return st;
    }
    const size_t lists = static_cast<size_t>(kJoinWarps) * b.chunks * a.K * sizeof(uint64_t);   // at most 128 KB
    static std::atomic<bool> configured[64];
    const int st = allow_smem(beam_join_kernel, kJoinWarps * kMaxChunks * kMaxBeams * sizeof(uint64_t), configured);
    if (st != Q4_OK) return st;
    return launch_overlappable(beam_join_kernel, dim3(static_cast<unsigned>(a.groups)), dim3(32 * kJoinWarps), lists,
                               stream, true, a, b.chunks, stats, keys);
}

}  // namespace q4
