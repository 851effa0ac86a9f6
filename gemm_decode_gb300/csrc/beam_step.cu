// beam_step.cu -- one step of a beam search: the K best of score_w + l_wv - log sum exp l_w over
// a group's beams and the vocabulary.
//
// Within a beam the order of the continuations is that of its logits, so the first kernel
// needs no sums: a CTA reads a chunk of one beam's logits, sixteen to a thread at a time, and
// keeps of each sixteen the largest, and the maximum and the sum of exponentials of all.  The
// K best of the chunk lie in the sixteens with the K largest maxima: of 32 threads whose own
// largest are sorted, the K-th is a bound that K sixteens or more reach, and a few more than K
// do.  Those are read once more and the K best chosen as 64-bit keys (the logit's bits in an
// order that compares as an integer, then the token, lower first).  (Picking out the best while
// reading cost 470 instructions for 512 logits, three times the sums.)  The second kernel joins
// the chunks of each beam, forms the scores (binary64: the order of continuations of different
// beams whose scores are close hangs on it) and takes the K best of the group.
//
// Bound: latency for one group (9 us for four beams of 151936 tokens: two dependent launches, each
// a chain of loads, a sort and counts); for many the chain of a CTA's blocks and its choice at the
// end: 16 groups of 8 beams of 128256 tokens (66 MB) 28.5 us a call on changing logits, 2.3 TB/s,
// 0.34 of measured (21 in a graph on the same logits, which L2 holds); for wide beams the choice: 16
// beams, K = 32, 131 us.  More or fewer chunks than one wave of CTAs gains nothing (of 152 SMs: 304
// 29.9 us, 608 26.9, 760 26.5, 912 34.1, 1824 41.3).
#include <algorithm>
#include <atomic>

#include "q4_decode.cuh"

namespace q4 {

namespace {

constexpr int kBeamThreads = 256;
constexpr int kPerThread = 16;
constexpr int kBlock = kBeamThreads * kPerThread;   // logits in registers at a time
constexpr int kMaxChunks = 64;                      // of one beam
constexpr int kChunkCtas = 4;                       // of an SM: chunks wanted

// What a chunk leaves: maximum, sum of exponentials, and keys.
struct BeamLayout {
    int chunks;
    int64_t chunk;   // logits
};
// As many chunks as CTAs are resident on the current device at a time, so that there is one wave of
// them; a block at least to a chunk.
BeamLayout beam_layout(int64_t rows, int64_t V) {
    const int64_t blocks = (V + kBlock - 1) / kBlock;
    const int64_t want = std::min({blocks, std::max<int64_t>(kChunkCtas * device_info().sms / std::max<int64_t>(rows, 1), 1),
                                   static_cast<int64_t>(kMaxChunks)});
    const int64_t chunk = ((V + want - 1) / want + 31) / 32 * 32;   // (chunks start where rows of 16 bytes do)
    return BeamLayout{static_cast<int>((V + chunk - 1) / chunk), chunk};
}

constexpr float kLargest = 3.402823466e38f;

// exp(x), x <= 0, within 2^-21: the product and the function each within 2^-23 and a half
__device__ __forceinline__ float exp_of(float x) { return exp2_fast(x * 1.44269504088896341f); }

// Larger logit first, then lower token; 0: no logit.  (l + 0: both zeros are one value.)
__device__ __forceinline__ uint64_t key_of(float l, uint32_t token) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    const uint32_t u = (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
    return static_cast<uint64_t>(u) << 32 | (0xffffffffu - token);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((u & 0x80000000u) != 0 ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint32_t token_of(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }

// A binary64 number as an integer of the same order (compares of binary64 are slow here), and back.
__device__ __forceinline__ int64_t order_of(double v) {
    const int64_t b = __double_as_longlong(v + 0.0);
    return b < 0 ? b ^ 0x7fffffffffffffffll : b;
}
__device__ __forceinline__ double score_of(int64_t o) {
    return __longlong_as_double(o < 0 ? o ^ 0x7fffffffffffffffll : o);
}

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t n = __shfl_xor_sync(~0u, k, o);
        k = n > k ? n : k;
    }
    return k;
}

constexpr int kRanked = 64;   // keys that are ranked against one another, two a lane
struct WarpScratch {
    uint64_t top[32], key[kRanked];
};

// The K largest of n distinct keys (zeros: none) by one warp, in descending order, into out
// (zeros where there are fewer): each key's place is the number of larger ones.  (Taking the
// maximum K times cost 700 cycles a time.)  Of a long list those that reach the K-th largest of
// the lanes' maxima, as K keys or more do; where that leaves many, they are taken out one by one
// after all, which uses the list up.
__device__ __forceinline__ void warp_top(uint64_t *list, int n, int K, uint64_t *out, WarpScratch &w, int lane) {
    for (int i = lane; i < K; i += 32) out[i] = 0;
    const uint64_t *from = list;
    int count = n;
    uint64_t best = 0;
    if (n > kRanked) {
        for (int i = lane; i < n; i += 32) best = list[i] > best ? list[i] : best;
        w.top[lane] = best;
        __syncwarp();
        int larger = 0;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) larger += w.top[i] > best || (w.top[i] == best && i < lane);
        const uint64_t bound = __shfl_sync(~0u, best, __ffs(__ballot_sync(~0u, larger == K - 1)) - 1);
        count = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const uint64_t k = i0 + lane < n ? list[i0 + lane] : 0;
            const bool in = k != 0 && k >= bound;
            const unsigned all = __ballot_sync(~0u, in);
            const int at = count + __popc(all & ((1u << lane) - 1));
            if (in && at < kRanked) w.key[at] = k;
            count += __popc(all);
        }
        from = w.key;
    }
    __syncwarp();
    if (count <= kRanked) {
        const uint64_t a = lane < count ? from[lane] : 0, b = lane + 32 < count ? from[lane + 32] : 0;
        int ra = 0, rb = 0;
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const uint64_t k = from[i];
            ra += k > a;
            rb += k > b;
        }
        if (a != 0 && ra < K) out[ra] = a;
        if (b != 0 && rb < K) out[rb] = b;
    } else {
        for (int j = 0; j < K; ++j) {
            int at = 0;
            best = 0;
            for (int i = lane; i < n; i += 32)
                if (list[i] > best) best = list[i], at = i;
            const uint64_t top = warp_max(best);
            if (lane == 0) out[j] = top;
            if (top != 0 && best == top) list[at] = 0;
            __syncwarp();
        }
    }
    __syncwarp();
}

// log s, s >= 1, in binary64 and within 2^-24: the power of two apart from the rest (the
// binary64 logarithm itself takes 3000 cycles here).
__device__ __forceinline__ double log_of(float s) {
    int e = static_cast<int>(__float_as_uint(s) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u);   // [1, 2)
    if (f > 1.4142135f) f *= 0.5f, ++e;
    return e * 0.693147180559945309417 + static_cast<double>(log1pf(f - 1.0f));
}

}  // namespace

constexpr int kLong = 64;      // keys of a warp before the best are chosen
constexpr int kSteps = 16;     // blocks whose sixteens' maxima are held
constexpr int kBatch = 16;     // sixteens that a warp reads once more at a time
constexpr int kWarps = kBeamThreads / 32;
struct BeamShared {
    union {
        float top[kSteps][kBeamThreads];                  // of each sixteen
        uint64_t key[kWarps][kLong + kBatch * kPerThread];    // then: keys of each warp
    };
    uint16_t sixteen[kSteps * kBeamThreads];              // those that are read once more
    WarpScratch scratch[kWarps];
    uint64_t kept[(kWarps + 1) * kMaxBeams], chosen[kMaxBeams];
    float bound[kWarps];
    float2 sums[kWarps];
    int count, keys;
};
constexpr int kFew = (kWarps * (kLong + kBatch * kPerThread) - kMaxBeams) / kPerThread;   // sixteens whose keys all have room

__global__ void __launch_bounds__(kBeamThreads, kChunkCtas) beam_chunk_kernel(const BeamArgs g, int64_t chunk, int wide,
                                                                     float2 *stats, uint64_t *keys) {
    extern __shared__ __align__(16) unsigned char beam_raw[];
    BeamShared &sh = *reinterpret_cast<BeamShared *>(beam_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x, K = g.K;   // (rows in the grid's first dimension: up to 2^31 of them)
    wait_prior_grid();
    allow_next_grid();
    const float cum = g.scores[row];
    if (!(fabsf(cum) <= kLargest) || (g.finished != nullptr && g.finished[row] != 0)) return;
    const float *l = g.logits + row * g.row_stride;
    const int64_t v0 = blockIdx.y * chunk, v1 = v0 + chunk < g.V ? v0 + chunk : g.V;
    const float none = -__int_as_float(0x7f800000);
    auto ib = [&](int64_t v, int n) {
        return q4_in_bounds(v >= 0 && v + n <= g.V && row < g.groups * g.W, g.bounds);
    };
    // a thread's sixteen of a block, four side by side where rows are aligned for it
    auto place = [&](int i) { return wide ? i / 4 * (4 * kBeamThreads) + i % 4 : i * kBeamThreads; };
    auto fetch = [&](int64_t b0, int mine, float *x) {
        const float *p = l + b0 + mine;
        const int left = static_cast<int>(v1 - b0 < kBlock ? v1 - b0 : kBlock) - mine;   // this thread's, from p on
        if (wide) {
#pragma unroll
            for (int i = 0; i < kPerThread; i += 4) {
                float4 f = make_float4(none, none, none, none);
                if (place(i) + 4 <= left) {
                    if (ib(b0 + mine + place(i), 4)) f = __ldg(reinterpret_cast<const float4 *>(p + place(i)));
                } else {
                    if (place(i) < left && ib(b0 + mine + place(i), 1)) f.x = p[place(i)];
                    if (place(i) + 1 < left && ib(b0 + mine + place(i) + 1, 1)) f.y = p[place(i) + 1];
                    if (place(i) + 2 < left && ib(b0 + mine + place(i) + 2, 1)) f.z = p[place(i) + 2];
                }
                x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
                x[i] = place(i) < left && ib(b0 + mine + place(i), 1) ? __ldg(p + place(i)) : none;
        }
    };
    // what is not finite counts as -inf, and is never chosen
    auto finite = [&](float *x) {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
            if (!(fabsf(x[i]) <= kLargest)) x[i] = none;
    };
    const int mine = wide ? 4 * threadIdx.x : threadIdx.x;
    float m = none, s = 0.0f;   // the thread's maximum and sum
    for (int i = threadIdx.x; i < kMaxBeams; i += kBeamThreads) sh.kept[i] = 0;
    float x[kPerThread];
    fetch(v0, mine, x);
    for (int64_t part0 = v0; part0 < v1; part0 += kSteps * kBlock) {
        const int steps = static_cast<int>(std::min<int64_t>(kSteps, (v1 - part0 + kBlock - 1) / kBlock));
        float most = none;
        if (threadIdx.x == 0) sh.count = sh.keys = 0;
        for (int step = 0; step < steps; ++step) {
            const int64_t b0 = part0 + static_cast<int64_t>(step) * kBlock;
            float next[kPerThread];
            if (b0 + kBlock < v1) fetch(b0 + kBlock, mine, next);   // on its way while these are looked at
            float top, part;
            auto look = [&]() {   // the largest, and the sum relative to the running maximum
                top = fmaxf(x[0], x[1]);
#pragma unroll
                for (int i = 2; i < kPerThread; i += 2) top = max3(top, x[i], x[i + 1]);
                const float nm = fmaxf(m, top), ref = nm > none ? nm : 0.0f;
                float2 sum = make_float2(0.0f, 0.0f);
                const float2 minus = make_float2(-ref, -ref), log2e = make_float2(1.44269504088896341f, 1.44269504088896341f);
#pragma unroll
                for (int i = 0; i < kPerThread; i += 2) {
                    const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), minus), log2e);
                    sum = __fadd2_rn(sum, make_float2(exp2_fast(y.x), exp2_fast(y.y)));
                }
                part = sum.x + sum.y;
            };
            look();
            if (!(top <= kLargest && part <= kLargest)) {   // (infinities show in the maximum, NaN in the sum)
                finite(x);
                look();
            }
            if (top > m) {
                s *= exp_of(m - top);   // m = -inf at first: 0
                m = top;
            }
            s += part;
            most = fmaxf(most, top);
            sh.top[step][threadIdx.x] = top;
            if (steps > 1) {
#pragma unroll
                for (int i = 0; i < kPerThread; ++i) x[i] = next[i];
            }
        }
        // ---- the K best of the part, and of those before it
        // the K-th largest of the lanes' maxima: lane i holds the i-th largest after the sort
        float o = most;
#pragma unroll
        for (int w = 2; w <= 32; w <<= 1) {
#pragma unroll
            for (int d = w >> 1; d > 0; d >>= 1) {
                const float n = __shfl_xor_sync(~0u, o, d);
                const bool down = (lane & w) == 0 || w == 32;   // descending half
                const bool lower = (lane & d) == 0;
                o = lower == down ? fmaxf(o, n) : fminf(o, n);
            }
        }
        const float kth = __shfl_sync(~0u, o, K - 1);
        if (lane == 0) sh.bound[warp] = kth;
        __syncthreads();
        float least = sh.kept[K - 1] != 0 ? logit_of(sh.kept[K - 1]) : none;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) least = fmaxf(least, sh.bound[w]);
        if (most >= least && most > none)
            for (int step = 0; step < steps; ++step) {
                const float top = sh.top[step][threadIdx.x];
                if (top >= least && top > none)
                    sh.sixteen[atomicAdd(&sh.count, 1)] = static_cast<uint16_t>(step * kBeamThreads + threadIdx.x);
            }
        __syncthreads();   // (the maxima are not needed any more: the keys take their place)
        // the order of the lists is that of the atomics, but keys are distinct, so what is chosen is not
        if (steps == 1 && sh.count <= kFew) {
            // one block: its logits are in registers still
            if (most >= least && most > none) {
#pragma unroll
                for (int i = 0; i < kPerThread; ++i)
                    if (x[i] >= least && x[i] > none)
                        sh.key[0][atomicAdd(&sh.keys, 1)] = key_of(x[i], static_cast<uint32_t>(part0 + mine + place(i)));
            }
            __syncthreads();
            if (warp == 0) {
                if (lane < K) sh.key[0][sh.keys + lane] = sh.kept[lane];
                __syncwarp();
                warp_top(sh.key[0], sh.keys + K, K, sh.chosen, sh.scratch[0], lane);
                if (lane < K) sh.kept[lane] = sh.chosen[lane];
            }
            __syncthreads();
            continue;
        }
        uint64_t *list = sh.key[warp], *best = sh.kept + (1 + warp) * K;
        int count = 0;
        const int sixteens = sh.count;
        for (int b = warp * kBatch; b < sixteens; b += kWarps * kBatch) {
            float y[kPerThread];
            int64_t from = 0;
            int have = 0;
            if (lane < kBatch && b + lane < sixteens) {
                const int which = sh.sixteen[b + lane], thread = which % kBeamThreads;
                const int64_t b0 = part0 + static_cast<int64_t>(which / kBeamThreads) * kBlock;
                const int at = wide ? 4 * thread : thread;
                fetch(b0, at, y);
                finite(y);
                from = b0 + at;
#pragma unroll
                for (int i = 0; i < kPerThread; ++i) have += y[i] >= least && y[i] > none;
            }
            int upto = have;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int n = __shfl_up_sync(~0u, upto, d);
                if (lane >= d) upto += n;
            }
            uint64_t *to = list + count + upto - have;
            if (have > 0) {
#pragma unroll
                for (int i = 0; i < kPerThread; ++i)
                    if (y[i] >= least && y[i] > none) *to++ = key_of(y[i], static_cast<uint32_t>(from + place(i)));
            }
            count += __shfl_sync(~0u, upto, 31);
            __syncwarp();
            if (count > kLong) {   // room for another batch
                warp_top(list, count, K, best, sh.scratch[warp], lane);
                list[lane] = lane < K ? best[lane] : 0;
                count = K;
                __syncwarp();
            }
        }
        warp_top(list, count, K, best, sh.scratch[warp], lane);
        __syncthreads();
        if (warp == 0) {
            warp_top(sh.kept, (kWarps + 1) * K, K, sh.chosen, sh.scratch[0], lane);
            if (lane < K) sh.kept[lane] = sh.chosen[lane];
        }
        __syncthreads();
    }
    // the warps' maxima and sums, in a fixed order
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(~0u, wm, o));
    float ws = m > none ? s * expf(m - wm) : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(~0u, ws, o);
    if (lane == 0) sh.sums[warp] = make_float2(wm, ws);
    __syncthreads();
    const int64_t slot = static_cast<int64_t>(row) * gridDim.y + blockIdx.y;
    if (threadIdx.x < K) keys[slot * K + threadIdx.x] = sh.kept[threadIdx.x];
    if (threadIdx.x == 32) {
        float am = sh.sums[0].x, as = 0.0f;
        for (int w = 1; w < kWarps; ++w) am = fmaxf(am, sh.sums[w].x);
        for (int w = 0; w < kWarps; ++w)
            if (sh.sums[w].y > 0.0f) as += sh.sums[w].y * expf(sh.sums[w].x - am);
        stats[slot] = make_float2(am, as);
    }
}

// One CTA per group: warps take its beams in turn, then the first warp chooses.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps) beam_join_kernel(const BeamArgs g, int chunks, const float2 *stats,
                                                                    const uint64_t *keys) {
    extern __shared__ uint64_t lists[];   // [kJoinWarps][chunks * K]
    __shared__ uint64_t best[kMaxBeams * kMaxBeams];
    __shared__ int64_t score[kMaxBeams * kMaxBeams];   // as integers of the same order
    __shared__ uint64_t taken[kJoinWarps][kMaxBeams];
    __shared__ WarpScratch scratch[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = g.K;
    const int group = blockIdx.x;
    const float none = -__int_as_float(0x7f800000);
    static_assert(kMaxChunks <= 64, "two chunks a lane");
    wait_prior_grid();
    allow_next_grid();
    for (int w = warp; w < g.W; w += kJoinWarps) {
        const int64_t row = static_cast<int64_t>(group) * g.W + w;
        // everything that is read is on its way before any of it is looked at (a beam that is
        // finished or dead has left nothing: what is read in its place is not used)
        const float cum = g.scores[row];
        const uint8_t end = g.finished != nullptr ? g.finished[row] : 0;
        uint64_t *list = lists + static_cast<size_t>(warp) * chunks * K;
        const float2 first = lane < chunks ? __ldcg(stats + row * chunks + lane) : make_float2(none, 0.0f);
        const float2 second = lane + 32 < chunks ? __ldcg(stats + row * chunks + lane + 32) : make_float2(none, 0.0f);
        for (int i = lane; i < chunks * K; i += 32) list[i] = __ldcg(keys + row * chunks * K + i);
        const bool live = fabsf(cum) <= kLargest;
        if (!live || end != 0) {
            for (int j = lane; j < K; j += 32) {
                const bool last = live && j == 0;
                best[w * K + j] = last ? 0xffffffffu - static_cast<uint32_t>(g.eos) : 0;
                score[w * K + j] = last ? order_of(static_cast<double>(cum)) : INT64_MIN;
            }
            __syncwarp();
            continue;
        }
        float m = fmaxf(first.x, second.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        float part = (first.y > 0.0f ? first.y * expf(first.x - m) : 0.0f) + (second.y > 0.0f ? second.y * expf(second.x - m) : 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(~0u, part, o);
        const double lse = static_cast<double>(m) + log_of(part);
        __syncwarp();
        warp_top(list, chunks * K, K, taken[warp], scratch[warp], lane);
        for (int j = lane; j < K; j += 32) {
            const uint64_t k = taken[warp][j];
            best[w * K + j] = k;
            score[w * K + j] =
                k != 0 ? order_of(static_cast<double>(cum) + (static_cast<double>(logit_of(k)) - lse)) : INT64_MIN;
        }
        __syncwarp();
    }
    __syncthreads();
    // The places are in the order of beams, and within a beam of logits, then tokens: the order of
    // its exact scores, also of two that round to one binary64 number.  Of equal scores the lower
    // place is the one with the lower beam.  A candidate's place among the chosen is the number of
    // better ones.
    const int n = g.W * K;
    if (threadIdx.x < K) {   // for places that nothing fills
        const int64_t to = static_cast<int64_t>(group) * K + threadIdx.x;
        int have = 0;
        for (int i = 0; i < n; ++i) have += best[i] != 0;
        if (static_cast<int>(threadIdx.x) >= have) {
            g.tokens[to] = g.parents[to] = -1;
            g.out_scores[to] = none;
            if (g.out_finished != nullptr) g.out_finished[to] = 0;
        }
    }
    for (int i = threadIdx.x; i < n; i += 32 * kJoinWarps) {
        if (best[i] == 0) continue;
        const int64_t mine = score[i];
        int better = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) better += score[j] > mine || (score[j] == mine && j < i);
        if (better >= K) continue;
        const int64_t to = static_cast<int64_t>(group) * K + better;
        const int token = static_cast<int>(token_of(best[i]));
        g.tokens[to] = token;
        g.parents[to] = i / K;
        g.out_scores[to] = static_cast<float>(score_of(mine));
        if (g.out_finished != nullptr) g.out_finished[to] = token == g.eos;
    }
}

int64_t beam_workspace_bytes(int groups, int W, int K, int64_t V) {
    const BeamLayout b = beam_layout(static_cast<int64_t>(groups) * W, V);
    return static_cast<int64_t>(groups) * W * b.chunks * (8 + 8 * static_cast<int64_t>(K));
}

int launch_beam_step(const BeamArgs &a, cudaStream_t stream) {
    const int rows = a.groups * a.W;
    const BeamLayout b = beam_layout(rows, a.V);
    uint64_t *keys = static_cast<uint64_t *>(a.workspace);
    float2 *stats = reinterpret_cast<float2 *>(keys + static_cast<int64_t>(rows) * b.chunks * a.K);
    const int wide = aligned(a.logits, 16) && a.row_stride % 4 == 0;
    static_assert(sizeof(BeamShared) <= 48 * 1024, "shared memory without asking for more");
    const bool overlap = call_options().overlap;
    int st = launch_overlappable(beam_chunk_kernel, dim3(static_cast<unsigned>(rows), static_cast<unsigned>(b.chunks)),
                                 dim3(kBeamThreads), sizeof(BeamShared), stream, overlap, a, b.chunk, wide, stats, keys);
    if (st != Q4_OK) return st;
    const size_t lists = static_cast<size_t>(kJoinWarps) * b.chunks * a.K * sizeof(uint64_t);   // at most 128 KB
    static std::atomic<bool> configured[64];
    st = allow_smem(beam_join_kernel, kJoinWarps * kMaxChunks * kMaxBeams * sizeof(uint64_t), configured);
    if (st != Q4_OK) return st;
    return launch_overlappable(beam_join_kernel, dim3(static_cast<unsigned>(a.groups)), dim3(32 * kJoinWarps), lists,
                               stream, true, a, b.chunks, stats, keys);
}

}  // namespace q4
