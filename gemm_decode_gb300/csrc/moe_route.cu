// moe_route.cu -- the router of a mixture of experts: each token's top-k experts with
// their weights, and the rows grouped by expert.
//
// A warp owns a token.  Its E logits sit in registers (E / 32 per lane; above 256 experts
// some are spilled); each becomes a 32-bit key that orders as the binary32 value does (0:
// never chosen), so a round of the choice is one integer maximum over the warp and one
// minimum over the indices that hold it -- exact, with ties to the lower expert, and without
// a floating-point comparison of rounded scores: softmax and sigmoid rise with the logit, so
// the choice needs them only where a bias is added to the score itself.
//
// The grouped order is a counting sort that keeps the order of the tokens.  A block of
// 512 choices counts them per warp with one match over the warp (the rank inside the
// warp is the number of earlier lanes of the match), then sums the counts of the warps
// before.  With one block (up to 512 choices: decoding) the same launch adds the
// prefix over the experts and is done; with more, each block writes its histogram and a
// second launch adds the histograms of the blocks before it; with more than kDirect blocks,
// whose histograms together every block would have to read, a launch between the two sums
// them once.  No atomics: the order is the same on every run.
//
// Bound: latency (the k dependent rounds of one warp, the block barriers, the later launches);
// with up to kDirect blocks also the histograms, which each of them reads.
// Measured: one token, 8 of 64 experts 3.1 us; 8191 tokens, 8 of 128 experts 16.5 us (20.4
// with blocks of 1024 choices and no logits fetched ahead); 131072 tokens 135 us.
#include "q4_moe.cuh"

namespace q4 {

namespace {

constexpr int kChoices = 512;   // choices (token, place) ranked by one block
// Blocks up to which each adds the histograms of the others itself (every block reads them
// all, so the time grows with the square).  8 of 128 experts, without / with the scan: 257
// blocks 24.0 / 24.9 us, 512 51.8 / 42.3, 2048 320 / 135, 16384 13202 / 1085.
constexpr int kDirect = 256;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// An integer that orders as the float does; 0 for NaN and -inf, which are never chosen.
__device__ __forceinline__ uint32_t choice_key(float sel) {
    if (!(sel > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(sel == 0.0f ? 0.0f : sel);   // -0 equals +0
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// 1 / (1 + exp(-l)) without an exponential that overflows: relative accuracy for any l.
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return (l < 0.0f ? e : 1.0f) / (1.0f + e);
}

// Exclusive prefix over v[0..E) held by thread e, E <= blockDim.x; sums: 33 ints of shared
// memory.  Returns the prefix of thread e; *total receives the sum of all.
__device__ __forceinline__ int block_prefix(int v, int *sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += n;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int w = lane < warps ? sums[lane] : 0;
        int winc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(~0u, winc, o);
            if (lane >= o) winc += n;
        }
        sums[lane] = winc - w;
        if (lane == 31) sums[32] = winc;
    }
    __syncthreads();
    *total = sums[32];
    return sums[warp] + inc - v;
}

}  // namespace

// One block: the choices of tokens [blockIdx.x * per_block, ...).  NV: logits per lane;
// ON_SCORE: the choice is by score + bias.
template <int NV, bool ON_SCORE>
__global__ void __launch_bounds__(kMaxExperts) route_choose_kernel(const RouteArgs a, int per_block, int single) {
    extern __shared__ unsigned char route_smem[];
    int *chosen = reinterpret_cast<int *>(route_smem);                     // [kChoices]
    int *base = chosen + kChoices;                                         // [E] first row of an expert (single)
    int *sums = base + a.E;                                                // [33]
    uint8_t *count = reinterpret_cast<uint8_t *>(sums + 33);               // [warps][E], at most 32 each
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int t0 = blockIdx.x * per_block;
    const int tokens = min(per_block, a.T - t0);
    const int choices = tokens * a.k;
    auto ib = [&](bool ok) { return q4_in_bounds(ok, a.bounds); };   // bounds-checking builds
    const int64_t all_choices = static_cast<int64_t>(a.T) * a.k;

    for (int i = threadIdx.x; i < warps * a.E; i += blockDim.x) count[i] = 0;
    wait_prior_grid();
    allow_next_grid();
    // the logits of the warp's next token are on their way while this one's are ranked
    float ahead[NV];
    bool ahead_live = false;
    auto fetch = [&](int i) {
        if (i >= tokens) return;
        const int t = t0 + i;
        if (!ib(t >= 0 && t < a.T)) return;
        ahead_live = a.mask == nullptr || a.mask[t] != 0;
        const float *l = a.logits + static_cast<int64_t>(t) * a.E;
#pragma unroll
        for (int c = 0; c < NV; ++c) ahead[c] = c * 32 + lane < a.E ? l[c * 32 + lane] : -INFINITY;
    };
    fetch(warp);
    for (int i = warp; i < tokens; i += warps) {
        const int t = t0 + i;
        const int64_t at = static_cast<int64_t>(t) * a.k;
        const bool live = ahead_live;
        float v[NV];
#pragma unroll
        for (int c = 0; c < NV; ++c) v[c] = ahead[c] == ahead[c] ? ahead[c] : -INFINITY;   // NaN counts as -inf
        fetch(i + warps);
        int mine = -1;   // lane j: the token's j-th choice
        float m_all = -INFINITY, s_all = 0.0f;
        if (live) {
            if (!a.sigmoid && (!a.renorm || ON_SCORE)) {
#pragma unroll
                for (int c = 0; c < NV; ++c) m_all = fmaxf(m_all, v[c]);
                m_all = warp_max(m_all);
#pragma unroll
                for (int c = 0; c < NV; ++c)
                    if (v[c] > -INFINITY) s_all += expf(v[c] - m_all);
                s_all = warp_sum(s_all);
            }
            if constexpr (ON_SCORE) {
#pragma unroll
                for (int c = 0; c < NV; ++c)   // (an expert whose logit is -inf stays out, whatever its bias)
                    if (v[c] > -INFINITY)
                        v[c] = a.sigmoid ? sigmoid(v[c]) : expf(v[c] - m_all) / s_all;
            }
            uint32_t key[NV], best = 0;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                const int e = c * 32 + lane;
                const float b = a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
                key[c] = choice_key(a.bias != nullptr ? v[c] + b : v[c]);
                best = max(best, key[c]);
            }
            for (int j = 0; j < a.k; ++j) {
                const uint32_t top = __reduce_max_sync(~0u, best);
                if (top == 0u) break;
                unsigned cand = 0xFFFFFFFFu;
                if (best == top) {
#pragma unroll
                    for (int c = NV - 1; c >= 0; --c)
                        if (key[c] == top) cand = c * 32 + lane;
                }
                const int e = static_cast<int>(__reduce_min_sync(~0u, cand));
                if (lane == j) mine = e;
                if ((e & 31) == lane) {
                    best = 0;
#pragma unroll
                    for (int c = 0; c < NV; ++c) {
                        if (c == (e >> 5)) key[c] = 0u;
                        best = max(best, key[c]);
                    }
                }
            }
        }
        float w = 0.0f;
        const float l = mine >= 0 ? a.logits[static_cast<int64_t>(t) * a.E + mine] : -INFINITY;
        if (a.sigmoid) {
            w = mine >= 0 ? sigmoid(l) : 0.0f;
            if (a.renorm) w = w / (warp_sum(w) + 1e-20f);
        } else {
            const float m = a.renorm ? warp_max(l) : m_all;
            w = mine >= 0 && l > -INFINITY ? expf(l - m) : 0.0f;
            w = w / (a.renorm ? warp_sum(w) : s_all);
        }
        if (lane < a.k && ib(at + lane < all_choices && i * a.k + lane < kChoices && mine < a.E)) {
            a.ids[at + lane] = mine;
            a.weights[at + lane] = mine >= 0 ? w * a.scale : 0.0f;
            chosen[i * a.k + lane] = mine;
        }
    }
    __syncthreads();
    // rank of each choice among the block's choices of the same expert
    const int i = threadIdx.x;
    const int e = i < choices ? chosen[i] : -1;
    const unsigned same = __match_any_sync(~0u, e);
    int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0 && ib(warp < warps && e < a.E)) count[warp * a.E + e] = static_cast<uint8_t>(__popc(same));
    __syncthreads();
    if (e >= 0)
        for (int w = 0; w < warp; ++w) rank += count[w * a.E + e];
    int total = 0;
    if (i < a.E)
        for (int w = 0; w < warps; ++w) total += count[w * a.E + i];
    if (single) {
        int all;
        const int first = block_prefix(i < a.E ? total : 0, sums, &all);
        if (i < a.E) {
            base[i] = first;
            a.offsets[i] = first;
        }
        if (i == 0) a.offsets[a.E] = all;
        __syncthreads();
        if (i < choices) {
            const int row = e >= 0 ? base[e] + rank : -1;
            a.pos[i] = row;
            if (row >= 0 && ib(row < all_choices)) a.rows[row] = i / a.k;
            if (i >= all && ib(i < all_choices)) a.rows[i] = -1;
        }
    } else {
        if (i < a.E) a.hist[static_cast<int64_t>(blockIdx.x) * a.E + i] = total;
        if (i < choices && ib(static_cast<int64_t>(t0) * a.k + i < all_choices))
            a.pos[static_cast<int64_t>(t0) * a.k + i] = e >= 0 ? rank : -1;
    }
}

// Histograms [blocks][E] to exclusive prefixes over the blocks, in place, and the totals of
// the experts behind them.  A block takes 32 experts, a warp a 32nd of the blocks.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteArgs a, int blocks) {
    __shared__ int part[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    const int each = (blocks + 31) / 32, b0 = warp * each, b1 = min(b0 + each, blocks);
    wait_prior_grid();
    allow_next_grid();
    int sum = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += a.hist[static_cast<int64_t>(b) * a.E + e];
    }
    part[warp][lane] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += part[w][lane];
    if (e >= a.E) return;
    if (warp == 31) a.hist[static_cast<int64_t>(blocks) * a.E + e] = before + sum;
    for (int b = b0; b < b1; b += 8) {   // eight loads in flight together
        int h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = b + i < b1 ? a.hist[static_cast<int64_t>(b + i) * a.E + e] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (b + i < b1) a.hist[static_cast<int64_t>(b + i) * a.E + e] = before;
            before += h[i];
        }
    }
}

// The last launch of a long prompt: first row of each expert for this block (all choices
// of lower experts, and this expert's choices in the blocks before), then the rows.
// scanned: the histograms are prefixes already.
__global__ void __launch_bounds__(1024) route_place_kernel(const RouteArgs a, int per_block, int scanned) {
    __shared__ int part_all[1024], part_before[1024], base[kMaxExperts], sums[33];
    int width = 32;
    while (width < a.E) width <<= 1;            // <= 1024: threads of one slice of the blocks
    const int slices = 1024 / width;
    const int e = threadIdx.x & (width - 1), slice = threadIdx.x / width;
    wait_prior_grid();
    allow_next_grid();
    int all = 0, before = 0;
    if (scanned) {
        if (slice == 0 && e < a.E) {
            all = a.hist[static_cast<int64_t>(gridDim.x) * a.E + e];
            before = a.hist[static_cast<int64_t>(blockIdx.x) * a.E + e];
        }
    } else if (e < a.E) {
#pragma unroll 8
        for (int b = slice; b < static_cast<int>(gridDim.x); b += slices) {
            const int h = a.hist[static_cast<int64_t>(b) * a.E + e];
            all += h;
            if (b < static_cast<int>(blockIdx.x)) before += h;
        }
    }
    part_all[threadIdx.x] = all;
    part_before[threadIdx.x] = before;
    __syncthreads();
    all = before = 0;
    if (threadIdx.x < a.E) {
        for (int s = 0; s < slices; ++s) {
            all += part_all[s * width + threadIdx.x];
            before += part_before[s * width + threadIdx.x];
        }
    }
    int total;
    const int first = block_prefix(threadIdx.x < a.E ? all : 0, sums, &total);
    if (threadIdx.x < a.E) {
        base[threadIdx.x] = first + before;
        if (blockIdx.x == 0) a.offsets[threadIdx.x] = first;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = total;
    __syncthreads();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * per_block * a.k + threadIdx.x;
    const bool mine = threadIdx.x < per_block * a.k && at < static_cast<int64_t>(a.T) * a.k;
    if (mine) {
        const int id = a.ids[at];
        if (id >= 0 && q4_in_bounds(id < a.E, a.bounds)) {
            const int row = base[id] + a.pos[at];
            a.pos[at] = row;
            if (q4_in_bounds(row >= 0 && row < total, a.bounds)) a.rows[row] = static_cast<int>(at / a.k);
        }
        if (at >= total) a.rows[at] = -1;
    }
}

static int route_per_block(int k) { return kChoices / k; }
static int route_blocks(int T, int k) {
    const int per = route_per_block(k);
    return T / per + (T % per != 0);
}

int64_t route_workspace_bytes(int T, int E, int k) {
    const int blocks = route_blocks(T, k);
    return blocks > 1 ? (static_cast<int64_t>(blocks) + (blocks > kDirect)) * E * 4 : 0;
}

template <int NV>
static int launch_choose(const RouteArgs &a, int blocks, int threads, int per, cudaStream_t stream) {
    const size_t smem = 4 * (kChoices + a.E + 33) + static_cast<size_t>(threads / 32) * a.E;
    return launch_overlappable(a.score_bias && a.bias != nullptr ? route_choose_kernel<NV, true> : route_choose_kernel<NV, false>,
                               dim3(blocks), dim3(threads), smem, stream, call_options().overlap, a, per,
                               blocks == 1 ? 1 : 0);
}

int launch_route(const RouteArgs &a, cudaStream_t stream) {
    const int per = route_per_block(a.k);
    const int blocks = route_blocks(a.T, a.k);
    // a thread per choice and per expert of the block
    const int choices = blocks > 1 ? kChoices : a.T * a.k, need = choices > a.E ? choices : a.E;
    const int threads = need <= 128 ? 128 : (need + 31) / 32 * 32;
    int st;
    if (a.E <= 32) st = launch_choose<1>(a, blocks, threads, per, stream);
    else if (a.E <= 64) st = launch_choose<2>(a, blocks, threads, per, stream);
    else if (a.E <= 128) st = launch_choose<4>(a, blocks, threads, per, stream);
    else if (a.E <= 256) st = launch_choose<8>(a, blocks, threads, per, stream);
    else if (a.E <= 512) st = launch_choose<16>(a, blocks, threads, per, stream);
    else st = launch_choose<32>(a, blocks, threads, per, stream);
    if (st != Q4_OK || blocks == 1) return st;
    const bool scan = blocks > kDirect;
    if (scan)
        st = launch_overlappable(route_scan_kernel, dim3((a.E + 31) / 32), dim3(1024), 0, stream, true, a, blocks);
    if (st != Q4_OK) return st;
    return launch_overlappable(route_place_kernel, dim3(blocks), dim3(1024), 0, stream, true, a, per, scan ? 1 : 0);
}

}  // namespace q4
