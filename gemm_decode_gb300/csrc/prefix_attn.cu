// prefix_attn.cu -- attention over a shared and an own segment of the paged cache: the plan of
// a call, the joining of the parts, and the launches.  The kernels that multiply are in
// attn_few.cuh and attn_many.cuh, the division of the work in attn_common.cuh.
//
//   plan     one CTA reads the lengths and lists the segments of both kinds, units numbered
//            through by prefix sums
//   many     segments of more than 16 rows, on the tensor cores (left out where the sizes of
//            the call allow none)
//   few      the others (likewise)
//   join     adds the parts of each row, where several kernels or CTAs have one
#include <algorithm>
#include <atomic>

#include "attn_few.cuh"
#include "attn_many.cuh"

namespace q4 {

// The status word of the bounded waits (q4gemm.cu).
unsigned int *gemm_status_word();

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kJoinThreads = 256;

// Inclusive sums of a and b over the block, in place; the totals in ta and tb.
__device__ __forceinline__ void block_scan(int64_t &a, int &b, int64_t &ta, int &tb, int64_t *sa, int *sb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t na = __shfl_up_sync(~0u, a, o);
        const int nb = __shfl_up_sync(~0u, b, o);
        if (lane >= o) a += na, b += nb;
    }
    __syncthreads();   // (sa and sb may still be read from the call before)
    if (lane == 31) sa[warp] = a, sb[warp] = b;
    __syncthreads();
    int64_t wa = sa[lane];
    int wb = sb[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t na = __shfl_up_sync(~0u, wa, o);
        const int nb = __shfl_up_sync(~0u, wb, o);
        if (lane >= o) wa += na, wb += nb;
    }
    ta = __shfl_sync(~0u, wa, 31);
    tb = __shfl_sync(~0u, wb, 31);
    if (warp > 0) {
        a += __shfl_sync(~0u, wa, warp - 1);
        b += __shfl_sync(~0u, wb, warp - 1);
    }
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const AttnArgs g) {
    static_assert(kPlanThreads == 1024, "block_scan: 32 warps");
    __shared__ int64_t sa[32];
    __shared__ int sb[32];
    const int t = threadIdx.x;
    wait_prior_grid();
    allow_next_grid();
    const int run = kManyTiles * g.tile_queries;   // queries of an entry of the kernel for many rows
    auto few_group = [&](int n) { return n * g.G <= kFewRows; };
    // ---- groups: offsets in order, and the first run of each
    int carry_off = 0, carry_runs = 0;
    for (int g0 = 0; g0 <= g.groups; g0 += kPlanThreads) {
        const int i = g0 + t;
        int off = 0;
        if (i <= g.groups) off = g.group_offsets != nullptr ? min(max(g.group_offsets[i], 0), g.S) : (i == 0 ? 0 : g.S);
        off = max(off, carry_off);
        // running maximum over the block
        {
            const int lane = t & 31, warp = t >> 5;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(~0u, off, o);
                if (lane >= o) off = max(off, n);
            }
            __syncthreads();
            if (lane == 31) sb[warp] = off;
            __syncthreads();
            int w = sb[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(~0u, w, o);
                if (lane >= o) w = max(w, n);
            }
            carry_off = __shfl_sync(~0u, w, 31);
            const int before = __shfl_sync(~0u, w, max(warp - 1, 0));
            if (warp > 0) off = max(off, before);
        }
        if (i <= g.groups) g.first_of[i] = off;
        __syncthreads();   // the next group's offset is written
        int runs = 0;
        if (i > 0 && i <= g.groups) {
            const int n = off - g.first_of[i - 1];
            runs = few_group(n) ? 0 : (n + run - 1) / run;
        }
        // place i holds the runs of group i - 1, so its inclusive sum is the first run of group i
        int64_t dummy = 0, td;
        int tr;
        block_scan(dummy, runs, td, tr, sa, sb);
        if (i <= g.groups) g.tile_of[i] = carry_runs + runs;
        carry_runs += tr;
    }
    const int all_runs = carry_runs;
    __syncthreads();
    // ---- the most keys a run of queries sees
    for (int i = t; i < all_runs; i += kPlanThreads) g.run_keys[i] = 0;
    __syncthreads();
    auto group_of = [&](int s) {   // the group with first_of[g] <= s < first_of[g + 1], or -1
        if (g.groups == 0 || s < g.first_of[0] || s >= g.first_of[g.groups]) return -1;
        int lo = 0, hi = g.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (g.first_of[mid] <= s) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    auto keys_seen = [&](int group, int s) {
        const int n = clamp_len(g.shared_lens[group], g.max_shared, g.page);
        return g.limits != nullptr ? max(0, min(n, g.limits[s])) : n;
    };
    for (int s = t; s < g.S; s += kPlanThreads) {
        const int group = group_of(s);
        int of = -1;
        if (group >= 0) {
            const int first = g.first_of[group];
            if (few_group(g.first_of[group + 1] - first)) {
                of = -2 - group;   // for now: the group
            } else {
                const int r = g.tile_of[group] + (s - first) / run;
                of = r;
                if (g.limits != nullptr || (s - first) % run == 0) atomicMax(g.run_keys + r, keys_seen(group, s));
            }
        }
        g.shared_of[s] = of;
        g.own_of[s] = -1;
    }
    __syncthreads();
    // ---- entries of many rows: runs with keys
    int64_t units0 = 0;
    int entries0 = 0;
    for (int r0 = 0; r0 < all_runs; r0 += kPlanThreads) {
        const int r = r0 + t;
        const int keys = r < all_runs ? __ldcg(g.run_keys + r) : 0;
        const int64_t mine = static_cast<int64_t>((keys + kManyKeys - 1) / kManyKeys) * g.Hkv;
        int64_t u = mine, tu;
        int e = keys > 0 ? 1 : 0, te;
        block_scan(u, e, tu, te, sa, sb);
        if (r < all_runs) {
            const int at = entries0 + e - 1;
            g.run_entry[r] = keys > 0 ? at : -1;
            if (keys > 0) {
                int lo = 0, hi = g.groups;   // the group with tile_of[g] <= r < tile_of[g + 1]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (g.tile_of[mid] <= r) lo = mid;
                    else hi = mid;
                }
                const int first = g.first_of[lo] + (r - g.tile_of[lo]) * run;
                g.many_entries[at] = AttnEntry{first, min(run, g.first_of[lo + 1] - first), lo, keys};
                g.many_start[at] = units0 + u - mine;
            }
        }
        units0 += tu;
        entries0 += te;
    }
    if (t == 0) *g.many = AttnCounts{units0, entries0, 0};
    // ---- entries of few rows: own segments, then small groups
    const bool own = g.own_lens != nullptr;
    const int places = (own ? g.S : 0) + g.groups;
    int64_t units1 = 0;
    int entries1 = 0;
    for (int p0 = 0; p0 < places; p0 += kPlanThreads) {
        const int p = p0 + t;
        AttnEntry a = {0, 0, -1, 0};
        if (p < places) {
            if (own && p < g.S) {
                a = AttnEntry{p, 1, -1, clamp_len(g.own_lens[p], g.max_own, g.page)};
            } else {
                const int group = p - (own ? g.S : 0), first = g.first_of[group], n = g.first_of[group + 1] - first;
                if (n > 0 && few_group(n)) {
                    int keys = 0;
                    for (int s = first; s < first + n; ++s) keys = max(keys, keys_seen(group, s));
                    a = AttnEntry{first, n, group, keys};
                }
            }
        }
        const int tiles = (a.queries * g.G + kFewRows - 1) / kFewRows;
        const int64_t mine = static_cast<int64_t>((a.keys + kFewKeys - 1) / kFewKeys) * g.Hkv * tiles;
        int64_t u = mine, tu;
        int e = a.keys > 0 ? 1 : 0, te;
        block_scan(u, e, tu, te, sa, sb);
        if (a.keys > 0) {
            const int at = entries1 + e - 1;
            g.few_entries[at] = a;
            g.few_start[at] = units1 + u - mine;
            if (a.group < 0) g.own_of[a.first] = at;
            else g.tile_of[a.group] = at;   // (a small group has no runs: its place is free)
        } else if (p < places && a.group >= 0) {
            g.tile_of[a.group] = -1;
        }
        units1 += tu;
        entries1 += te;
    }
    if (t == 0) *g.few = AttnCounts{units1, entries1, 0};
    __syncthreads();
    // ---- each query's entries
    if (g.groups > 0)
        for (int s = t; s < g.S; s += kPlanThreads) {
            int of = g.shared_of[s];
            if (of >= 0) of = g.run_entry[of];
            else if (of <= -2) of = g.tile_of[-2 - of] >= 0 ? -2 - g.tile_of[-2 - of] : -1;
            g.shared_of[s] = of;
        }
}

// Where the parts of a row of one segment are.
struct AttnParts {
    int count;             // 0: none
    const float *at;       // the first part's row
    const float2 *stats;
    int64_t step;          // rows from a part to the next (but from the first to the second)
    int64_t second;        // rows from the first to the second
    bool final;            // already in the output
};

__device__ __forceinline__ AttnParts parts_of(const AttnArgs &g, bool many, int entry, int s, int head, int kind) {
    AttnParts p = {};
    const AttnEntry e = many ? g.many_entries[entry] : g.few_entries[entry];
    const AttnCounts n = many ? *g.many : *g.few;
    const int ctas = ctas_of(n.units, many ? g.many_ctas : g.few_ctas);
    const int keys = many ? kManyKeys : kFewKeys;
    const int units = (e.keys + keys - 1) / keys;
    const int kv = head / g.G, row = (s - e.first) * g.G + (head - kv * g.G);
    int seg = kv, at_row = row, rows;
    if (many) {
        rows = 128 * kManyTiles;
        const int per = g.tile_queries * g.G;
        at_row = row / per * 128 + row % per;
    } else {
        rows = kFewRows;
        const int tiles = (e.queries * g.G + kFewRows - 1) / kFewRows;
        seg = kv * tiles + row / kFewRows;
        at_row = row % kFewRows;
    }
    const int64_t u0 = (many ? g.many_start[entry] : g.few_start[entry]) + static_cast<int64_t>(seg) * units;
    const int c0 = owner_of(n.units, ctas, u0), c1 = owner_of(n.units, ctas, u0 + units - 1);
    p.count = c1 - c0 + 1;
    p.final = p.count == 1 && g.alone;
    const float *part = many ? g.many_part : g.few_part;
    const float2 *stats = many ? g.many_stats : g.few_stats;
    int64_t at;
    if (p.count == 1) {
        part = g.whole[kind];
        stats = g.whole_stats[kind];
        at = static_cast<int64_t>(s) * g.Hq + head;
    } else {
        at = static_cast<int64_t>(2 * c0 + 1) * rows + at_row;   // the first CTA's second slot, then first slots
        p.second = rows;
        p.step = 2 * rows;
    }
    p.at = part + at * g.D;
    p.stats = stats + at;
    return p;
}

// A warp takes `each` rows (query, query head): which of them have parts to join is looked at
// a lane each, then the warp joins one after another.
template <typename C, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs g, int each) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(g.S) * g.Hq;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5)) * each;
    wait_prior_grid();
    allow_next_grid();
    AttnParts a = {}, b = {};   // shared, own
    bool todo = false;
    if (lane < each && first + lane < rows) {
        const int s = static_cast<int>((first + lane) / g.Hq), head = static_cast<int>((first + lane) - static_cast<int64_t>(s) * g.Hq);
        const int of = g.groups > 0 ? g.shared_of[s] : -1, own = g.own_lens != nullptr ? g.own_of[s] : -1;
        if (of != -1) a = parts_of(g, of >= 0, of >= 0 ? of : -2 - of, s, head, 0);
        if (own >= 0) b = parts_of(g, false, own, s, head, 1);
        todo = !(a.final || b.final);
    }
    unsigned left = __ballot_sync(~0u, todo);
    while (left != 0) {
        const int from = __ffs(left) - 1;
        left &= left - 1;
        const int64_t row = first + from;
        float o[V], m = neg_inf(), l = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
        auto add = [&](const AttnParts &mine) {
            const int count = __shfl_sync(~0u, mine.count, from);
            const float *at = reinterpret_cast<const float *>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(mine.at), from));
            const float2 *stats =
                reinterpret_cast<const float2 *>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(mine.stats), from));
            const int64_t step = __shfl_sync(~0u, mine.step, from), second = __shfl_sync(~0u, mine.second, from);
            for (int c0 = 0; c0 < count; c0 += 32) {
                const int n = min(32, count - c0);
                // a part a lane: its maximum and sum, then its weight among these
                const int c = c0 + lane;
                const int64_t place = c == 0 ? 0 : c * step - step + second;
                float2 st = make_float2(neg_inf(), 0.0f);
                if (lane < n) st = __ldcg(stats + place);
                float top = st.x;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const float nm = fmaxf(m, top), base = nm == neg_inf() ? 0.0f : nm;
                const float old = exp2_fast(m - base), w = exp2_fast(st.x - base);
                float sum = st.y * w;
                if (lane >= n) sum = 0.0f;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
                m = nm;
                l = l * old + sum;
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] *= old;
#pragma unroll 4
                for (int j = 0; j < n; ++j) {
                    const float f = __shfl_sync(~0u, w, j);
                    const int cj = c0 + j;
                    const float *src = at + (cj == 0 ? 0 : cj * step - step + second) * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                        o[0] = fmaf(f, v.x, o[0]), o[1] = fmaf(f, v.y, o[1]);
                        o[2] = fmaf(f, v.z, o[2]), o[3] = fmaf(f, v.w, o[3]);
                    } else {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                        o[0] = fmaf(f, v.x, o[0]), o[1] = fmaf(f, v.y, o[1]);
                    }
                }
            }
        };
        add(a);
        add(b);
        const float r = l != 0.0f ? 1.0f / l : 0.0f;   // (no key: zeros)
        if (!q4_in_bounds(row < rows, g.bounds)) continue;
        if (lane == 0 && g.lse != nullptr) g.lse[row] = lse_of(m, l);
        const int64_t to = row * D + lane * V;
        if (g.out_f32) {
            float *p = static_cast<float *>(g.out) + to;
#pragma unroll
            for (int i = 0; i < V; i += 2) *reinterpret_cast<float2 *>(p + i) = make_float2(o[i] * r, o[i + 1] * r);
        } else {
            uint32_t *p = reinterpret_cast<uint32_t *>(static_cast<C *>(g.out) + to);
#pragma unroll
            for (int i = 0; i < V; i += 2) p[i / 2] = pack2<C>(o[i] * r, o[i + 1] * r);
        }
    }
}

namespace {

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

int tile_queries_of(int G) { return 128 / G; }
bool many_possible(int64_t S, int groups, int G) { return groups > 0 && S * G > kFewRows; }

// Places in the workspace.
struct Layout {
    int64_t counts, many_entries, few_entries, many_start, few_start, shared_of, own_of, first_of, tile_of, run_keys,
        run_entry, many_part, few_part, many_stats, few_stats, whole[2], whole_stats[2], total;
    int many_ctas, few_ctas;
};
Layout layout_of(int S, int groups, int Hq, int Hkv, int D) {
    const int G = Hq / Hkv, sms = device_info().sms;
    Layout l;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t p = at;
        at += round256(bytes);
        return p;
    };
    const bool many = many_possible(S, groups, G);
    l.many_ctas = many ? sms : 0;
    l.few_ctas = 2 * sms;
    const int64_t runs = many ? groups + static_cast<int64_t>(S) / (kManyTiles * tile_queries_of(G)) : 0;
    l.counts = take(2 * sizeof(AttnCounts));
    l.many_entries = take(runs * sizeof(AttnEntry));
    l.few_entries = take((static_cast<int64_t>(S) + groups) * sizeof(AttnEntry));
    l.many_start = take(runs * 8);
    l.few_start = take((static_cast<int64_t>(S) + groups) * 8);
    l.shared_of = take(4ll * S);
    l.own_of = take(4ll * S);
    l.first_of = take(4ll * (groups + 1));
    l.tile_of = take(4ll * (groups + 1));
    l.run_keys = take(4 * runs);
    l.run_entry = take(4 * runs);
    const int64_t mrows = 2ll * l.many_ctas * 128 * kManyTiles, frows = 2ll * l.few_ctas * kFewRows;
    l.many_part = take(mrows * D * 4);
    l.many_stats = take(mrows * 8);
    l.few_part = take(frows * D * 4);
    l.few_stats = take(frows * 8);
    for (int i = 0; i < 2; ++i) {
        const int64_t rows = groups > 0 ? static_cast<int64_t>(S) * Hq : 0;
        l.whole[i] = take(rows * D * 4);
        l.whole_stats[i] = take(rows * 8);
    }
    l.total = at;
    return l;
}

// A tensor map of rows of 64 features (128-byte swizzle).
bool encode(CUtensorMap *map, int dtype, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return enc(map, dtype == Q4_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename C, int D>
int launch_attn(const q4_prefix_attn_t &a, const AttnArgs &g, cudaStream_t stream) {
    const q4_kv_cache_t &c = a.cache;
    // (a stride that nothing steps over still has to be one that a map takes)
    auto bytes = [&](int64_t stride, int64_t count) { return static_cast<cuuint64_t>(count > 1 ? 2 * stride : 2 * D); };
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(c.page),
                                static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[3] = {bytes(c.row_stride, c.page), bytes(c.head_stride, c.heads),
                                   bytes(c.page_stride, c.pages)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(g.box), 1, 1};
    CUtensorMap map_k, map_v, map_q;
    if (!encode(&map_k, c.dtype, c.k, 4, dims, strides, box) || !encode(&map_v, c.dtype, c.v, 4, dims, strides, box))
        return Q4_ERR_UNSUPPORTED;
    int st = launch_overlappable(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, call_options().overlap, g);
    if (st != Q4_OK) return st;
    if (g.many_ctas > 0) {
        using M = ManyAttn<D>;
        static_assert(M::smem() <= 227 * 1024, "shared memory of one CTA");
        static std::atomic<bool> configured[64];
        if ((st = allow_smem(attn_many_kernel<C, D>, M::smem(), configured)) != Q4_OK) return st;
        const cuuint64_t qd[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.S)};
        const cuuint64_t qs[2] = {2 * D, bytes(a.q_stride, a.S)};
        const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(g.G), static_cast<cuuint32_t>(g.tile_queries)};
        if (!encode(&map_q, c.dtype, a.q, 3, qd, qs, qb)) return Q4_ERR_UNSUPPORTED;
        st = launch_overlappable(attn_many_kernel<C, D>, dim3(static_cast<unsigned>(g.many_ctas)), dim3(M::kThreads),
                                 M::smem(), stream, true, map_q, map_k, map_v, g);
        if (st != Q4_OK) return st;
    }
    // (no own segments and one group: all its queries have more than 16 rows, or all are few)
    if (a.own_lens != nullptr || g.many_ctas == 0 || a.groups > 1 || a.group_offsets != nullptr) {
        using F = FewAttn<D>;
        static_assert(2 * (F::smem() + 1024) <= 228 * 1024, "two CTAs of an SM");
        static std::atomic<bool> configured[64];
        if ((st = allow_smem(attn_few_kernel<C, D>, F::smem(), configured)) != Q4_OK) return st;
        st = launch_overlappable(attn_few_kernel<C, D>, dim3(static_cast<unsigned>(g.few_ctas)), dim3(F::kThreads),
                                 F::smem(), stream, true, map_k, map_v, g);
        if (st != Q4_OK) return st;
    }
    // rows of a warp: one where there are few, so that the parts are read by many warps
    const int64_t rows = static_cast<int64_t>(a.S) * a.Hq;
    const int each = static_cast<int>(std::min<int64_t>(32, std::max<int64_t>(1, rows / (64 * device_info().sms))));
    const int64_t per = static_cast<int64_t>(each) * (kJoinThreads / 32);
    return launch_overlappable(attn_join_kernel<C, D>, dim3(static_cast<unsigned>((rows + per - 1) / per)),
                               dim3(kJoinThreads), 0, stream, true, g, each);
}

int shift_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

}  // namespace

int64_t prefix_attn_workspace_bytes(int S, int groups, int Hq, int Hkv, int D) {
    return layout_of(S, groups, Hq, Hkv, D).total;
}

int launch_prefix_attn(const q4_prefix_attn_t &a, cudaStream_t stream) {
    const q4_kv_cache_t &c = a.cache;
    const Layout l = layout_of(a.S, a.groups, a.Hq, c.heads, c.D);
    unsigned char *w = static_cast<unsigned char *>(a.workspace);
    AttnArgs g = {};
    g.S = a.S;
    g.Hq = a.Hq;
    g.Hkv = c.heads;
    g.G = a.Hq / c.heads;
    g.groups = a.groups;
    g.D = c.D;
    g.page = c.page;
    g.page_shift = shift_of(c.page);
    g.pages = static_cast<int>(c.pages);
    g.box = std::min(c.page, 64);
    g.box_shift = shift_of(g.box);
    g.max_shared = a.max_shared_pages;
    g.max_own = a.max_own_pages;
    g.tile_queries = tile_queries_of(g.G);
    g.out_f32 = a.out_dtype == Q4_F32;
    g.alone = a.groups == 0 || a.own_lens == nullptr;
    // (times 0: so small that every score counts as 0, but a masked one, -inf, stays)
    g.scale2 = a.scale != 0.0f ? a.scale * 1.44269504088896341f : 1e-30f;
    g.q = a.q;
    g.q_stride = a.q_stride;
    g.group_offsets = a.group_offsets;
    g.shared_pages = a.shared_pages;
    g.shared_lens = a.shared_lens;
    g.limits = a.limits;
    g.own_pages = a.own_pages;
    g.own_lens = a.own_lens;
    g.out = a.out;
    g.lse = a.lse;
    g.many = reinterpret_cast<AttnCounts *>(w + l.counts);
    g.few = g.many + 1;
    g.many_entries = reinterpret_cast<AttnEntry *>(w + l.many_entries);
    g.few_entries = reinterpret_cast<AttnEntry *>(w + l.few_entries);
    g.many_start = reinterpret_cast<int64_t *>(w + l.many_start);
    g.few_start = reinterpret_cast<int64_t *>(w + l.few_start);
    g.shared_of = reinterpret_cast<int *>(w + l.shared_of);
    g.own_of = reinterpret_cast<int *>(w + l.own_of);
    g.first_of = reinterpret_cast<int *>(w + l.first_of);
    g.tile_of = reinterpret_cast<int *>(w + l.tile_of);
    g.run_keys = reinterpret_cast<int *>(w + l.run_keys);
    g.run_entry = reinterpret_cast<int *>(w + l.run_entry);
    g.many_ctas = l.many_ctas;
    g.few_ctas = l.few_ctas;
    g.many_part = reinterpret_cast<float *>(w + l.many_part);
    g.many_stats = reinterpret_cast<float2 *>(w + l.many_stats);
    g.few_part = reinterpret_cast<float *>(w + l.few_part);
    g.few_stats = reinterpret_cast<float2 *>(w + l.few_stats);
    for (int i = 0; i < 2; ++i) {
        g.whole[i] = reinterpret_cast<float *>(w + l.whole[i]);
        g.whole_stats[i] = reinterpret_cast<float2 *>(w + l.whole_stats[i]);
    }
    g.timeout_ns = call_options().wait_ns;
    g.status = gemm_status_word();
    g.bounds = bounds_counter();
    if (g.status == nullptr) return Q4_ERR_CUDA;
    const bool half_type = c.dtype == Q4_F16;
    if (c.D == 64)
        return half_type ? launch_attn<__half, 64>(a, g, stream) : launch_attn<__nv_bfloat16, 64>(a, g, stream);
    return half_type ? launch_attn<__half, 128>(a, g, stream) : launch_attn<__nv_bfloat16, 128>(a, g, stream);
}

}  // namespace q4
