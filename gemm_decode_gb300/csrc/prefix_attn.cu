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
//
// The four are launched overlapped, and the kernels for many and few rows run side by side (256
// sequences: 162 us one after the other, 157-160 so).  Four beams of a prompt of 1000 tokens take
// 16 us, most of it latency: the plan 3-4 us (13 us for a prompt of 4096 queries with a limit
// each before its tables lay in shared memory and its records were those that are read), the
// join 5.
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
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t na = __shfl_up_sync(~0u, a, o);
        const int nb = __shfl_up_sync(~0u, b, o);
        if (lane >= o) a += na, b += nb;
    }
    __syncthreads();   // (sa and sb may still be read from the call before)
    if (lane == 31) sa[warp] = a, sb[warp] = b;
    __syncthreads();
    int64_t wa = lane < warps ? sa[lane] : 0;
    int wb = lane < warps ? sb[lane] : 0;
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

// Inclusive running maximum over the block.
__device__ __forceinline__ int block_max_scan(int v, int &total, int *sb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v = max(v, n);
    }
    __syncthreads();
    if (lane == 31) sb[warp] = v;
    __syncthreads();
    int w = lane < warps ? sb[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w = max(w, n);
    }
    total = __shfl_sync(~0u, w, 31);
    const int before = __shfl_sync(~0u, w, max(warp - 1, 0));
    return warp > 0 ? max(v, before) : v;
}

// The last i of [0, n) with at[i] <= v (at ascending, at[0] <= v).
__device__ __forceinline__ int last_at_most(const int *at, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace

// One CTA.  A run is the queries of one entry of the kernel for many rows; tables of groups and
// runs are in shared memory where they fit.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const AttnArgs g) {
    constexpr int kHeldGroups = 1024, kHeldRuns = 1024;
    __shared__ int64_t sa[32];
    __shared__ int sb[32];
    __shared__ int s_first[kHeldGroups + 1], s_run[kHeldGroups + 1], s_len[kHeldGroups], s_keys[kHeldRuns];
    __shared__ int64_t s_start[kHeldRuns];
    const int t = threadIdx.x, T = blockDim.x;
    const bool own = g.own_lens != nullptr, held = g.groups <= kHeldGroups;
    int *first_of = held ? s_first : g.first_of, *run_of = held ? s_run : g.run_of;
    wait_prior_grid();
    allow_next_grid();
    // what the queries' own segments need is on its way meanwhile
    int own_len = own && t < g.S ? g.own_lens[t] : 0;
    const int run = kManyTiles * g.tile_queries;
    auto few_group = [&](int n) { return n * g.G <= kFewRows; };
    auto group_len = [&](int group) { return held ? s_len[group] : clamp_len(g.shared_lens[group], g.max_shared, g.page); };
    auto keys_seen = [&](int group, int s) {
        const int n = group_len(group);
        return g.limits != nullptr ? max(0, min(n, g.limits[s])) : n;
    };
    // ---- groups: offsets in order, and the first run of each
    int carry_off = 0, all_runs = 0;
    bool any_few = own || g.groups >= 32;   // whether there can be entries of few rows
    if (g.groups > 0 && g.groups < 32) {   // each warp for itself, a place a lane
        const int i = t & 31;
        int off = 0, len = 0;
        if (i <= g.groups) off = g.group_offsets != nullptr ? min(max(g.group_offsets[i], 0), g.S) : (i == 0 ? 0 : g.S);
        if (i < g.groups) len = clamp_len(g.shared_lens[i], g.max_shared, g.page);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(~0u, off, o);
            if (i >= o) off = max(off, n);
        }
        const int n = off - __shfl_up_sync(~0u, off, 1);
        int runs = i > 0 && i <= g.groups && !few_group(n) ? (n + run - 1) / run : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int r = __shfl_up_sync(~0u, runs, o);
            if (i >= o) runs += r;
        }
        all_runs = __shfl_sync(~0u, runs, g.groups);
        any_few |= __any_sync(~0u, i > 0 && i <= g.groups && n > 0 && few_group(n)) != 0;
        if (t <= g.groups) {
            s_first[t] = off;
            s_run[t] = runs;
            if (t < g.groups) s_len[t] = len;
        }
        __syncthreads();
    } else if (g.groups > 0) {
        for (int g0 = 0; g0 <= g.groups; g0 += T) {
            const int i = g0 + t;
            int off = 0;
            if (i <= g.groups)
                off = g.group_offsets != nullptr ? min(max(g.group_offsets[i], 0), g.S) : (i == 0 ? 0 : g.S);
            if (held && i < g.groups) s_len[i] = clamp_len(g.shared_lens[i], g.max_shared, g.page);
            int total;
            off = block_max_scan(max(off, carry_off), total, sb);
            carry_off = total;
            if (i <= g.groups) first_of[i] = off;
            __syncthreads();
            // place i holds the runs of group i - 1, so its inclusive sum is the first run of group i
            int runs = 0, tr;
            if (i > 0 && i <= g.groups) {
                const int n = off - first_of[i - 1];
                runs = few_group(n) ? 0 : (n + run - 1) / run;
            }
            int64_t none = 0, tn;
            block_scan(none, runs, tn, tr, sa, sb);
            if (i <= g.groups) run_of[i] = all_runs + runs;
            all_runs += tr;
        }
        __syncthreads();
    }
    const bool held_runs = held && all_runs <= kHeldRuns;
    int *run_keys = held_runs ? s_keys : g.run_keys;
    int64_t *run_start = held_runs ? s_start : g.run_start;
    // ---- the most keys that a query of a run sees
    if (g.limits != nullptr && all_runs > 0) {
        for (int i = t; i < all_runs; i += T) run_keys[i] = 0;
        __syncthreads();
        // (four limits on their way at a time; a warp's queries are of one run as a rule, and one lane
        // answers for those that are)
        for (int s0 = 0; s0 < g.S; s0 += 4 * T) {
            int seen[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) seen[i] = s0 + i * T + t < g.S ? g.limits[s0 + i * T + t] : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = s0 + i * T + t;
                int r = -1, keys = 0;
                if (s < g.S && s >= first_of[0] && s < first_of[g.groups]) {
                    const int group = last_at_most(first_of, g.groups, s), first = first_of[group];
                    if (!few_group(first_of[group + 1] - first)) {
                        r = run_of[group] + (s - first) / run;
                        keys = max(0, min(group_len(group), seen[i]));
                    }
                }
                if (__reduce_min_sync(~0u, r) == __reduce_max_sync(~0u, r)) {
                    keys = __reduce_max_sync(~0u, keys);
                    if (r >= 0 && (t & 31) == 0) atomicMax(run_keys + r, keys);
                } else if (r >= 0) {
                    atomicMax(run_keys + r, keys);
                }
            }
        }
        __syncthreads();
    }
    // ---- entries of many rows: runs with keys
    int64_t units0 = 0;
    int entries0 = 0;
    for (int r0 = 0; r0 < all_runs; r0 += T) {
        const int r = r0 + t;
        int keys = 0, group = 0;
        if (r < all_runs) {
            group = last_at_most(run_of, g.groups, r);
            keys = g.limits != nullptr ? run_keys[r] : group_len(group);
        }
        const int64_t mine = keys > 0 ? static_cast<int64_t>(units_of(keys, kManyKeys) + kManyCost) * g.Hkv : 0;
        int64_t u = mine, tu;
        int e = keys > 0 ? 1 : 0, te;
        block_scan(u, e, tu, te, sa, sb);
        if (r < all_runs) {
            run_start[r] = units0 + u - mine;
            if (g.limits == nullptr) run_keys[r] = keys;
            if (keys > 0) {
                const int first = first_of[group] + (r - run_of[group]) * run;
                g.many_entries[entries0 + e - 1] = AttnEntry{first, min(run, first_of[group + 1] - first), group, keys};
                g.many_start[entries0 + e - 1] = units0 + u - mine;
            }
        }
        units0 += tu;
        entries0 += te;
    }
    if (t == 0) *g.many = AttnCounts{units0, entries0, 0};
    // ---- entries of few rows: own segments, then small groups
    const int places = any_few ? (own ? g.S : 0) + g.groups : 0;
    int64_t units1 = 0;
    int entries1 = 0;
    for (int p0 = 0; p0 < places; p0 += T) {
        const int p = p0 + t;
        AttnEntry a = {0, 0, -1, 0};
        if (own && p < g.S) {
            a = AttnEntry{p, 1, -1, clamp_len(p0 == 0 ? own_len : g.own_lens[p], g.max_own, g.page)};
        } else if (p < places) {
            const int group = p - (own ? g.S : 0), first = first_of[group], n = first_of[group + 1] - first;
            if (n > 0 && few_group(n)) {
                int keys = 0;
                if (g.limits == nullptr) keys = group_len(group);
                else
                    for (int s = first; s < first + n; ++s) keys = max(keys, keys_seen(group, s));
                a = AttnEntry{first, n, group, keys};
            }
        }
        const int tiles = (a.queries * g.G + kFewRows - 1) / kFewRows;
        const int units = units_of(a.keys, kFewKeys);
        const int64_t mine = a.keys > 0 ? static_cast<int64_t>(units + kFewCost) * g.Hkv * tiles : 0;
        int64_t u = mine, tu;
        int e = a.keys > 0 ? 1 : 0, te;
        block_scan(u, e, tu, te, sa, sb);
        const int64_t start = units1 + u - mine;
        if (a.keys > 0) {
            g.few_entries[entries1 + e - 1] = a;
            g.few_start[entries1 + e - 1] = start;
        }
        if (own && p < g.S) g.places[g.S + p] = AttnPlace{start, units, 0, 0, tiles, {}};
        if (a.group >= 0)   // a small group's queries, 16 at most (with no key among them: 0 units)
            for (int i = 0; i < a.queries; ++i) g.places[a.first + i] = AttnPlace{start, units, 0, i, tiles, {}};
        units1 += tu;
        entries1 += te;
    }
    if (t == 0) *g.few = AttnCounts{units1, entries1, 0};
    // ---- the other queries' places (runs: written above, by other threads).  A call with shared
    // segments alone looks at nothing of them but whether there is a key.
    if (g.groups > 0) {
        __syncthreads();
        int group = 0;   // of the query before, as a rule
        for (int s = t; s < g.S; s += T) {
            AttnPlace at = {};
            if (s >= first_of[0] && s < first_of[g.groups]) {
                if (s < first_of[group] || s >= first_of[group + 1]) group = last_at_most(first_of, g.groups, s);
                const int first = first_of[group];
                if (few_group(first_of[group + 1] - first)) continue;
                const int r = (s - first) / run, keys = run_keys[run_of[group] + r];
                at.units = units_of(keys, kManyKeys);
                if (own) {
                    at.start = run_start[run_of[group] + r];
                    at.many = 1;
                    at.place = (s - first) - r * run;
                    at.tiles = 1;
                }
            }
            if (own) g.places[s] = at;
            else g.places[s].units = at.units;
        }
    }
}

// Where the parts of a row of one segment are.
struct AttnParts {
    int count;             // 0: none
    const float *at;       // the first part's row
    const float2 *stats;
    int step;              // rows from a part to the next (but from the first to the second, half of it)

    __device__ __forceinline__ int64_t place(int c) const {
        return c == 0 ? 0 : static_cast<int64_t>(2 * c - 1) * (step >> 1);
    }
    __device__ __forceinline__ AttnParts from(int lane) const {   // a lane's, for all
        AttnParts p;
        p.count = __shfl_sync(~0u, count, lane);
        p.at = reinterpret_cast<const float *>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(at), lane));
        p.stats = reinterpret_cast<const float2 *>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(stats), lane));
        p.step = __shfl_sync(~0u, step, lane);
        return p;
    }
};

// (n: the counts of the kernel that the query's entry is of, shared out among ctas)
__device__ __forceinline__ AttnParts parts_of(const AttnArgs &g, const AttnPlace &q, const AttnCounts &n, int ctas,
                                              int64_t whole, int head, int kind) {
    AttnParts p = {};
    if (q.units == 0) return p;
    const bool many = q.many != 0;
    const int cost = many ? kManyCost : kFewCost;
    const int kv = head / g.G, row = q.place * g.G + (head - kv * g.G);
    const int rows = many ? 128 * kManyTiles : kFewRows;
    const int seg = many ? kv : kv * q.tiles + row / kFewRows;
    const int per = g.tile_queries * g.G;
    const int at_row = many ? (row < per ? row : row - per + 128) : row % kFewRows;
    const int64_t u0 = q.start + static_cast<int64_t>(seg) * (q.units + cost) + cost;
    const int c0 = owner_of(n.units, ctas, u0), c1 = owner_of(n.units, ctas, u0 + q.units - 1);
    p.count = c1 - c0 + 1;
    int64_t at = whole;
    if (p.count == 1) {
        p.at = g.whole[kind];
        p.stats = g.whole_stats[kind];
    } else {
        at = static_cast<int64_t>(2 * c0 + 1) * rows + at_row;   // the first CTA's second slot, then first slots
        p.at = many ? g.many_part : g.few_part;
        p.stats = many ? g.many_stats : g.few_stats;
        p.step = 2 * rows;
    }
    p.at += at * g.D;
    p.stats += at;
    return p;
}

// The parts of R rows added up by a warp: the maxima and sums a part a lane, the values V to a
// lane.  Everything of a kind is on its way at once; the parts come in the order of their index.
template <typename C, int D, int R>
struct JoinedRows {
    static constexpr int V = D / 32;
    float o[R][V], m[R], l[R];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = neg_inf();
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) o[r][i] = 0.0f;
        }
    }
    // part(c): the first row's values and statistics in part c; row r lies r * row_step rows on
    template <typename F>
    __device__ __forceinline__ void add(int count, int row_step, int lane, F part) {
        for (int c0 = 0; c0 < count; c0 += 32) {
            const int n = min(32, count - c0);
            const float *at = nullptr;
            const float2 *stats = nullptr;
            if (lane < n) part(c0 + lane, at, stats);
            float2 st[R];
            float w[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
                st[r] = lane < n ? __ldcg(stats + r * row_step) : make_float2(neg_inf(), 0.0f);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float top = st[r].x;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const float nm = fmaxf(m[r], top), base = nm == neg_inf() ? 0.0f : nm;
                const float old = exp2_fast(m[r] - base);
                w[r] = exp2_fast(st[r].x - base);
                float sum = lane < n ? st[r].y * w[r] : 0.0f;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
                m[r] = nm;
                l[r] = l[r] * old + sum;
#pragma unroll
                for (int i = 0; i < V; ++i) o[r][i] *= old;
            }
#pragma unroll(R == 1 ? 8 : 2)
            for (int j = 0; j < n; ++j) {
                const float *src = reinterpret_cast<const float *>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(at), j)) + lane * V;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = __shfl_sync(~0u, w[r], j);
                    if constexpr (V == 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + static_cast<int64_t>(r) * row_step * D));
                        o[r][0] = fmaf(f, v.x, o[r][0]), o[r][1] = fmaf(f, v.y, o[r][1]);
                        o[r][2] = fmaf(f, v.z, o[r][2]), o[r][3] = fmaf(f, v.w, o[r][3]);
                    } else {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + static_cast<int64_t>(r) * row_step * D));
                        o[r][0] = fmaf(f, v.x, o[r][0]), o[r][1] = fmaf(f, v.y, o[r][1]);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void put(const AttnArgs &g, int which, int64_t row, int lane) const {
        if (!q4_in_bounds(row >= 0 && row < static_cast<int64_t>(g.S) * g.Hq, g.bounds)) return;
        const float f = l[which] != 0.0f ? 1.0f / l[which] : 0.0f;   // (no key: zeros)
        if (lane == 0 && g.lse != nullptr) g.lse[row] = lse_of(m[which], l[which]);
        const int64_t to = row * D + lane * V;
        const float *v = o[which];
        if (g.out_f32) {
            float *p = static_cast<float *>(g.out) + to;
#pragma unroll
            for (int i = 0; i < V; i += 2) *reinterpret_cast<float2 *>(p + i) = make_float2(v[i] * f, v[i + 1] * f);
        } else {
            uint32_t *p = reinterpret_cast<uint32_t *>(static_cast<C *>(g.out) + to);
#pragma unroll
            for (int i = 0; i < V; i += 2) p[i / 2] = pack2<C>(v[i] * f, v[i + 1] * f);
        }
    }
};

// Calls with both kinds of segments: every row has parts to join.  A warp takes `each` rows
// (query, query head), where their parts are is looked up a lane each.
template <typename C, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs g, int each) {
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(g.S) * g.Hq;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5)) * each;
    wait_prior_grid();
    allow_next_grid();
    AttnParts a = {}, b = {};   // shared, own
    if (lane < each && first + lane < rows) {
        const int s = static_cast<int>((first + lane) / g.Hq), head = static_cast<int>((first + lane) - static_cast<int64_t>(s) * g.Hq);
        const AttnCounts many = *g.many, few = *g.few;
        const AttnPlace qa = g.places[s], qb = g.places[g.S + s];
        const int fc = few_ctas_of(g, few.units), mc = many_ctas_of(g, many.units, few.units);
        a = parts_of(g, qa, qa.many != 0 ? many : few, qa.many != 0 ? mc : fc, first + lane, head, 0);
        b = parts_of(g, qb, few, fc, first + lane, head, 1);
    }
    for (int i = 0; i < each && first + i < rows; ++i) {
        const AttnParts pa = a.from(i), pb = b.from(i);
        JoinedRows<C, D, 1> row;
        row.clear();
        row.add(pa.count + pb.count, 0, lane, [&](int c, const float *&at, const float2 *&stats) {
            const AttnParts &p = c < pa.count ? pa : pb;
            const int64_t place = p.place(c < pa.count ? c : c - pa.count);
            at = p.at + place * D;
            stats = p.stats + place;
        });
        row.put(g, 0, first + i, lane);
    }
}

// Calls with one kind of segments: whole ones are in the output already, and what is left are
// the segments that the border between two CTAs' shares cuts (each dealt with at the first
// border that does), and the queries without a key.
constexpr int kBorderRows = 8;   // CTAs of the rows of a border of the kernel for many rows (few rows: one)

template <typename C, int D, int KEYS, int COST, bool FEW>
__device__ __forceinline__ void join_border(const AttnArgs &g, int c, int part, int lane, int warp) {
    const AttnCounts many = *g.many, few = *g.few, n = FEW ? few : many;
    const int ctas = FEW ? few_ctas_of(g, few.units) : many_ctas_of(g, many.units, few.units);
    if (c + 1 >= ctas) return;
    const int64_t *start = FEW ? g.few_start : g.many_start;
    const int64_t border = units_before(n.units, ctas, c + 1);
    const int entry = entry_at(start, n.entries, border, lane);
    const AttnEntry e = FEW ? g.few_entries[entry] : g.many_entries[entry];
    const int units = units_of(e.keys, KEYS), each = units + COST;
    const int seg = static_cast<int>(quotient(border - start[entry], each));
    const int64_t u0 = start[entry] + static_cast<int64_t>(seg) * each + COST;   // its first unit
    const int count = owner_of(n.units, ctas, u0 + units - 1) - c + 1;
    if (owner_of(n.units, ctas, u0) != c || count < 2) return;
    const int tiles = FEW ? (e.queries * g.G + kFewRows - 1) / kFewRows : 1;
    const int kv = seg / tiles, tile = seg - kv * tiles, rows = FEW ? kFewRows : 128 * kManyTiles;
    const int per = g.tile_queries * g.G, all = e.queries * g.G;
    const float *base = (FEW ? g.few_part : g.many_part) + static_cast<int64_t>(2 * c + 1) * rows * D;
    const float2 *stats = (FEW ? g.few_stats : g.many_stats) + static_cast<int64_t>(2 * c + 1) * rows;
    // a warp's rows, four at a time: those of no query are added up as well, but not put
    constexpr int kWarps = kJoinThreads / 32, kApart = (FEW ? 1 : kBorderRows) * kWarps, R = FEW ? kFewRows / kWarps : 4;
    AttnParts p = {count, nullptr, nullptr, 2 * rows};
    for (int r0 = part * kWarps + warp; r0 < rows; r0 += R * kApart) {
        JoinedRows<C, D, R> out;
        out.clear();
        out.add(count, kApart, lane, [&](int i, const float *&at, const float2 *&st) {
            at = base + (p.place(i) + r0) * D;
            st = stats + p.place(i) + r0;
        });
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = r0 + i * kApart;   // row of the parts: which query and head
            const int row = FEW ? tile * kFewRows + r : r / 128 * per + r % 128;
            if (row >= all || (!FEW && r % 128 >= per)) continue;
            out.put(g, i, static_cast<int64_t>(e.first + row / g.G) * g.Hq + kv * g.G + row % g.G, lane);
        }
    }
}

template <typename C, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_borders_kernel(const AttnArgs g, int many_borders) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_prior_grid();
    allow_next_grid();
    const int c = blockIdx.x, many = many_borders * kBorderRows;
    if (c < many) join_border<C, D, kManyKeys, kManyCost, false>(g, c / kBorderRows, c % kBorderRows, lane, warp);
    else join_border<C, D, kFewKeys, kFewCost, true>(g, c - many, 0, lane, warp);
    // queries without a key: a warp looks at 32 at a time
    const AttnPlace *places = g.groups > 0 ? g.places : g.places + g.S;
    const int warps = gridDim.x * (kJoinThreads / 32);
    for (int s0 = (blockIdx.x * (kJoinThreads / 32) + warp) * 32; s0 < g.S; s0 += warps * 32) {
        unsigned empty = __ballot_sync(~0u, s0 + lane < g.S && places[min(s0 + lane, g.S - 1)].units == 0);
        while (empty != 0) {
            const int s = s0 + __ffs(empty) - 1;
            empty &= empty - 1;
            JoinedRows<C, D, 1> none;
            none.clear();
            for (int h = 0; h < g.Hq; ++h) none.put(g, 0, static_cast<int64_t>(s) * g.Hq + h, lane);
        }
    }
}

namespace {

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

int tile_queries_of(int G) { return 128 / G; }
bool many_possible(int64_t S, int groups, int G) { return groups > 0 && S * G > kFewRows; }

// Places in the workspace.
struct Layout {
    int64_t counts, many_entries, few_entries, many_start, few_start, places, first_of, run_of, run_keys, run_start,
        many_part, few_part, many_stats, few_stats, whole[2], whole_stats[2], total;
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
    l.places = take(2ll * S * sizeof(AttnPlace));
    l.first_of = take(4ll * (groups + 1));
    l.run_of = take(4ll * (groups + 1));
    l.run_keys = take(4 * runs);
    l.run_start = take(8 * runs);
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

// Whether a kernel was compiled to have `registers` with `threads` a block, looked up once per device.
template <typename... P>
int has_registers(void (*kernel)(P...), int threads, int registers, std::atomic<bool> *known) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && known[dev]) return Q4_OK;
    cudaFuncAttributes a = {};
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error(e);
        return Q4_ERR_CUDA;
    }
    if (a.numRegs * threads < registers) return Q4_ERR_UNSUPPORTED;
    if (dev >= 0 && dev < 64) known[dev] = true;
    return Q4_OK;
}

template <typename C, int D>
int launch_attn(const q4_prefix_attn_t &a, AttnArgs &g, cudaStream_t stream) {
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
    using M = ManyAttn<D>;
    using F = FewAttn<D>;
    static_assert(M::smem() <= 227 * 1024, "shared memory of one CTA");
    static_assert(2 * (F::smem() + 1024) <= 228 * 1024, "two CTAs of an SM");
    // (no own segments and one group: all its queries have more than 16 rows, or all are few)
    const bool few = a.own_lens != nullptr || g.many_ctas == 0 || a.groups > 1 || a.group_offsets != nullptr;
    int st = Q4_OK;
    // whatever can be refused, before anything is launched
    if (g.many_ctas > 0) {
        static std::atomic<bool> known[64], configured[64];
        if ((st = has_registers(attn_many_kernel<C, D>, M::kThreads, M::kRegisters, known)) != Q4_OK) return st;
        if ((st = allow_smem(attn_many_kernel<C, D>, M::smem(), configured)) != Q4_OK) return st;
        const cuuint64_t qd[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.S)};
        const cuuint64_t qs[2] = {2 * D, bytes(a.q_stride, a.S)};
        const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(g.G), static_cast<cuuint32_t>(g.tile_queries)};
        if (!encode(&map_q, c.dtype, a.q, 3, qd, qs, qb)) return Q4_ERR_UNSUPPORTED;
    }
    if (few) {
        static std::atomic<bool> configured[64];
        if ((st = allow_smem(attn_few_kernel<C, D>, F::smem(), configured)) != Q4_OK) return st;
    }
    // no more warps than there are queries or groups: each barrier costs by the warp
    const int places = std::max(a.S, a.groups + 1);
    const unsigned threads = static_cast<unsigned>(std::min(kPlanThreads, (places + 31) / 32 * 32));
    st = launch_overlappable(attn_plan_kernel, dim3(1), dim3(threads), 0, stream, call_options().overlap, g);
    if (st != Q4_OK) return st;
    if (g.many_ctas > 0) {
        st = launch_overlappable(attn_many_kernel<C, D>, dim3(static_cast<unsigned>(g.many_ctas)), dim3(M::kThreads),
                                 M::smem(), stream, true, map_q, map_k, map_v, g);
        if (st != Q4_OK) return st;
    }
    if (few) {
        g.beside_many = g.many_ctas > 0;
        st = launch_overlappable(attn_few_kernel<C, D>, dim3(static_cast<unsigned>(g.few_ctas)), dim3(F::kThreads),
                                 F::smem(), stream, true, map_k, map_v, g);
        if (st != Q4_OK) return st;
    }
    if (g.alone) {
        const int borders = g.many_ctas * kBorderRows + (few ? g.few_ctas : 0);
        return launch_overlappable(attn_borders_kernel<C, D>, dim3(static_cast<unsigned>(borders)), dim3(kJoinThreads), 0,
                                   stream, true, g, g.many_ctas);
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
    g.places = reinterpret_cast<AttnPlace *>(w + l.places);
    g.first_of = reinterpret_cast<int *>(w + l.first_of);
    g.run_of = reinterpret_cast<int *>(w + l.run_of);
    g.run_keys = reinterpret_cast<int *>(w + l.run_keys);
    g.run_start = reinterpret_cast<int64_t *>(w + l.run_start);
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
