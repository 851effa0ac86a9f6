// attn_common.cuh -- what the kernels of the attention over a shared and an own segment have
// in common: how the work is divided, and where the parts of a result wait to be joined.
//
// Segments.  An entry is a run of queries and the keys they see: queries of a group with the
// group's shared segment, or one query with its own.  With each kv head (and each tile of 16
// rows in the kernel for few rows) it makes a segment: rows (query, query head of that kv
// head) by keys.  Entries whose rows fill a tensor-core tile go to the kernel for many rows,
// the others to the one for few; the planning kernel lists both kinds with their keys, in
// units (tiles of keys), numbered through: entry by entry, within it segment by segment.
//
// Each kernel's CTAs share its units evenly, CTA c takes [c U / C, (c + 1) U / C), whatever the
// lengths are; a segment counts for some units more than it has, for what its beginning and
// its end cost.  A segment that falls to several CTAs leaves a part with each of them, in one
// of two slots that a CTA has (only its first and its last segment can be shared); one that a
// CTA holds whole goes straight to the output where nothing else can add to it, else to a
// place by query and head.  A part is the row's sum of weighted values, relative to the
// part's own maximum, with that maximum (in powers of two) and the sum of weights; the joining
// kernel adds the parts of a row in the order of the keys, so results do not depend on timing.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "q4_decode.cuh"
#include "q4_tc.cuh"

namespace q4 {

using namespace tc;

constexpr int kManyKeys = 128, kFewKeys = 64;   // keys of a unit
constexpr int kManyCost = 2, kFewCost = 2;      // units that a segment's beginning and end count for
constexpr int kFewRows = 16;                    // rows of a segment of the kernel for few rows
constexpr int kManyTiles = 2;                   // tiles of 128 rows of one segment of the kernel for many

struct AttnEntry {
    int first, queries;   // queries [first, first + queries)
    int group;            // whose shared segment, or -1: the query's own
    int keys;             // the most that one of the queries sees
};

// Where the joining kernel finds the parts of a query's rows of one entry.
struct alignas(16) AttnPlace {
    int64_t start;        // the entry's first unit
    int units;            // of a segment; 0: the query sees no key of this kind
    int many;             // kernel: many rows (1) or few
    int place, tiles;     // the query's place in its entry; tiles of 16 rows per kv head (few rows)
    int pad[2];
};

struct AttnCounts {
    int64_t units;   // with the cost of each segment
    int entries;
    int pad;
};

struct AttnArgs {
    int S, Hq, Hkv, G, groups;   // G: query heads of a kv head
    int D;
    int page, page_shift, pages;
    int box, box_shift;          // rows of a page that one copy brings
    int max_shared, max_own;
    int tile_queries;            // of a tile of 128 rows
    int out_f32, alone;          // alone: a call with one kind of segment, so whole ones are final
    float scale2;                // scale * log2(e)
    const void *q;
    int64_t q_stride;
    const int *group_offsets, *shared_pages, *shared_lens, *limits, *own_pages, *own_lens;
    void *out;
    float *lse;
    // workspace
    AttnCounts *many, *few;
    AttnEntry *many_entries, *few_entries;
    int64_t *many_start, *few_start;   // first unit of each entry
    AttnPlace *places;   // [2][S]: shared, own
    int *first_of;       // [groups + 1] clamped offsets
    int *run_of;         // [groups + 1] first run of each group's queries
    int *run_keys;       // [runs] the most keys that a query of the run sees
    int64_t *run_start;  // [runs] first unit of the run
    int many_ctas, few_ctas;
    int beside_many;             // the kernel for few rows runs beside the one for many
    float *many_part, *few_part;     // [2 CTAs][rows][D]
    float2 *many_stats, *few_stats;  // [2 CTAs][rows]: maximum, sum of weights
    float *whole[2];                 // [S][Hq][D]: shared, own
    float2 *whole_stats[2];
    unsigned long long timeout_ns;
    unsigned int *status;
    unsigned int *bounds;
};

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ int clamp_len(int n, int most_pages, int page) {
    const int64_t most = static_cast<int64_t>(most_pages) * page;   // below 2^31: checked by the call
    return n < 0 ? 0 : n > most ? static_cast<int>(most) : n;
}

// Units of a number of keys.  A table may name just below 2^31 tokens: the sum is unsigned, where
// no such number passes the type.
__host__ __device__ constexpr int units_of(int keys, int unit) {
    return static_cast<int>((static_cast<uint32_t>(keys) + static_cast<uint32_t>(unit - 1)) / static_cast<uint32_t>(unit));
}
static_assert(units_of(0, kManyKeys) == 0 && units_of(1, kManyKeys) == 1 && units_of(129, kManyKeys) == 2, "units");
static_assert(units_of(0x7fffffff, kManyKeys) == 1 << 24 && units_of(0x7fffffff, kFewKeys) == 1 << 25, "units");

// CTAs that take part (each has a unit), the units that CTA c of them takes, and the CTA that
// takes unit u.
__device__ __forceinline__ int few_ctas_of(const AttnArgs &g, int64_t few) {
    return few < g.few_ctas ? static_cast<int>(few) : g.few_ctas;
}
// The two kernels run at the same time, on different SMs.  Where the many rows have a unit for each
// SM and the few rows ten for each of their CTAs, the many rows take no more CTAs than have five
// units each, and the other SMs read keys and values meanwhile: a segment of the many rows then
// falls to fewer CTAs, and what its beginning costs is paid less often.  us with a unit each and
// with five, 64 sequences of 32 heads of 128 (many, few units):
//   528, 6656  70.6  65.2     272, 8192  75.2  68.4     272, 2560  37.9  39.2
//   528, 3584  51.4  48.7     272, 3584  47.1  43.8     80, 2560   33.2  38.2
// Few rows with little to do do not make up for the wait for the longer runs of the many (24, 576:
// 22.9 and 28.6; 36, 727: 22.8 and 27.7), and many rows of less than a unit an SM leave SMs free as
// it is (18, 3120: 24.4 and 28.4; 120, 3384: 28.5 and 30.8).  (What the rule leaves: 16 sequences of
// 14 heads of 64, one tile of rows: 68, 2048 33.6 and 31.6.)
__device__ __forceinline__ int many_ctas_of(const AttnArgs &g, int64_t many, int64_t few) {
    const bool fewer = many >= g.many_ctas && few >= 10 * static_cast<int64_t>(g.few_ctas);
    const int64_t n = fewer ? (many + 4) / 5 : many;
    return n < g.many_ctas ? static_cast<int>(n) : g.many_ctas;
}
__device__ __forceinline__ AttnCounts counts_at(const AttnCounts *n) {
    const int4 raw = __ldcg(reinterpret_cast<const int4 *>(n));
    return AttnCounts{static_cast<int64_t>(static_cast<uint32_t>(raw.x)) | static_cast<int64_t>(raw.y) << 32, raw.z, 0};
}
// (divisions in 32 bits where the numbers allow it: in 64 they take several hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
__device__ __forceinline__ int64_t units_before(int64_t units, int ctas, int c) { return quotient(units * c, ctas); }
__device__ __forceinline__ int owner_of(int64_t units, int ctas, int64_t u) {
    return static_cast<int>(quotient((u + 1) * ctas - 1, units));
}

// The entry of unit u: the last of `n` with start <= u, by a warp, 32 places a round.
__device__ __forceinline__ int entry_at(const int64_t *start, int n, int64_t u, int lane) {
    int lo = 0, hi = n;   // start[lo] <= u < start[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, p = lo + lane * step;
        const unsigned below = __ballot_sync(~0u, p < hi && __ldcg(start + p) <= u);
        const int k = 31 - __clz(below);   // (lane 0 always)
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Walks the segments of a CTA's share; every role of a CTA has one of its own.
struct AttnSegment {
    AttnEntry e;
    int head, tile;       // kv head, tile of rows (few rows)
    int u0, u1;           // units of the segment, [0, units) when whole
    int units;
    bool whole;
    int slot;             // where a part goes: 2 * CTA + (the segment's first CTA: 1)
};
// The first entries of a CTA's share, in shared memory.
struct AttnHeld {
    static constexpr int kMost = 32;
    int4 entry[kMost];
    int64_t start[kMost];
};
template <int KEYS, int COST, bool FEW>
struct AttnWalk {
    int64_t at, end;
    int entry, first;
    const AttnHeld *held;
    const AttnEntry *entries;
    const int64_t *start;

    // To the CTA's first unit, by a warp.
    __device__ __forceinline__ void begin(const AttnCounts &n, const AttnEntry *all, const int64_t *starts, int ctas,
                                          int lane) {
        const int64_t units = n.units;
        const bool takes_part = static_cast<int>(blockIdx.x) < ctas;
        entries = all;
        start = starts;
        at = takes_part ? units_before(units, ctas, blockIdx.x) : 0;
        end = takes_part ? units_before(units, ctas, blockIdx.x + 1) : 0;
        const int lo = at < end ? entry_at(start, n.entries, at, lane) : 0;
        entry = first = lo;
        left_ = n.entries - lo;
    }
    // The entries from the first on into shared memory, by all threads (a barrier is to follow).
    __device__ __forceinline__ void hold(AttnHeld *to) {
        held = to;
        const int i = threadIdx.x;
        if (i < AttnHeld::kMost && i < left_ && at < end) {
            to->entry[i] = __ldcg(reinterpret_cast<const int4 *>(entries + first + i));
            to->start[i] = __ldcg(start + first + i);
        }
    }
    // The next segment, or false.
    __device__ __forceinline__ bool next(AttnSegment &s, int heads, int G) {
        while (at < end) {
            const int i = entry - first;
            const int4 raw = i < AttnHeld::kMost ? held->entry[i] : __ldcg(reinterpret_cast<const int4 *>(entries + entry));
            const int64_t from = at - (i < AttnHeld::kMost ? held->start[i] : __ldcg(start + entry));
            s.e = AttnEntry{raw.x, raw.y, raw.z, raw.w};
            s.units = units_of(s.e.keys, KEYS);
            const int each = s.units + COST, tiles = FEW ? (s.e.queries * G + kFewRows - 1) / kFewRows : 1;
            const int seg = static_cast<int>(quotient(from, each)), off = static_cast<int>(from - static_cast<int64_t>(seg) * each);
            const int take = static_cast<int>(min(static_cast<int64_t>(each - off), end - at));
            at += take;
            if (off + take == each && seg + 1 == heads * tiles) ++entry;
            s.head = seg / tiles;
            s.tile = seg - s.head * tiles;
            s.u0 = max(off - COST, 0);
            s.u1 = off + take - COST;
            s.whole = s.u0 == 0 && s.u1 == s.units;
            s.slot = 2 * blockIdx.x + (s.u0 == 0 ? 1 : 0);
            if (s.u1 > s.u0) return true;
        }
        return false;
    }

private:
    int left_;
};

// Row `row` of a segment's rows: query and query head.
__device__ __forceinline__ void row_of(const AttnArgs &g, const AttnSegment &s, int row, int &query, int &head) {
    const int i = row / g.G;
    query = s.e.first + i;
    head = s.head * g.G + (row - i * g.G);
}
// Keys of the segment that a query sees.
__device__ __forceinline__ int limit_of(const AttnArgs &g, const AttnSegment &s, int query) {
    if (s.e.group < 0 || g.limits == nullptr) return s.e.keys;
    return max(0, min(s.e.keys, __ldcg(g.limits + query)));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
template <typename C>
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // a in the lower half
    uint32_t r;
    if constexpr (std::is_same<C, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// log sum exp, natural, from a maximum in powers of two and the sum relative to it
__device__ __forceinline__ float lse_of(float m, float l) {
    return l != 0.0f ? (m + log2f(l)) * 0.693147180559945f : neg_inf();
}

}  // namespace q4
