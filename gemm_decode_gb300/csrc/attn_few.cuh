// attn_few.cuh -- attention of few rows by many keys: a query's own segment, and the shared
// segment of a small group.
//
// A segment is up to 16 rows (queries times the query heads of one kv head) by the keys.  The
// bytes of the keys and values bound it, whatever the rows, so the products go to the
// warp-wide matrix instructions (m16n8k16), whose 16 rows a segment may leave mostly empty,
// and whose accumulators turn into the next product's operand without leaving the registers;
// a tile of the big tensor-core instructions has 128 rows, and its round trip through tensor
// memory would cost more than all of a unit's arithmetic.
//
// One warp brings units of 64 keys into a ring of stages (bulk tensor copies, a box per page or
// 64 rows of one, 128-byte swizzle), four warps compute: each takes 16 of a unit's keys, with a
// running maximum, sum and accumulators of its own, joined in a fixed order when the segment
// ends.  Two CTAs to an SM, three stages of 32 KB each (128 features).  The weights are rounded to
// the cache's type, as the products' other operand is of it (attn_many.cuh has what that costs).
//
// Measured (cold caches): own segments of 64 sequences, 768 keys on average, 8 heads of 128
// (201 MB) 41 us, 4.9 TB/s, 0.72 of measured (38 without the fence before a stage is given back,
// and wrong); of 256 sequences, 218 keys (228 MB) 53 us: there a segment is four units, and its
// queries' loads and its join cost two.  A batch of own segments alone, plan and join among it (graphs):
// 64 sequences of 4000 keys (1.05 GB) 172-178 us, 5.9-6.1 TB/s, 0.87-0.90 of measured; 256 of 1076 on
// average 188 us, 0.88; 8 of 2000 (66 MB) 19.5 us.
#pragma once

#include "attn_common.cuh"

namespace q4 {

template <int D>
struct FewAttn {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kFewKeys * D * 2;            // keys or values of a unit
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kBars = 2 * kStages;   // (an even number: what follows is aligned to 16 bytes)
    static constexpr int kJoinBytes = kFewRows * D * 4;            // one warp's accumulators
    static constexpr size_t smem() {
        return 1024 + static_cast<size_t>(kStages) * kStageBytes + kJoinBytes + 8 * kBars + kWarps * kFewRows * 8 + sizeof(AttnHeld) + 16;
    }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename C>
__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<C, __half>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename C, int D>
__global__ void __launch_bounds__(FewAttn<D>::kThreads, 2)
attn_few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const AttnArgs g) {
    using namespace tc;
    using F = FewAttn<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *ring = smem;
    float *join = reinterpret_cast<float *>(ring + F::kStages * F::kStageBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(join + kFewRows * D);
    float2 *stats = reinterpret_cast<float2 *>(bars + F::kBars);   // [warps][16 rows]
    AttnHeld *held = reinterpret_cast<AttnHeld *>(stats + F::kWarps * kFewRows);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(held + 1);
    const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const unsigned long long limit_ns = g.timeout_ns;
    auto ib = [&](bool ok) { return q4_in_bounds(ok, g.bounds); };
    const uint32_t bar0 = smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (F::kStages + s); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), F::kWarps);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // Beside the kernel for many rows, which is the one before: it lets this one start only after
    // it has waited for the plan itself, and nothing that is read here comes from it, so it is
    // waited for at the end (the kernel behind reads the results of both).  What the plan and the
    // kernels before it wrote is read past the first-level cache.
    if (!g.beside_many) wait_prior_grid();
    allow_next_grid();

    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (limit_ns != 0 ? mbar_try(bar, parity) : mbar_test(bar, parity)) return true;
        if (limit_ns != 0) {
            const unsigned long long t0 = global_ns();
            for (;;) {
                if (mbar_try_sleep(bar, parity, 20000u)) return true;
                if (*abort_flag || global_ns() - t0 > limit_ns) break;
            }
        }
        *abort_flag = 1;
        atomicOr(g.status, 1u);
        return false;
    };

    AttnWalk<kFewKeys, kFewCost, true> walk;
    {
        const AttnCounts few = counts_at(g.few);
        walk.begin(few, g.few_entries, g.few_start, few_ctas_of(g, few.units), lane);
    }
    walk.hold(held);
    __syncthreads();
    AttnSegment s;

    if (warp == F::kWarps) {
        // ------------------------------------------------------------ copies
        Ring<F::kStages> r;
        int64_t issued = 0;
        bool ok = true;
        // a lane's copy: keys or values, 64 features, box of the unit
        const int boxes = kFewKeys >> g.box_shift, copies = 2 * F::kHalves * boxes;
        const int box = lane % boxes, half = lane / boxes % F::kHalves, kv = lane / (boxes * F::kHalves);
        const uint32_t to = smem_addr(ring) + kv * F::kTileBytes + half * (kFewKeys * 128) + (box << g.box_shift) * 128;
        const CUtensorMap *map = kv == 0 ? &map_k : &map_v;
        while (ok && walk.next(s, g.Hkv, g.G)) {
            const int *table = s.e.group < 0 ? g.own_pages + static_cast<int64_t>(s.e.first) * g.max_own
                                             : g.shared_pages + static_cast<int64_t>(s.e.group) * g.max_shared;
            auto page_of = [&](int u) {   // the lane's page of unit u; one outside the pool reads as zeros
                const int key = u * kFewKeys + (box << g.box_shift);
                int id = g.pages;
                if (lane < copies && key < s.e.keys &&
                    ib((key >> g.page_shift) < (s.e.group < 0 ? g.max_own : g.max_shared)))
                    id = __ldcg(table + (key >> g.page_shift));
                return id < 0 || id > g.pages ? g.pages : id;
            };
            int page = page_of(s.u0);
            for (int u = s.u0; u < s.u1; ++u) {
                const int next = u + 1 < s.u1 ? page_of(u + 1) : 0;
                if (!wait(empty(r.s), r.ph ^ 1u)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(full(r.s), F::kStageBytes);
                __syncwarp();
                if (lane < copies)
                    tma_load_4d(to + r.s * F::kStageBytes, map, full(r.s), half * 64,
                                (u * kFewKeys + (box << g.box_shift)) & (g.page - 1), s.head, page);
                r.step();
                ++issued;
                page = next;
            }
        }
        // every copy lands before the CTA may exit, whichever role gives up
        for (int64_t j = issued > F::kStages ? issued - F::kStages : 0; j < issued; ++j)
            mbar_wait(full(static_cast<int>(j % F::kStages)), static_cast<uint32_t>(j / F::kStages) & 1u,
                      50ull * 1000 * 1000);
        if (g.beside_many) wait_prior_grid();
        return;
    }

    // ---------------------------------------------------------------- rows by keys
    constexpr int kK = D / 16, kN = D / 8;
    Ring<F::kStages> r;
    bool ok = true;
    const int row0 = lane >> 2, col0 = 2 * (lane & 3);   // the lane's rows (and 8 further) and columns of a tile
    const float off = g.scale2 >= 0.0f ? neg_inf() : -neg_inf();
    auto sync4 = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    auto all4 = [&](bool v) {   // sync4, and the same answer for all four warps
        uint32_t a;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 p, %1, 0;\n\t"
            "bar.red.and.pred q, 1, 128, p;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(a)
            : "r"(static_cast<uint32_t>(v))
            : "memory");
        return a != 0;
    };
    while (ok && walk.next(s, g.Hkv, g.G)) {
        const int rows = min(kFewRows, s.e.queries * g.G - s.tile * kFewRows);
        // operand A: the rows' queries
        uint32_t q[kK][4];
        int limit[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = row0 + 8 * i;
            int query = 0, head = 0;
            row_of(g, s, s.tile * kFewRows + min(row, rows - 1), query, head);
            const bool have = row < rows && ib(query < g.S && head < g.Hq);
            limit[i] = have ? limit_of(g, s, query) : s.e.keys;   // (a row of zeros that nobody reads)
            const C *src = static_cast<const C *>(g.q) + query * g.q_stride + static_cast<int64_t>(head) * D + col0;
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                q[k][i] = have ? __ldcg(reinterpret_cast<const uint32_t *>(src + 16 * k)) : 0u;
                q[k][i + 2] = have ? __ldcg(reinterpret_cast<const uint32_t *>(src + 16 * k + 8)) : 0u;
            }
        }
        float o[kN][4];
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
        float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};
        for (int u = s.u0; u < s.u1; ++u) {
            if (!wait(full(r.s), r.ph)) ok = false;
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            const uint32_t kt = smem_addr(ring + r.s * F::kStageBytes), vt = kt + F::kTileBytes;
            const int key0 = u * kFewKeys + warp * 16;
            // scores: keys 0-7 and 8-15 of the warp's
            float x[2][4] = {};
            {
                const int key = warp * 16 + (lane & 7) + ((lane >> 4) << 3);   // matrices 2, 3: the later keys
                const int c = (lane >> 3) & 1;                                 // matrices 1, 3: the later features
#pragma unroll
                for (int k = 0; k < kK; ++k) {
                    uint32_t b[4];
                    ldsm4(kt + (k / 4) * (kFewKeys * 128) + sw128_offset(key, 2 * (k % 4) + c), b);
                    mma16816<C>(x[0], q[k], b[0], b[1]);
                    mma16816<C>(x[1], q[k], b[2], b[3]);
                }
            }
            // keys that a row does not see
            const int first = min(limit[0], limit[1]);
            if (__any_sync(~0u, first - key0 < 16)) {   // (key0 + 16 may be 2^31)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key0 + 8 * n + col0 + (i & 1) >= limit[i >> 1]) x[n][i] = off;
            }
            uint32_t p[4];
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a[4] = {x[0][2 * i] * g.scale2, x[0][2 * i + 1] * g.scale2, x[1][2 * i] * g.scale2,
                              x[1][2 * i + 1] * g.scale2};
                float top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                const float nm = fmaxf(m[i], top), base = nm == neg_inf() ? 0.0f : nm;
                f[i] = exp2_fast(m[i] - base);
                m[i] = nm;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[j] = exp2_fast(a[j] - base);
                    sum += a[j];
                }
                l[i] = fmaf(l[i], f[i], sum);   // the lane's columns: joined at the end
                p[i] = pack2<C>(a[0], a[1]);
                p[i + 2] = pack2<C>(a[2], a[3]);
            }
            if (__any_sync(~0u, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    o[n][0] *= f[0], o[n][1] *= f[0];
                    o[n][2] *= f[1], o[n][3] *= f[1];
                }
            }
            // values behind the segment's last key are not the sequence's: zeros, whatever they are
            uint32_t keep[2] = {~0u, ~0u};
            const bool ragged = s.e.keys - key0 < 16;
            if (ragged) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    keep[i] = (key0 + 8 * i + col0 < s.e.keys ? 0xffffu : 0u) |
                              (key0 + 8 * i + col0 + 1 < s.e.keys ? 0xffff0000u : 0u);
            }
            {
                const int key = warp * 16 + (lane & 15);   // matrices 1, 3: the later keys
                const int c = lane >> 4;                   // matrices 2, 3: the later features
#pragma unroll
                for (int n = 0; n < kN; n += 2) {
                    uint32_t b[4];
                    ldsm4_trans(vt + (n / 8) * (kFewKeys * 128) + sw128_offset(key, n % 8 + c), b);
                    if (ragged) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) b[i] &= keep[i & 1];
                    }
                    mma16816<C>(o[n], p, b[0], b[1]);
                    mma16816<C>(o[n + 1], p, b[2], b[3]);
                }
            }
            // The stage goes back to copies, which write it through the asynchronous proxy: every
            // lane's reads are ordered before them.  An arrival alone lets a copy overtake matrix
            // loads whose products come later (without the fence, 20 to 570 of 2048 segments had
            // the last chunks of their values from another unit, at random).
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(r.s));
            r.step();
        }
        // ---- the four warps' parts into one, in their order
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(~0u, l[i], 1);
            l[i] += __shfl_xor_sync(~0u, l[i], 2);
            if ((lane & 3) == 0) stats[warp * kFewRows + row0 + 8 * i] = make_float2(m[i], l[i]);
        }
        ok = all4(ok);
        if (!ok) break;   // all four: nobody waits for a warp that has left
        float f[2], top[2], sum[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = neg_inf();
            sum[i] = 0.0f;
            float2 v[F::kWarps];
#pragma unroll
            for (int w = 0; w < F::kWarps; ++w) {
                v[w] = stats[w * kFewRows + row0 + 8 * i];
                top[i] = fmaxf(top[i], v[w].x);
            }
            const float base = top[i] == neg_inf() ? 0.0f : top[i];
#pragma unroll
            for (int w = 0; w < F::kWarps; ++w) sum[i] += v[w].y * exp2_fast(v[w].x - base);
            f[i] = exp2_fast(m[i] - base);
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            o[n][0] *= f[0], o[n][1] *= f[0];
            o[n][2] *= f[1], o[n][3] *= f[1];
        }
        // warp 3 hands its sums to warp 2, that one to warp 1, that one to warp 0 (lane to lane)
        float4 *box = reinterpret_cast<float4 *>(join);
#pragma unroll 1
        for (int w = F::kWarps - 1; w > 0; --w) {
            if (warp == w) {
#pragma unroll
                for (int n = 0; n < kN; ++n) box[n * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
            }
            sync4();
            if (warp == w - 1) {
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float4 v = box[n * 32 + lane];
                    o[n][0] += v.x, o[n][1] += v.y, o[n][2] += v.z, o[n][3] += v.w;
                }
            }
            sync4();
        }
        if (warp != 0) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = row0 + 8 * i;
            if (row >= rows) continue;
            int query, head;
            row_of(g, s, s.tile * kFewRows + row, query, head);
            const int64_t at = static_cast<int64_t>(query) * g.Hq + head;
            if (!ib(query >= 0 && query < g.S && head < g.Hq && s.slot < 2 * g.few_ctas)) continue;
            if (s.whole && g.alone) {
                const float v = sum[i] != 0.0f ? 1.0f / sum[i] : 0.0f;
                if ((lane & 3) == 0 && g.lse != nullptr) g.lse[at] = lse_of(top[i], sum[i]);
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const int64_t to = at * D + 8 * n + col0;
                    if (g.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(g.out) + to) =
                        make_float2(o[n][2 * i] * v, o[n][2 * i + 1] * v);
                    else *reinterpret_cast<uint32_t *>(static_cast<C *>(g.out) + to) =
                        pack2<C>(o[n][2 * i] * v, o[n][2 * i + 1] * v);
                }
            } else {
                const int kind = s.e.group < 0 ? 1 : 0;
                const int64_t part = s.whole ? at : static_cast<int64_t>(s.slot) * kFewRows + row;
                float *to = (s.whole ? g.whole[kind] : g.few_part) + part * D + col0;
                if ((lane & 3) == 0) (s.whole ? g.whole_stats[kind] : g.few_stats)[part] = make_float2(top[i], sum[i]);
#pragma unroll
                for (int n = 0; n < kN; ++n)
                    *reinterpret_cast<float2 *>(to + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
            }
        }
    }
    if (g.beside_many) wait_prior_grid();
}

}  // namespace q4
