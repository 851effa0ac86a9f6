// moe_gemm_many.cuh -- matrix product grouped by expert, many rows per expert (bfloat16
// prompts).  Shared parts, and how the work is divided: moe_gemm_common.cuh.
//
// An item is 256 weight rows (two tiles) by up to 128 rows of one expert: each row of x that
// a CTA reads serves 256 weight rows, half the L2 traffic of one tile.  Operand A is
// (q - z) s, rounded once to binary16, and one sum goes over K: sums of their own for each
// group of weights, as with few rows, would cost more to take out of tensor memory than the
// multiplication by s does.
//
// One CTA per SM, 28 warps:
//   warp 0       bulk tensor copies of the codes of a unit (256 rows x 64 bytes) into a ring
//   warp 1       the MMAs: the whole warp walks the loop, one elected lane issues
//   warps 2, 3   scales and zero points, 16 groups per row at a time
//   warps 4-11   epilogue, four warps per weight tile: sums to registers, scale, SwiGLU,
//                rounding, store; a tile's accumulators are free for the next item while the
//                other tile's are still being read
//   warps 12-15  copy the rows of x, by index, one unit each in turn (16-byte asynchronous
//                copies: a bulk copy of four rows by index took a lane 80 to 140 cycles)
//   warps 16-27  dequantisers, three groups of four warps taking the jobs (unit, weight tile)
//                in turn: a thread owns a weight row, reads 64 bytes of codes and writes 128
//                weights into 64 columns of tensor memory
//
// What bounds it: the hand-overs between the roles.  The tensor core is busy 930 of 2160
// cycles per unit (43 %, ncu; 1024 were all 128 rows in use); in the rest the issuing warp
// waits for weights, for rows of x or, at an item's end, for the epilogue.  Measured: 4096 tokens, 8 of 64 experts of 2048 x 2048 (groups
// of 64, SwiGLU): 302 us, 911 TFLOP/s (0.48 of measured bf16).  A fourth dequantiser group
// (310 us) and an MMA warp per weight tile (323 us, with registers spilled) gained nothing.
#pragma once

#include "moe_gemm_common.cuh"

namespace q4 {

struct ManyShape {
    static constexpr int RT = 2, NT = 128;                     // weight tiles and rows of x per item
    static constexpr int kGroups = 3;                          // dequantiser groups of four warps
    static constexpr int kXWarp = 4 + 4 * RT;                  // first of the four that copy x
    static constexpr int kDqWarp = kXWarp + 4;                 // first dequantiser
    static constexpr int kThreads = 32 * (kDqWarp + 4 * kGroups);
    static constexpr int kAccCols = RT * NT;
    static constexpr int kSlots = (kTmemCols - kAccCols) / kSlotCols;   // jobs of weights
    static constexpr int kCodeBytes = RT * 128 * (kUnit / 2);
    static constexpr int kCodeStages = 3;
    // A dequantiser group skips the jobs of the others, and a wait by parity tells a phase
    // from the one before it only.  So the ring of weights holds a job per group (the job a
    // group finished last then lies within the ring), and no more units than the codes' ring
    // (a free slot of weights then proves that the codes' previous use has landed).
    static_assert(kGroups <= kSlots && kSlots <= RT * kCodeStages && kGroups <= kCodeStages,
                  "a parity could be taken for an older phase's");
    static constexpr int kXHalf = NT * 128;                    // rows of x, 64 k
    static constexpr int kXBytes = 2 * kXHalf;
    static constexpr int kXStages = 4;
    static constexpr int kScaleBytes = RT * 128 * kScaleRow;
    static constexpr int kScaleBufs = 2;
    static constexpr int kBars = 2 * (kCodeStages + kXStages + kScaleBufs + kSlots + RT) + 1;
    static constexpr size_t fixed() {
        return 1024 + static_cast<size_t>(kXStages) * kXBytes + static_cast<size_t>(kCodeStages) * kCodeBytes +
               static_cast<size_t>(kScaleBufs) * kScaleBytes + 8 * kBars + RT * 2 * NT * 4 + 4 * NT * 4 + 64;
    }
    static constexpr size_t smem(int E) { return fixed() + 8 * (static_cast<size_t>(E) + 1); }
};

__global__ void __launch_bounds__(ManyShape::kThreads, 1)
moe_gemm_many_kernel(const __grid_constant__ CUtensorMap map_codes, const MoeKernelArgs g) {
    using S = ManyShape;
    constexpr int RT = S::RT, NT = S::NT;
    using Out = __nv_bfloat16;
    static_assert(S::smem(kMaxExperts) <= 227 * 1024, "shared memory of one CTA");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *x_ring = smem;
    unsigned char *code_ring = x_ring + S::kXStages * S::kXBytes;
    unsigned char *scale_ring = code_ring + S::kCodeStages * S::kCodeBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(scale_ring + S::kScaleBufs * S::kScaleBytes);
    float *row_scale = reinterpret_cast<float *>(bars + S::kBars);   // [RT][2][NT]
    int *x_rows = reinterpret_cast<int *>(row_scale + RT * 2 * NT);  // [4][NT] rows of x, a list per copying warp
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(x_rows + 4 * NT);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *last_flag = reinterpret_cast<int *>(tmem_slot + 2);         // [RT]
    int *first_row = reinterpret_cast<int *>(tmem_slot + 4);         // [E + 1]
    int *first_tile = first_row + g.E + 1;                           // [E + 1]

    const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const unsigned long long limit = g.timeout_ns;
    auto ib = [&](bool ok) { return q4_in_bounds(ok, g.bounds); };   // bounds-checking builds

    const uint32_t bar0 = smem_addr(bars);
    auto code_full = [&](int s) { return bar0 + 8u * s; };
    auto code_empty = [&](int s) { return bar0 + 8u * (S::kCodeStages + s); };
    constexpr int kX = 2 * S::kCodeStages, kSc = kX + 2 * S::kXStages, kA = kSc + 2 * S::kScaleBufs,
                  kD = kA + 2 * S::kSlots;
    auto x_full = [&](int s) { return bar0 + 8u * (kX + s); };
    auto x_empty = [&](int s) { return bar0 + 8u * (kX + S::kXStages + s); };
    auto sc_full = [&](int s) { return bar0 + 8u * (kSc + s); };
    auto sc_empty = [&](int s) { return bar0 + 8u * (kSc + S::kScaleBufs + s); };
    auto a_full = [&](int s) { return bar0 + 8u * (kA + s); };
    auto a_empty = [&](int s) { return bar0 + 8u * (kA + S::kSlots + s); };
    auto d_full = [&](int s) { return bar0 + 8u * (kD + s); };
    auto d_empty = [&](int s) { return bar0 + 8u * (kD + RT + s); };
    const uint32_t done_bar = bar0 + 8u * (S::kBars - 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kCodeStages; ++s) {
            mbar_init(code_full(s), 1);
            mbar_init(code_empty(s), 4 * RT);
        }
        for (int s = 0; s < S::kXStages; ++s) {
            mbar_init(x_full(s), 1);
            mbar_init(x_empty(s), 1);
        }
        for (int s = 0; s < S::kScaleBufs; ++s) {
            mbar_init(sc_full(s), 2);
            mbar_init(sc_empty(s), 4 * S::kGroups);
        }
        for (int s = 0; s < S::kSlots; ++s) {
            mbar_init(a_full(s), 4);
            mbar_init(a_empty(s), 1);
        }
        for (int s = 0; s < RT; ++s) {
            mbar_init(d_full(s), 1);
            mbar_init(d_empty(s), 4);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    wait_prior_grid();
    if (warp == 2) expert_tables<NT>(g, lane, first_row, first_tile);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
    allow_next_grid();

    MoePlan plan = make_plan<RT>(g, first_row, first_tile);

    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(g.status, 1u);
    };
    // bounded wait; false (and the abort flag) on expiry or when another role gave up
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (limit != 0 ? mbar_try(bar, parity) : mbar_test(bar, parity)) return true;   // (try suspends)
        if (limit != 0) {
            const unsigned long long t0 = global_ns();
            for (;;) {
                if (mbar_try_sleep(bar, parity, 20000u)) return true;
                if (*abort_flag || global_ns() - t0 > limit) break;
            }
        }
        fail();
        return false;
    };

    if (warp < 4) {
    if (warp == 0) {
        // ------------------------------------------------------------ codes
        if (lane == 0) {
            Ring<S::kCodeStages> r;
            int64_t issued = 0;
            MoeSegment s = {};
            bool ok = true;
            while (ok && next_segment<NT>(plan, s)) {
                const int row = s.expert * g.N + s.group * (128 * RT);
                for (int u = s.k0; u < s.k1; ++u) {
                    if (!wait(code_empty(r.s), r.ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(code_full(r.s), S::kCodeBytes);
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        tma_load_2d(smem_addr(code_ring + r.s * S::kCodeBytes + t * (128 * kUnit / 2)), &map_codes,
                                    code_full(r.s), u * (kUnit / 2), row + t * 128);
                    r.step();
                    ++issued;
                }
            }
            // Every copy lands before the CTA may exit, whichever role gives up, and when: a
            // flag read here could be raised a moment later.  (Otherwise the copies are waited
            // for anyway, by the dequantisers.)
            for (int64_t j = issued > S::kCodeStages ? issued - S::kCodeStages : 0; j < issued; ++j)
                mbar_wait(code_full(static_cast<int>(j % S::kCodeStages)),
                          static_cast<uint32_t>(j / S::kCodeStages) & 1u, 50ull * 1000 * 1000);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        Ring<S::kXStages> rx;
        Ring<S::kSlots> ra;
        uint32_t d_ph = 0;
        MoeSegment s = {};
        bool ok = true;
        const uint64_t x_desc = umma_desc(smem_addr(x_ring));
        const int half_unit = g.K % kUnit != 0 && g.K % kUnit <= kHalf ? g.K / kUnit : -1;   // the unit of one half
        while (ok && next_segment<NT>(plan, s)) {
            const int n16 = (s.rows + 15) / 16 * 16;
            const uint32_t idesc = idesc_f16(false, 128, n16);
            for (int u = s.k0; ok && u < s.k1; ++u) {
                const uint64_t xd = x_desc + static_cast<uint32_t>(rx.s) * (S::kXBytes / 16);
                const bool both = u != half_unit;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    // all the barriers of the step are looked at together: one after another,
                    // each costs the latency of its own round trip
                    const bool need_x = t == 0, need_d = u == s.k0;
                    const bool ra_ok = mbar_test(a_full(ra.s), ra.ph);
                    const bool rx_ok = !need_x || mbar_test(x_full(rx.s), rx.ph);
                    const bool rd_ok = !need_d || mbar_test(d_empty(t), d_ph ^ 1u);
                    if (!__all_sync(~0u, ra_ok && rx_ok && rd_ok)) {
                        if (need_d && !wait(d_empty(t), d_ph ^ 1u)) ok = false;
                        if (need_x && !wait(x_full(rx.s), rx.ph)) ok = false;
                        if (!wait(a_full(ra.s), ra.ph)) ok = false;
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const uint32_t a = tmem + S::kAccCols + ra.s * kSlotCols;
                    const uint32_t d = tmem + static_cast<uint32_t>(t * NT);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // 16 k: 32 bytes of a row of x, 8 columns of weights
                            umma_f16_ts(d, a + kk * 8, xd + kk * 2, idesc, kk > 0 || u > s.k0 ? 1u : 0u);
                        if (both) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_f16_ts(d, a + 32 + kk * 8, xd + S::kXHalf / 16 + kk * 2, idesc, 1u);
                        }
                        umma_commit(a_empty(ra.s));
                        if (t == RT - 1) umma_commit(x_empty(rx.s));
                        if (u + 1 == s.k1) umma_commit(d_full(t));
                    }
                    __syncwarp();
                    ra.step();
                }
                rx.step();
            }
            d_ph ^= 1u;
        }
        if (elect_one()) umma_commit(done_bar);   // every MMA issued (waited for before tensor memory is freed)
        __syncwarp();
    } else {
        // ------------------------------------------------------------ scales and zero points
        Ring<S::kScaleBufs> r;
        MoeSegment s = {};
        bool ok = true;
        while (ok && next_segment<NT>(plan, s)) {
            for (int c = s.k0 >> (g.gshift - 3); c <= (s.k1 - 1) >> (g.gshift - 3); ++c) {   // 2^(gshift - 3) units each
                if (!wait(sc_empty(r.s), r.ph ^ 1u)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                load_scales<RT>(g, s.expert, s.group * (128 * RT), c, warp & 1, lane, scale_ring + r.s * S::kScaleBytes);
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full(r.s));
                r.step();
            }
        }
    }
    } else if (warp < S::kXWarp) {
        // ------------------------------------------------------------ epilogue
        const int rt = (warp - 4) >> 2;           // weight tile: four warps each
        const int t = threadIdx.x - 128 * (1 + rt);   // lane of tensor memory: weight row of the tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int cols = g.swiglu ? g.N >> 1 : g.N;
        auto sync4 = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + rt) : "memory"); };
        auto all4 = [&](bool v) {   // the same answer for all four warps
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 p, %1, 0;\n\t"
                "bar.red.and.pred q, %2, 128, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(static_cast<uint32_t>(v)), "r"(1 + rt)
                : "memory");
            return r != 0;
        };
        auto put = [&](Out *p, float v, bool have) {
            if (!have || !ib(p >= static_cast<Out *>(g.y) && p < static_cast<Out *>(g.y) + static_cast<int64_t>(g.R) * cols)) return;
            *p = __float2bfloat16_rn(v);
        };
        uint32_t d_ph = 0;
        MoeSegment s = {};
        int buf = 0;
        // 16 columns (rows of x from j0 on) of weight row n, unscaled sums in v
        auto finish = [&](int n, int j0, const float *v, const float *scale) {
            if (g.swiglu) {
                // lanes 2i (gate) and 2i + 1 (up) exchange: the even lane takes rows j, the odd one j + 1
                const int odd = lane & 1;
                Out *p = static_cast<Out *>(g.y) + static_cast<int64_t>(s.row0 + j0 + odd) * cols + (n >> 1);
                float h[8];
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float other = __shfl_xor_sync(~0u, odd ? v[j] : v[j + 1], 1);
                    const float f = scale[j0 + j + odd];
                    const float gate = (odd ? other : v[j]) * f, up = (odd ? v[j + 1] : other) * f;
                    // the fast exponential and division are off by 2^-20, the rounding by 2^-8
                    h[j / 2] = __fdividef(gate, 1.0f + __expf(-gate)) * up;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    put(p + static_cast<int64_t>(2 * j) * cols, h[j], j0 + 2 * j + odd < s.rows && n < g.N);
            } else {
                Out *p = static_cast<Out *>(g.y) + static_cast<int64_t>(s.row0 + j0) * cols + n;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    put(p + static_cast<int64_t>(j) * cols, v[j] * scale[j0 + j], j0 + j < s.rows && n < g.N);
            }
        };
        while (next_segment<NT>(plan, s)) {
            float *scale = row_scale + (rt * 2 + buf) * NT;
            buf ^= 1;
            for (int j = t; j < NT; j += 128) {
                float f = 0.0f;
                if (j < s.rows) {
                    int src = g.rows != nullptr ? g.rows[s.row0 + j] : s.row0 + j;
                    if (src < 0 || src >= g.Tx) src = g.Tx;
                    f = g.xscale[src];
                }
                scale[j] = f;
            }
            sync4();
            const int n = s.group * (128 * RT) + rt * 128 + t;
            const bool whole = s.k1 - s.k0 == static_cast<int>(plan.units);
            // a CTA that holds part of an item's K leaves its sums in a slot of its own
            const uint32_t u0 = s.item * plan.units;
            const uint32_t c0 = whole ? 0 : plan.owner(u0), c1 = whole ? 0 : plan.owner(u0 + plan.units - 1);
            auto slot_of = [&](uint32_t c) {
                return g.partial + ((2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * RT + rt) * (128 * NT) + t;
            };
            float *mine = slot_of(blockIdx.x);
            auto emit = [&](int j0, const float *v) {
                if (whole) {
                    finish(n, j0, v, scale);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j0 + j < s.rows &&
                            ib(mine + (j0 + j) * 128 < g.partial + static_cast<int64_t>(2 * gridDim.x) * RT * 128 * NT))
                            mine[(j0 + j) * 128] = v[j];
                }
            };
            const uint32_t acc0 = tmem + lane_base + static_cast<uint32_t>(rt * NT);
            if (!all4(wait(d_full(rt), d_ph))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 0; j0 < s.rows; j0 += 16) {
                float v[16];
                tmem_ld16(acc0 + j0, v);
                emit(j0, v);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(d_empty(rt));
            d_ph ^= 1u;
            if (!whole) {
                __threadfence();
                sync4();
                if (t == 0)
                    last_flag[rt] = atomicAdd(g.arrived + c0 * RT + rt, 1u) == c1 - c0;
                sync4();
                if (last_flag[rt] != 0) {
                    __threadfence();
#pragma unroll 1
                    for (int j0 = 0; j0 < s.rows; j0 += 16) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0.0f;
                        for (uint32_t c = c0; c <= c1; ++c) {
                            const float *p = slot_of(c);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (j0 + j < s.rows) v[j] += __ldcg(p + (j0 + j) * 128);
                        }
                        finish(n, j0, v, scale);
                    }
                }
                sync4();   // last_flag is read before the next item's
            }
        }
    } else if (warp < S::kDqWarp) {
        // ------------------------------------------------------------ rows of x
        // The four warps take the units in turn.  Eight lanes copy the 128 bytes of a row's
        // 64 k, 16 bytes each, to where the 128-byte swizzle wants them.  A unit is handed
        // over when its copies have landed: after the warp's next unit has been issued if
        // there is room for that already, else before the warp waits for room.
        const int me = warp - S::kXWarp;
        Ring<S::kXStages> r;
        r.step(me % S::kXStages);
        int full = -1;     // stage whose copies are in flight
        uint32_t next = static_cast<uint32_t>(me), before = 0;   // the warp's next unit; units of earlier segments
        MoeSegment s = {};
        bool ok = true;
        const int chunk = lane & 7, sub = lane >> 3;
        const uint32_t x_base = smem_addr(x_ring);
        int *list = x_rows + me * NT;
        auto hand_over = [&]() {
            fence_proxy_async();   // the copies' writes, for the tensor core
            __syncwarp();
            if (lane == 0) mbar_arrive(x_full(full));
        };
        while (ok && next_segment<NT>(plan, s)) {
            const uint32_t units = static_cast<uint32_t>(s.k1 - s.k0);
            if (next - before >= units) {   // none of this segment's units is this warp's
                before += units;
                continue;
            }
            const int n16 = (s.rows + 15) & ~15;
            __syncwarp();
            for (int j = lane; j < n16; j += 32) {
                int src = g.Tx;   // the row of zeros
                if (j < s.rows) {
                    src = g.rows != nullptr ? g.rows[s.row0 + j] : s.row0 + j;
                    if (src < 0 || src >= g.Tx) src = g.Tx;
                }
                list[j] = src;
            }
            __syncwarp();
            for (; next - before < units; next += 4) {
                const int u = s.k0 + static_cast<int>(next - before);
                if (!__all_sync(~0u, mbar_test(x_empty(r.s), r.ph ^ 1u))) {
                    if (full >= 0) {
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        hand_over();
                        full = -1;
                    }
                    if (!wait(x_empty(r.s), r.ph ^ 1u)) ok = false;
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                }
                const int k = u * kUnit + chunk * 8;
                const uint32_t dst = x_base + r.s * S::kXBytes;
                const bool have0 = k < g.K, have1 = k + kHalf < g.K;
                const __half *from = g.xparts + (have0 ? k : 0);
#pragma unroll 4
                for (int j = sub; j < n16; j += 4) {
                    if (!ib(list[j] >= 0 && list[j] <= g.Tx)) continue;
                    const __half *row = from + static_cast<int64_t>(list[j]) * g.K;
                    const uint32_t to = dst + sw128_offset(j, chunk);
                    copy16(to, row, have0);
                    copy16(to + S::kXHalf, row + (have1 ? kHalf : 0), have1);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (full >= 0) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    hand_over();
                }
                full = r.s;
                r.ph ^= 1u;   // four warps, four stages: the same stage again
            }
            before += units;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (full >= 0) hand_over();
    } else {
        // ------------------------------------------------------------ dequantisers
        const int group_id = (warp - S::kDqWarp) >> 2;
        const int row = (warp & 3) * 32 + lane;   // weight row of the tile = lane of tensor memory
        const uint32_t slots = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + S::kAccCols;
        // Jobs are (unit, weight tile) in the order the MMAs take them; this group takes every
        // kGroups-th, whatever segment it falls into.
        constexpr int G = S::kGroups;
        Ring<S::kCodeStages> rc;
        Ring<S::kScaleBufs> rs;
        Ring<S::kSlots> ra;
        ra.step(group_id);
        uint32_t next = static_cast<uint32_t>(group_id), before = 0;   // the next job; jobs of earlier segments
        uint32_t chunk = 0, held = 0;                                  // chunks of earlier segments; chunks taken so far
        uint32_t unit_at = 0;                                          // unit whose codes are at rc
        MoeSegment s = {};
        bool ok = true;
        const int chunk_shift = g.gshift - 3;
        const int swz = (row >> 1) & 3;   // 64-byte swizzle: 16-byte chunk c of row r lies at c ^ ((r >> 1) & 3)
        auto take_chunk = [&]() {   // let go of the chunk held and wait for the next
            if (held > 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_empty(rs.s));
                rs.step();
            }
            ++held;
            if (!wait(sc_full(rs.s), rs.ph)) ok = false;
            ok = __all_sync(~0u, ok);
        };
        while (ok && next_segment<NT>(plan, s)) {
            const uint32_t jobs = static_cast<uint32_t>(s.k1 - s.k0) * RT;
            const int first_chunk = s.k0 >> chunk_shift;
            for (; next - before < jobs; next += G) {
                const int t = static_cast<int>((next - before) % RT);
                const int u = s.k0 + static_cast<int>((next - before) / RT);
                // the chunk of scales: every group passes through every chunk
                const uint32_t want = chunk + static_cast<uint32_t>((u >> chunk_shift) - first_chunk) + 1;
                while (ok && held < want) take_chunk();
                if (!ok) break;
                const uint32_t unit = next / RT;
                rc.step(static_cast<int>(unit - unit_at));
                unit_at = unit;
                const int slot = ra.s;
                if (!wait(a_empty(slot), ra.ph ^ 1u)) ok = false;   // before code_full: see ManyShape
                if (!wait(code_full(rc.s), rc.ph)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                ra.step(G);
                tc_fence_after();
                const unsigned char *codes = code_ring + rc.s * S::kCodeBytes + t * (128 * kUnit / 2) + row * 64;
                const unsigned char *sz = scale_ring + rs.s * S::kScaleBytes + (t * 128 + row) * kScaleRow;
                uint4 c4[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) c4[q] = *reinterpret_cast<const uint4 *>(codes + ((q ^ swz) << 4));
                // the unit's groups: scales, and zero points as nibbles from the unit's first group on
                const int g0 = ((u * kUnit) >> g.gshift) % kChunk;
                const __half *sc = reinterpret_cast<const __half *>(sz) + g0;
                const uint32_t zz = (*reinterpret_cast<const uint16_t *>(sz + 32 + (g0 >> 2) * 2)) >> (4 * (g0 & 3));
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // 32 codes of one group (beyond K: zero scales)
                    const int i = (q * 32) >> g.gshift;
                    uint32_t out[16];
                    decode32<false>(c4[q], (zz >> (i * 4)) & 15u, __half2half2(sc[i]), out);
                    tmem_st16(slots + slot * kSlotCols + q * 16, out);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(code_empty(rc.s));
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(a_full(slot));
            }
            before += jobs;
            chunk += static_cast<uint32_t>(((s.k1 - 1) >> chunk_shift) - first_chunk) + 1;
        }
        while (ok && held < chunk) take_chunk();   // the other groups need the chunks after this group's last
    }
    // ---- every role is done; MMAs complete before tensor memory is freed ----
    __syncthreads();
    if (warp == 1) {
        mbar_wait(done_bar, 0, 50ull * 1000 * 1000);
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

}  // namespace q4
