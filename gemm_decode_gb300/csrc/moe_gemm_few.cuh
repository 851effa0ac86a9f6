// moe_gemm_few.cuh -- matrix product grouped by expert, few rows per expert (decoding, and
// binary32 of any length).  Shared parts, and how the work is divided: moe_gemm_common.cuh.
//
// Operand A is the whole number (q - z), and each group of weights has sums of its own in
// tensor memory, which the epilogue takes out, multiplies by the group's s and adds in
// registers.  No weight is rounded, and half the arithmetic of the dequantisers falls away.
// With two parts of x (binary32), these are adjacent rows of operand B.  The tensor core
// cuts what its binary32 sums cannot hold (measured: 2e-8 of the sum per MMA, all in one
// direction); here it adds up no more than eight times.
//
// One CTA per SM, 28 warps (24 with 64 rows of x).  Unit n of the CTA's sequence of units:
//   warp 0       bulk tensor copy of its codes (128 rows x 64 bytes) into a ring, several
//                units ahead: what keeps HBM busy
//   warp 1       its MMAs: the whole warp walks the loop and one elected lane issues them in
//                a row (issued from a branch on one lane, with a commit after every four, an
//                MMA took 107 cycles; this way 24, and 16 is what the tensor core needs for
//                up to 32 columns), then one commit
//   warps 2, 3   scales and zero points, 16 groups per row at a time
//   warps 4-11   epilogue, two groups of four warps taking the items in turn: the sums of each
//                unit's groups from tensor memory into registers; at the end of an item scale,
//                SwiGLU, rounding and store, while the other group takes the next item's sums
//   warps 12-15  copy the rows of x, by index, one unit each in turn (16-byte asynchronous
//                copies: a bulk copy of four rows by index took a lane 80 to 140 cycles)
//   the rest     dequantisers, three groups (two with 64 rows of x) of four warps taking the units in turn: a thread
//                owns a weight row, reads 64 bytes of codes and writes 128 weights into 64
//                columns of tensor memory
// Two barriers per unit tie them together: ready[n] (weights written, rows of x landed, the
// accumulators' last sums taken out) starts the MMAs, and their commit arrives at done[n],
// which frees the weights' slot, the stage of x, and hands the sums to the epilogue.
//
// What bounds it: the warps' instructions and the latency of the hand-overs, not HBM.  Logic
// and binary16 arithmetic together issue 2.5 warp instructions per clock and SM (measured),
// so dequantisation alone takes 250 cycles per unit, where HBM would deliver one in 360; with
// the other roles beside it a unit takes about 730 (from the time below; 826 in a profile of
// half as many tokens, where dequantisation is 41 % of the instructions).  Measured: 8 experts
// of 28672 x 4096 (groups of 128), 48 tokens bfloat16: 144 us, 3.4 TB/s (0.50 of measured).
// Scaled weights and one sum over K, as in moe_gemm_many.cuh, took 152 us there; one epilogue
// group for all units 187 us; two MMA warps 160 us.
#pragma once

#include "moe_gemm_common.cuh"

namespace q4 {

template <int PARTS, int NT>
struct FewShape {
    // groups of dequantisers (64 rows of x: two, for the registers), of the epilogue
    static constexpr int kDq = NT == 64 ? 2 : 3, kEpi = 2;
    static constexpr int kEpiWarp = 4, kXWarp = 12, kDqWarp = 16;
    static constexpr int kFours = 4 + kDq;                     // groups of four warps
    static constexpr int kThreads = 128 * kFours;
    // registers per thread: what the launch gives, and the roles' shares
    static constexpr int kRegLaunch = 65536 / kThreads / 8 * 8, kRegMisc = 64, kRegCopy = 48, kRegDq = 64;
    static constexpr int kRegSums = (kFours * kRegLaunch - kRegMisc - kRegCopy - kDq * kRegDq) / kEpi / 8 * 8;
    static_assert(kRegMisc + kRegCopy + kDq * kRegDq + kEpi * kRegSums <= kFours * kRegLaunch, "more than the launch has");
    // Accumulators: half of tensor memory, as sets of one unit's sums (its groups of weights
    // times the columns of a group); at least two, one per epilogue group, and up to eight,
    // which the MMAs fill while the epilogue finishes an item.
    static constexpr int kAccCols = 256;
    static constexpr int kMostGroups = kAccCols / 2 / (PARTS * NT);   // of a unit
    static constexpr int kSlots = 4;                           // units of weights
    static_assert(kAccCols + kSlots * kSlotCols <= kTmemCols, "tensor memory");
    static constexpr int kCodeBytes = 128 * (kUnit / 2);
    static constexpr int kXHalf = PARTS * NT * 128;            // rows of x, 64 k
    static constexpr int kXBytes = 2 * kXHalf;
    static constexpr int kStages = kXBytes <= 8192 ? 8 : (kXBytes <= 16384 ? 6 : 4);   // x, ready, done
    static constexpr int kCodeStages = kXBytes <= 8192 ? 10 : (kXBytes <= 16384 ? 8 : 4);
    // A role that skips units waits by parity, which tells a phase from the one before it
    // only: what it waited for last must lie within the ring.  The copies of x step by four,
    // and a free slot of weights proves that the codes' previous use has landed.
    static_assert(kStages >= 4 && kStages % 2 == 0 && kSlots <= kStages && kSlots <= kCodeStages && kDq <= kSlots, "rings");
    static constexpr int kScaleBytes = 128 * kScaleRow;
    static constexpr int kScaleBufs = 4;
    static constexpr int kBars = 2 * (kCodeStages + kStages + kScaleBufs);
    static constexpr size_t fixed() {
        return 1024 + static_cast<size_t>(kStages) * kXBytes + static_cast<size_t>(kCodeStages) * kCodeBytes +
               static_cast<size_t>(kScaleBufs) * kScaleBytes + 8 * kBars + 2 * kEpi * NT * 4 + 4 * NT * 4 + 64;
    }
    static constexpr size_t smem(int E) { return fixed() + 8 * (static_cast<size_t>(E) + 1); }
};

template <int PARTS, int NT>
__global__ void __launch_bounds__(FewShape<PARTS, NT>::kThreads, 1)
moe_gemm_few_kernel(const __grid_constant__ CUtensorMap map_codes, const MoeKernelArgs g) {
    using S = FewShape<PARTS, NT>;
    using Out = typename std::conditional<PARTS == 1, __nv_bfloat16, float>::type;
    static_assert(S::smem(kMaxExperts) <= 227 * 1024, "shared memory of one CTA");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *x_ring = smem;
    unsigned char *code_ring = x_ring + S::kStages * S::kXBytes;
    unsigned char *scale_ring = code_ring + S::kCodeStages * S::kCodeBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(scale_ring + S::kScaleBufs * S::kScaleBytes);
    float *row_scale = reinterpret_cast<float *>(bars + S::kBars);   // [epilogue group][2][NT]
    int *x_rows = reinterpret_cast<int *>(row_scale + 2 * S::kEpi * NT);   // [4][NT] rows of x, a list per copying warp
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(x_rows + 4 * NT);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *last_flag = reinterpret_cast<int *>(tmem_slot + 2);         // [epilogue group]
    int *first_row = reinterpret_cast<int *>(tmem_slot + 4);         // [E + 1]
    int *first_tile = first_row + g.E + 1;                           // [E + 1]

    const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const unsigned long long limit = g.timeout_ns;
    auto ib = [&](bool ok) { return q4_in_bounds(ok, g.bounds); };   // bounds-checking builds

    const uint32_t bar0 = smem_addr(bars);
    constexpr int kR = 2 * S::kCodeStages, kSc = kR + 2 * S::kStages;
    auto code_full = [&](int s) { return bar0 + 8u * s; };
    auto code_empty = [&](int s) { return bar0 + 8u * (S::kCodeStages + s); };
    auto ready = [&](int s) { return bar0 + 8u * (kR + s); };
    auto done = [&](int s) { return bar0 + 8u * (kR + S::kStages + s); };
    auto sc_full = [&](int s) { return bar0 + 8u * (kSc + s); };
    auto sc_empty = [&](int s) { return bar0 + 8u * (kSc + S::kScaleBufs + s); };

    const bool dq_scales = g.zeros != nullptr;   // the dequantisers read the chunks' zero points
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kCodeStages; ++s) {
            mbar_init(code_full(s), 1);
            mbar_init(code_empty(s), 4);
        }
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(ready(s), 4 + 1 + 4);   // dequantiser warps, the copying warp, epilogue warps
            mbar_init(done(s), 1);
        }
        for (int s = 0; s < S::kScaleBufs; ++s) {
            mbar_init(sc_full(s), 2);
            mbar_init(sc_empty(s), 4 + (dq_scales ? 4 * S::kDq : 0));   // one epilogue group, all dequantisers
        }
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
    MoePlan plan = make_plan<1>(g, first_row, first_tile);
    const int half_unit = g.K % kUnit != 0 && g.K % kUnit <= kHalf ? g.K / kUnit : -1;   // the unit of one half
    const int chunk_shift = g.gshift - 3;   // units per chunk of scales: 2^chunk_shift
    const int set_cols = (PARTS * NT * kUnit) >> g.gshift;                    // columns of a unit's sums
    const uint32_t sets = min(S::kAccCols / set_cols, S::kStages / 2 * 2);    // 2, 4 or 8 sets, taken in turn

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
    uint32_t units_issued = 0;   // warp 0 (lane 0): units whose codes are copied; warp 1: whose MMAs were issued

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegMisc));
        if (warp == 0) {
            // -------------------------------------------------------- codes
            if (lane == 0) {
                Ring<S::kCodeStages> r;
                MoeSegment s = {};
                bool ok = true;
                while (ok && next_segment<NT>(plan, s)) {
                    const int row = s.expert * g.N + s.group * 128;
                    for (int u = s.k0; u < s.k1; ++u) {
                        if (!wait(code_empty(r.s), r.ph ^ 1u)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(code_full(r.s), S::kCodeBytes);
                        tma_load_2d(smem_addr(code_ring + r.s * S::kCodeBytes), &map_codes, code_full(r.s),
                                    u * (kUnit / 2), row);
                        r.step();
                        ++units_issued;
                    }
                }
            }
            __syncwarp();
            // Every copy lands before the CTA may exit, whichever role gives up, and when: a flag
            // read here could be raised a moment later.  (Otherwise the copies are waited for
            // anyway, by the dequantisers.)  A lane per stage: one lane for all of them took
            // 0.8 us longer on 1024 binary32 tokens (112 us), behind the last barrier 2 us.
            const uint32_t copied = __shfl_sync(~0u, units_issued, 0);
            if (lane < S::kCodeStages && static_cast<uint32_t>(lane) < copied) {
                const uint32_t j = copied - 1 - lane;
                mbar_wait(code_full(static_cast<int>(j % S::kCodeStages)), (j / S::kCodeStages) & 1u, 50ull * 1000 * 1000);
            }
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA
            Ring<S::kStages> r;
            MoeSegment s = {};
            bool ok = true;
            const uint64_t x_desc = umma_desc(smem_addr(x_ring));
            auto segment = [&](auto per_group) {
                constexpr int PG = decltype(per_group)::value;   // MMAs per group of weights
                const uint32_t idesc = idesc_f16(false, 128, PARTS * ((s.rows + 15) / 16 * 16));
                for (int u = s.k0; u < s.k1; ++u) {
                    if (!__all_sync(~0u, mbar_test(ready(r.s), r.ph))) {
                        if (!wait(ready(r.s), r.ph)) ok = false;
                        ok = __all_sync(~0u, ok);
                        if (!ok) return;
                    }
                    tc_fence_after();
                    const uint64_t xd = x_desc + static_cast<uint32_t>(r.s) * (S::kXBytes / 16);
                    const uint32_t a = tmem + S::kAccCols + (units_issued % S::kSlots) * kSlotCols;
                    const uint32_t d = tmem + (units_issued & (sets - 1)) * set_cols;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // 16 k: 32 bytes of a row of x, 8 columns of weights
                            umma_f16_ts(d + kk / PG * (PARTS * NT), a + kk * 8, xd + kk * 2, idesc, kk % PG != 0);
                        if (u != half_unit) {
#pragma unroll
                            for (int kk = 4; kk < 8; ++kk)
                                umma_f16_ts(d + kk / PG * (PARTS * NT), a + kk * 8, xd + S::kXHalf / 16 + (kk - 4) * 2,
                                            idesc, kk % PG != 0);
                        }
                        umma_commit(done(r.s));
                    }
                    __syncwarp();
                    r.step();
                    ++units_issued;
                }
            };
            while (ok && next_segment<NT>(plan, s)) {
                if (S::kMostGroups == 1 || g.gshift == 7) segment(std::integral_constant<int, 8>());
                else if (S::kMostGroups == 2 || g.gshift == 6) segment(std::integral_constant<int, 4>());
                else segment(std::integral_constant<int, 2>());
            }
        } else {
            // -------------------------------------------------------- scales and zero points
            // Each warp 64 rows, two per lane.  Where the rows allow 8-byte accesses a chunk is
            // copied asynchronously, kAhead chunks before it is handed over: with groups of 32
            // a chunk lasts four units, less than the latency of one load after another.
            constexpr int kAhead = S::kScaleBufs - 2;
            Ring<S::kScaleBufs> r, full;
            int pending = 0;   // chunks copied and not handed over
            MoeSegment s = {};
            bool ok = true;
            auto hand_over = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full(full.s));
                full.step();
                --pending;
            };
            while (ok && next_segment<NT>(plan, s)) {
                for (int c = s.k0 >> chunk_shift; c <= (s.k1 - 1) >> chunk_shift; ++c) {
                    if (!__all_sync(~0u, mbar_test(sc_empty(r.s), r.ph ^ 1u))) {
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        while (pending > 0) hand_over();
                        if (!wait(sc_empty(r.s), r.ph ^ 1u)) ok = false;
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                    }
                    unsigned char *buf = scale_ring + r.s * S::kScaleBytes;
                    if (g.copy_scales) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int row = (warp & 1) * 64 + i * 32 + lane, n = s.group * 128 + row;
                            const bool have = n < g.N;
                            const int64_t at = static_cast<int64_t>(s.expert) * g.N + (have ? n : 0);
                            const uint32_t to = smem_addr(buf + row * kScaleRow);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int j = c * kChunk + 4 * q;   // four groups
                                const bool there = have && j < g.nb;
                                copy8(to + 8 * q, g.scales + at * g.nb + (there ? j : 0), there);
                            }
                            if (dq_scales) copy8(to + 32, g.zeros + at * g.zrow + c * (kChunk / 2), have);
                        }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        r.step();
                        if (++pending > kAhead) {
                            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
                            hand_over();
                        }
                    } else {
                        load_scales<1>(g, s.expert, s.group * 128, c, warp & 1, lane, buf);
                        r.step();
                        ++pending;
                        hand_over();
                    }
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            while (pending > 0) hand_over();
        }
    } else if (warp < S::kXWarp) {
        // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegSums));
        const int me = (warp - S::kEpiWarp) >> 2;                      // takes segments me, me + 2, ...
        const int t = (static_cast<int>(threadIdx.x) - 32 * S::kEpiWarp) & 127;   // lane of tensor memory: weight row
        const int cols = g.swiglu ? g.N >> 1 : g.N;
        const uint32_t acc0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        auto sync4 = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + me) : "memory"); };
        auto put = [&](Out *p, float v, bool have) {
            if (!have || !ib(p >= static_cast<Out *>(g.y) && p < static_cast<Out *>(g.y) + static_cast<int64_t>(g.R) * cols)) return;
            if constexpr (PARTS == 1) *p = __float2bfloat16_rn(v);
            else *p = v;
        };
        if (me == 0)
            for (uint32_t n = 0; n < sets; ++n)   // every set is free
                if (lane == 0) mbar_arrive(ready(n));
        uint32_t before = 0, chunk = 0;   // units and chunks of earlier segments
        MoeSegment s = {};
        int buf = 0;
        bool ok = true;
        float sum[NT];
        // The segment's units, kMostGroups groups of weights at a time: one wait and one round
        // of arrivals for up to four units (one at a time, a unit took 940 cycles).
        auto drain = [&]() {
            constexpr int MG = S::kMostGroups;
            const int lg = 7 - g.gshift;                      // a unit has 2^lg groups
            const int n16 = (s.rows + 15) & ~15;
            const int chunk0 = s.k0 >> chunk_shift, in_chunk = (1 << chunk_shift) - 1;
            uint32_t unit = before;
            const __half *sc = nullptr;
            for (int u = s.k0; u < s.k1;) {
                const uint32_t c = chunk + static_cast<uint32_t>((u >> chunk_shift) - chunk0);
                if (u == s.k0 || (u & in_chunk) == 0) {   // the next chunk of scales
                    if (ok && !wait(sc_full(c % S::kScaleBufs), c / S::kScaleBufs & 1u)) ok = false;
                    sc = reinterpret_cast<const __half *>(scale_ring + c % S::kScaleBufs * S::kScaleBytes + t * kScaleRow);
                }
                const int units = min(min(MG >> lg, s.k1 - u), in_chunk + 1 - (u & in_chunk));
                const bool half = u + units - 1 == half_unit;
                const int groups = (units << lg) - (half ? 1 << lg >> 1 : 0);
                const uint32_t last = unit + units - 1;
                if (ok && !wait(done(last % S::kStages), last / S::kStages & 1u)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                const __half *sg = sc + ((u << lg) & (kChunk - 1));
                auto at = [&](int i) {   // the sums of group i
                    return acc0 + ((unit + (i >> lg)) & (sets - 1)) * static_cast<uint32_t>(set_cols) +
                           (i & ((1 << lg) - 1)) * (PARTS * NT);
                };
                if constexpr (MG == 1) {
                    const float w0 = __half2float(sg[0]);
#pragma unroll
                    for (int j0 = 0; j0 < NT; j0 += 16)
                        if (j0 < s.rows) {
                            float v[16];
                            tmem_ld16(at(0) + j0, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[j0 + j] = fmaf(w0, v[j], sum[j0 + j]);
                            if constexpr (PARTS == 2) {   // from the second part of x
                                tmem_ld16(at(0) + n16 + j0, v);
#pragma unroll
                                for (int j = 0; j < 16; ++j) sum[j0 + j] = fmaf(w0, v[j], sum[j0 + j]);
                            }
                        }
                } else {
#pragma unroll 1   // (straight-line code would crowd the instruction cache)
                    for (int i = 0; i < MG; i += 2)   // two groups, their loads in flight together
                        if (i < groups) {
                            const bool two = i + 1 < groups;
                            const uint32_t a0 = at(i), a1 = two ? at(i + 1) : a0;
                            const float w0 = __half2float(sg[i]), w1 = two ? __half2float(sg[i + 1]) : 0.0f;
                            if constexpr (PARTS == 1) {
#pragma unroll
                                for (int j0 = 0; j0 < NT; j0 += 16)
                                    if (j0 < s.rows) {
                                        float v0[16], v1[16];
                                        tmem_ld16x2(a0 + j0, a1 + j0, v0, v1);
#pragma unroll
                                        for (int j = 0; j < 16; ++j)
                                            sum[j0 + j] = fmaf(w1, v1[j], fmaf(w0, v0[j], sum[j0 + j]));
                                    }
                            } else {
#pragma unroll
                                for (int j0 = 0; j0 < NT; j0 += 8)
                                    if (j0 < s.rows) {
                                        float v0[8], c0[8], v1[8], c1[8];
                                        tmem_ld8x4(a0 + j0, a0 + n16 + j0, a1 + j0, a1 + n16 + j0, v0, c0, v1, c1);
#pragma unroll
                                        for (int j = 0; j < 8; ++j)
                                            sum[j0 + j] = fmaf(w1, v1[j] + c1[j], fmaf(w0, v0[j] + c0[j], sum[j0 + j]));
                                    }
                            }
                        }
                }
                tc_fence_before();
                __syncwarp();
                // each set is free for the unit that comes `sets` later
                if (lane < units) mbar_arrive(ready(static_cast<int>((unit + lane + sets) % S::kStages)));
                unit += units;
                u += units;
                if (lane == 0 && (u == s.k1 || (u & in_chunk) == 0)) mbar_arrive(sc_empty(c % S::kScaleBufs));
            }
        };
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
                    // (bfloat16: the fast exponential and division are off by 2^-20, the rounding by 2^-8)
                    h[j / 2] = PARTS == 1 ? __fdividef(gate, 1.0f + __expf(-gate)) * up : gate / (1.0f + expf(-gate)) * up;
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
        // After a failed wait the groups go on through the barriers they share, without
        // waiting for anything else and without storing.
        for (int turn = 0; next_segment<NT>(plan, s); turn ^= 1) {
            const uint32_t units = static_cast<uint32_t>(s.k1 - s.k0);
            const uint32_t chunks = static_cast<uint32_t>(((s.k1 - 1) >> chunk_shift) - (s.k0 >> chunk_shift)) + 1;
            if (turn != me) {
                before += units;
                chunk += chunks;
                continue;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) sum[j] = 0.0f;
            float *scale = row_scale + (2 * me + buf) * NT;
            buf ^= 1;
            if (t < NT) {
                float f = 0.0f;
                if (t < s.rows) {
                    int src = g.rows != nullptr ? g.rows[s.row0 + t] : s.row0 + t;
                    if (src < 0 || src >= g.Tx) src = g.Tx;
                    f = g.xscale[src];
                }
                scale[t] = f;
            }
            // the other group has taken the sums of the segment before (barriers 3, 4)
            if (before > 0) asm volatile("bar.sync %0, 256;" ::"r"(3 + me) : "memory");
            sync4();   // the row scales are there
            drain();
            before += units;
            chunk += chunks;
            if (plan.at < plan.end) asm volatile("bar.arrive %0, 256;" ::"r"(4 - me) : "memory");
            const int n = s.group * 128 + t;
            if (s.k1 - s.k0 == static_cast<int>(plan.units)) {
                if (ok)
#pragma unroll
                    for (int j0 = 0; j0 < NT; j0 += 16)
                        if (j0 < s.rows) finish(n, j0, sum + j0, scale);
                continue;
            }
            // this CTA holds part of an item's K: its sums go to a slot of their own
            const uint32_t u0 = s.item * plan.units;
            const uint32_t c0 = plan.owner(u0), c1 = plan.owner(u0 + plan.units - 1);
            auto slot_of = [&](uint32_t c) {
                return g.partial + (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * (128 * NT) + t;
            };
            float *mine = slot_of(blockIdx.x);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (j < s.rows && ib(mine + j * 128 < g.partial + static_cast<int64_t>(2 * gridDim.x) * 128 * NT)) mine[j * 128] = sum[j];
            __threadfence();
            sync4();
            if (t == 0) last_flag[me] = atomicAdd(g.arrived + c0, 1u) == c1 - c0;
            sync4();
            if (last_flag[me] != 0 && ok) {
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
    } else if (warp < S::kDqWarp) {
        // ------------------------------------------------------------ rows of x
        // The four warps take the units in turn.  Eight lanes copy the 128 bytes of a row's
        // 64 k, 16 bytes each, to where the 128-byte swizzle wants them.  A unit is handed
        // over when its copies have landed: after the warp's next unit has been issued if
        // there is room for that already, else before the warp waits for room.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegCopy));
        const int me = warp - S::kXWarp;
        Ring<S::kStages> r;
        r.step(me);
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
            if (lane == 0) mbar_arrive(ready(full));
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
                if (!__all_sync(~0u, mbar_test(done(r.s), r.ph ^ 1u))) {
                    if (full >= 0) {
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        hand_over();
                        full = -1;
                    }
                    if (!wait(done(r.s), r.ph ^ 1u)) ok = false;
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                }
                const int k = u * kUnit + chunk * 8;
                const uint32_t dst = x_base + r.s * S::kXBytes;
                const bool have0 = k < g.K, have1 = k + kHalf < g.K;
                const __half *from = g.xparts + (have0 ? k : 0);
#pragma unroll 2
                for (int j = sub; j < n16; j += 4) {
                    if (!ib(list[j] >= 0 && list[j] <= g.Tx && r.s * S::kXBytes + 2 * S::kXHalf <= S::kStages * S::kXBytes)) continue;
                    const __half *row = from + static_cast<int64_t>(list[j]) * g.K;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {   // the second part's rows follow the first's
                        const uint32_t to = dst + sw128_offset(p * n16 + j, chunk);
                        copy16(to, row, have0);
                        copy16(to + S::kXHalf, row + (have1 ? kHalf : 0), have1);
                        row += static_cast<int64_t>(g.Tx + 1) * g.K;
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (full >= 0) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    hand_over();
                }
                full = r.s;
                r.step(4);
            }
            before += units;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (full >= 0) hand_over();
    } else {
        // ------------------------------------------------------------ dequantisers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegDq));
        constexpr int G = S::kDq;
        const int me = (warp - S::kDqWarp) >> 2;   // takes units me, me + kDq, ...
        const int row = (warp & 3) * 32 + lane;    // weight row of the tile = lane of tensor memory
        const uint32_t slots = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + S::kAccCols;
        Ring<S::kCodeStages> rc;
        Ring<S::kStages> rd, r;    // unit next - kSlots, unit next
        Ring<S::kScaleBufs> rs;
        rc.step(me);
        rd.step(((me - S::kSlots) % G + G) % G);   // the group's first unit that takes a slot again, less kSlots
        r.step(me);
        uint32_t next = static_cast<uint32_t>(me), before = 0;   // the group's next unit; units of earlier segments
        uint32_t chunk = 0, held = 0;                            // chunks of earlier segments; chunks taken so far
        MoeSegment s = {};
        bool ok = true;
        const int swz = (row >> 1) & 3;   // 64-byte swizzle: 16-byte chunk c of row r lies at c ^ ((r >> 1) & 3)
        bool holding = false;
        auto let_go = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_empty(rs.s));
            rs.step();
            holding = false;
        };
        auto take_chunk = [&]() {   // let go of the chunk held and wait for the next
            if (holding) let_go();
            ++held;
            holding = true;
            if (!wait(sc_full(rs.s), rs.ph)) ok = false;
            ok = __all_sync(~0u, ok);
        };
        while (ok && next_segment<NT>(plan, s)) {
            const uint32_t units = static_cast<uint32_t>(s.k1 - s.k0);
            const int first_chunk = s.k0 >> chunk_shift;
            for (; next - before < units; next += G) {
                const int u = s.k0 + static_cast<int>(next - before);
                if (dq_scales) {   // every group passes through every chunk
                    const uint32_t want = chunk + static_cast<uint32_t>((u >> chunk_shift) - first_chunk) + 1;
                    while (ok && held < want) take_chunk();
                    if (!ok) break;
                }
                if (next >= S::kSlots) {   // before code_full: see FewShape
                    if (!wait(done(rd.s), rd.ph)) ok = false;
                    rd.step(G);
                }
                if (!wait(code_full(rc.s), rc.ph)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                const unsigned char *codes = code_ring + rc.s * S::kCodeBytes + row * 64;
                const unsigned char *sz = scale_ring + rs.s * S::kScaleBytes + row * kScaleRow + 32;
                const uint32_t slot = slots + next % S::kSlots * kSlotCols;
                // 32 codes of one group at a time (beyond K: zero codes, which nothing reads)
                uint32_t zz = 0x8888u;
                if (dq_scales) {   // the zero points of the unit's groups: nibbles from the unit's first on
                    const int g0 = ((u * kUnit) >> g.gshift) % kChunk;
                    zz = (*reinterpret_cast<const uint16_t *>(sz + (g0 >> 2) * 2)) >> (4 * (g0 & 3));
                }
                uint4 c = *reinterpret_cast<const uint4 *>(codes + (swz << 4));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 now = c;
                    if (q < 3) c = *reinterpret_cast<const uint4 *>(codes + (((q + 1) ^ swz) << 4));
                    uint32_t out[16];
                    decode32<true>(now, (zz >> (((q * 32) >> g.gshift) * 4)) & 15u, __half2(), out);
                    tmem_st16(slot + q * 16, out);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(code_empty(rc.s));
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ready(r.s));
                rc.step(G);
                r.step(G);
                // at once when the group's next unit is not in the chunk
                if (dq_scales && (u + G >= s.k1 || (u + G) >> chunk_shift != u >> chunk_shift)) let_go();
            }
            before += units;
            chunk += static_cast<uint32_t>(((s.k1 - 1) >> chunk_shift) - first_chunk) + 1;
        }
        while (ok && dq_scales && held < chunk) take_chunk();   // the other readers need the chunks after this group's last
    }
    // ---- every role is done; MMAs complete before tensor memory is freed ----
    __syncthreads();
    if (warp == 1) {
        if (units_issued > 0)
            mbar_wait(done(static_cast<int>((units_issued - 1) % S::kStages)), ((units_issued - 1) / S::kStages) & 1u,
                      50ull * 1000 * 1000);
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

}  // namespace q4
