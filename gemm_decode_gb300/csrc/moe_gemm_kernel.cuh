// moe_gemm_kernel.cuh -- device code of the matrix product grouped by expert (tcgen05).
//
//   y[r] = W_e x[rows[r]],  r in [offsets[e], offsets[e+1]),  w = (q - z) s
//
// The weights are the MMA's A operand (128 weight rows are the 128 lanes of tensor memory)
// and the rows of x its B operand, so a group of any size pads to 16 rows, not to 128.
//
// Numbers.  A first kernel (moe_prepare_kernel) writes each row of x as binary16 parts of
// x 2^e with 2^14 <= max |x| 2^e < 2^15: one part carries bfloat16 exactly, two carry
// binary32 to 22 bits, whatever the row's range.  (q - z) is exact in binary16 and times s
// it is rounded once; with two parts the remainder of that rounding is a second binary16
// number, exactly (the product has 15 bits).  Products are exact and sums binary32 in
// tensor memory.  PARTS = 1 accumulates w x.  PARTS = 2 accumulates w_hi x_hi in one set of
// columns and w_hi x_lo + w_lo x_hi in a second (what is left out is 2^-22 of the product);
// both weights see x_hi and x_lo as adjacent rows of one operand, so the first costs no MMA
// of its own.  The tensor core cuts what its binary32 sums cannot hold (measured: 2e-8 of
// the sum per MMA, all in one direction), so with two parts the epilogue takes the sums
// over every kDrain units and adds them in registers, rounding to nearest.
//
// Work.  An item is 128 * RT weight rows by up to NT rows of one expert; its K is cut into
// units of 128.  When items are many each CTA takes whole items; when the last wave of
// items would leave SMs idle, the units of all items are laid end to end and every CTA
// takes the same number of them.  A CTA that does not hold an item's whole K stores its
// partial sums; the CTA that arrives last adds them in the order of K (so the result does
// not depend on who is last) and finishes the item.  Nobody waits for another CTA.
//
// One CTA per SM:
//   warp 0      bulk tensor copies of the codes of a unit (128 * RT rows x 64 bytes) into a
//               ring, several units ahead: what keeps HBM busy
//   warp 1      issues the MMAs, operand A from tensor memory: the whole warp walks the
//               loop and one elected lane issues a unit's MMAs in a row (issued from a
//               branch on one lane, with a commit after every four, an MMA took 107 cycles;
//               this way 24, and 16 is what the tensor core needs for up to 32 columns)
//   warps 2, 3  load scales and zero points, 16 groups per row at a time, and leave them
//               in shared memory as one word (s, z) per group and row, rows adjacent
//   next 4 RT   epilogue, four warps per weight tile: tensor memory -> scale, SwiGLU, rounding, store; partial sums
//   next 4      copy the rows of x of each unit, by index (16-byte asynchronous copies: a
//               bulk copy of four rows by index took a lane 80 to 140 cycles to issue)
//   the rest    dequantisers, four warps (128 rows) per unit and weight tile: a thread owns
//               a row, reads 64 bytes of codes and writes 128 weights into 64 columns of
//               tensor memory, where the MMA reads them -- no trip through shared memory
// A word of eight codes in natural order yields the pairs (0,4), (1,5), (2,6), (3,7) with
// one logic operation each; the prepared x has its elements in that order.
//
// Every wait is bounded; on expiry the CTA raises the device status word, waits for its
// copies in flight and returns.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "q4_moe.cuh"
#include "q4_tc.cuh"

namespace q4 {

using namespace tc;

constexpr int kUnit = 128;     // k per unit: 64 bytes of codes per row
constexpr int kHalf = 64;      // k per 128 bytes of binary16, a row of the swizzled tile of x
constexpr int kChunk = 16;     // groups per row that the scale loader brings at a time
constexpr int kSlotCols = 64;  // tensor-memory columns of 128 weights per lane
constexpr int kDrain = 2;      // units between the epilogue's additions in registers (PARTS = 2)
constexpr int kTmemCols = 512;

struct MoeKernelArgs {
    const uint16_t *scales;
    const uint8_t *zeros;
    const int *rows, *offsets;
    const __half *xparts;    // [PARTS][Tx + 1][K] prepared x (row Tx: zeros)
    const float *xscale;     // [Tx + 1] 2^-e of each prepared row
    void *y;
    float *partial;          // two slots of 128 RT x NT per CTA
    unsigned int *arrived;   // RT counters per CTA, zeroed by the first kernel
    int E, R, Tx, N, K, nb, zrow, gshift;   // group = 2^gshift
    int swiglu;
    int wide_scales, wide_zeros;   // rows of scales / zero points allow 16- / 8-byte loads
    unsigned long long timeout_ns;
    unsigned int *status;
    unsigned int *bounds;
};

template <int PARTS, int RT, int NT>
struct MoeShape {
    static_assert(PARTS == 1 || RT == 1, "two parts: the epilogue holds one tile's sums in registers");
    static constexpr int kGroups = PARTS == 2 && NT > 32 ? 2 : 3;   // dequantiser groups of four warps
    static constexpr int kXWarp = 4 + 4 * RT;                  // first of the four that copy x
    static constexpr int kDqWarp = kXWarp + 4;                 // first dequantiser
    static constexpr int kWarps = kDqWarp + 4 * kGroups;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kAccCols = RT * PARTS * NT;           // one accumulator set
    static constexpr int kAccs = kAccCols <= 128 ? 2 : 1;      // sets of accumulators
    static constexpr int kSlots = (kTmemCols - kAccs * kAccCols) / kSlotCols;
    static constexpr int kCodeBytes = RT * 128 * (kUnit / 2);
    static constexpr int kCodeStages = RT == 2 ? 3 : (NT == 32 ? 10 : 6);
    // A dequantiser group skips the jobs of the others, and a wait by parity tells a phase
    // from the one before it only.  So the ring of weights holds a job per group (the job a
    // group finished last then lies within the ring), and no more units than the codes' ring
    // (a free slot of weights then proves that the codes' previous use has landed).
    static constexpr int kJobs = kSlots / PARTS;
    static_assert(kSlots % PARTS == 0 && kGroups <= kCodeStages, "whole jobs; a group's next unit within the codes' ring");
    static_assert(kGroups <= kJobs && kJobs <= RT * kCodeStages, "a parity could be taken for an older phase's");
    static constexpr int kXHalf = PARTS * NT * 128;            // rows of x, 64 k
    static constexpr int kXBytes = 2 * kXHalf;
    static constexpr int kXStages = kXBytes <= 8192 ? 8 : (kXBytes <= 16384 ? 6 : 4);
    static constexpr int kScaleBytes = kChunk * RT * 128 * 4;
    static constexpr int kScaleBufs = 2;
    static constexpr int kBars = 2 * (kCodeStages + kXStages + kScaleBufs + kSlots + kAccs * RT) + 1;
    static constexpr size_t fixed() {
        return 1024 + static_cast<size_t>(kXStages) * kXBytes + static_cast<size_t>(kCodeStages) * kCodeBytes +
               static_cast<size_t>(kScaleBufs) * kScaleBytes + 8 * kBars + RT * 2 * NT * 4 + 4 * NT * 4 + 64;
    }
    static constexpr size_t smem(int E) { return fixed() + 8 * (static_cast<size_t>(E) + 1); }
};

// Whether the phase of the given parity is complete, without suspending.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
// 16 bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float *f) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }
// (a & mask) | magic in one operation
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
    return r;
}

// The items of the call and this CTA's share of their units.
struct MoePlan {
    const int *first_row;   // [E + 1] shared: first row of each expert
    const int *first_tile;  // [E + 1] shared: first tile of rows of each expert
    uint32_t E, row_groups, units;   // tiles of weight rows per expert, units per item
    uint32_t items, ctas;   // ctas: CTAs that take part
    bool whole;             // CTAs take whole items
    uint32_t at, end;       // items (whole) or units left to this CTA

    __device__ __forceinline__ uint32_t begin_of(uint32_t c) const {
        return static_cast<uint32_t>(static_cast<uint64_t>(items) * units * c / ctas);
    }
    // the CTA that holds unit u
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(u + 1) * ctas - 1) / (items * units));
    }
};

struct MoeSegment {
    int expert, group, row0, rows;   // rows [row0, row0 + rows) of the expert's group of rows
    int k0, k1;                      // units
    uint32_t item;
};

template <int NT>
__device__ __forceinline__ bool next_segment(MoePlan &p, MoeSegment &s) {
    if (p.at >= p.end) return false;
    if (p.whole) {
        s.item = p.at;
        s.k0 = 0;
        s.k1 = static_cast<int>(p.units);
        p.at += p.ctas;
    } else {
        s.item = p.at / p.units;
        s.k0 = static_cast<int>(p.at - s.item * p.units);
        s.k1 = static_cast<int>(min(p.units, s.k0 + (p.end - p.at)));
        p.at += static_cast<uint32_t>(s.k1 - s.k0);
    }
    const int tile = static_cast<int>(s.item / p.row_groups);
    s.group = static_cast<int>(s.item - static_cast<uint32_t>(tile) * p.row_groups);
    int lo = 0, hi = static_cast<int>(p.E);   // the expert with first_tile[e] <= tile < first_tile[e + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.first_tile[mid] <= tile) lo = mid;
        else hi = mid;
    }
    s.expert = lo;
    s.row0 = p.first_row[lo] + (tile - p.first_tile[lo]) * NT;
    s.rows = min(p.first_row[lo + 1] - s.row0, NT);
    return true;
}

// One lane of running ring position: stage and the parity its barrier is waited for with.
template <int STAGES>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
        if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
        }
    }
    __device__ __forceinline__ void step(int n) {   // n <= STAGES
        s += n;
        if (s >= STAGES) {
            s -= STAGES;
            ph ^= 1u;
        }
    }
};

// The parts of x, scaled by a power of two per row, elements permuted within eights;
// row Tx is zeros.  Also clears the arrival counters of the product.
template <bool BF16>
__global__ void __launch_bounds__(256) moe_prepare_kernel(const void *x, int Tx, int K, __half *parts, float *xscale,
                                                          unsigned int *arrived, int counters) {
    __shared__ float warp_high[8];
    wait_prior_grid();
    allow_next_grid();
    const int row = blockIdx.x;
    if (row == 0)
        for (int i = threadIdx.x; i < counters; i += blockDim.x) arrived[i] = 0u;
    const int64_t base = static_cast<int64_t>(row) * K;
    __half *hi = parts + base, *lo = parts + static_cast<int64_t>(Tx + 1) * K + base;
    const int eights = K / 8;
    auto load8 = [&](int c, float *v) {
        if constexpr (BF16) {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(x) + base + 8 * c);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + base + 8 * c);
            const float4 a = p[0], b = p[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
    };
    if (row == Tx) {
        for (int c = threadIdx.x; c < eights; c += blockDim.x) {
            reinterpret_cast<uint4 *>(hi)[c] = make_uint4(0, 0, 0, 0);
            if (!BF16) reinterpret_cast<uint4 *>(lo)[c] = make_uint4(0, 0, 0, 0);
        }
        if (threadIdx.x == 0) xscale[row] = 1.0f;
        return;
    }
    float high = 0.0f;
    for (int c = threadIdx.x; c < eights; c += blockDim.x) {
        float v[8];
        load8(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) high = fmaxf(high, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(~0u, high, o));
    if ((threadIdx.x & 31) == 0) warp_high[threadIdx.x >> 5] = high;
    __syncthreads();
    high = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) high = fmaxf(high, warp_high[w]);
    // 2^e, e = 14 - floor(log2(high)), at most 126 (a row of subnormals keeps its bits)
    int e = 0;
    if (high > 0.0f && high <= 3.4028235e38f) {
        e = 14 - ilogbf(high);
        e = e > 126 ? 126 : e;
    }
    const float scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    if (threadIdx.x == 0) xscale[row] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    for (int c = threadIdx.x; c < eights; c += blockDim.x) {
        float v[8];
        load8(c, v);
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = v[i] * scale, b = v[i + 4] * scale;   // pairs (0,4), (1,5), (2,6), (3,7)
            const __half2 p = __floats2half2_rn(a, b);
            h[i] = as_u32(p);
            if (!BF16) l[i] = as_u32(__floats2half2_rn(a - __low2float(p), b - __high2float(p)));
        }
        reinterpret_cast<uint4 *>(hi)[c] = make_uint4(h[0], h[1], h[2], h[3]);
        if (!BF16) reinterpret_cast<uint4 *>(lo)[c] = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

template <int PARTS, int RT, int NT>
__global__ void __launch_bounds__(MoeShape<PARTS, RT, NT>::kThreads, 1)
moe_gemm_kernel(const __grid_constant__ CUtensorMap map_codes, const MoeKernelArgs g) {
    using S = MoeShape<PARTS, RT, NT>;
    static_assert(S::smem(kMaxExperts) <= 227 * 1024, "shared memory of one CTA");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *x_ring = smem;
    unsigned char *code_ring = x_ring + S::kXStages * S::kXBytes;
    uint32_t *scale_ring = reinterpret_cast<uint32_t *>(code_ring + S::kCodeStages * S::kCodeBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<unsigned char *>(scale_ring) +
                                                  S::kScaleBufs * S::kScaleBytes);
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
    auto d_empty = [&](int s) { return bar0 + 8u * (kD + S::kAccs * RT + s); };
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
        for (int s = 0; s < S::kAccs * RT; ++s) {
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
    if (warp == 2) {
        // rows and tiles of each expert: offsets clamped to [0, R] and never falling
        int row_carry = min(max(g.offsets[0], 0), g.R), tile_carry = 0;
        if (lane == 0) {
            first_row[0] = row_carry;
            first_tile[0] = 0;
        }
        for (int e0 = 0; e0 < g.E; e0 += 32) {
            const int e = e0 + lane;
            int hi = e < g.E ? min(g.offsets[e + 1], g.R) : 0;
            hi = max(hi, row_carry);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(~0u, hi, o);
                if (lane >= o) hi = max(hi, n);
            }
            int lo = __shfl_up_sync(~0u, hi, 1);
            if (lane == 0) lo = row_carry;
            int tiles = e < g.E ? (hi - lo + NT - 1) / NT : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(~0u, tiles, o);
                if (lane >= o) tiles += n;
            }
            tiles += tile_carry;
            if (e < g.E) {
                first_row[e + 1] = hi;
                first_tile[e + 1] = tiles;
            }
            row_carry = __shfl_sync(~0u, hi, 31);
            tile_carry = __shfl_sync(~0u, tiles, 31);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
    allow_next_grid();

    MoePlan plan;
    plan.first_row = first_row;
    plan.first_tile = first_tile;
    plan.E = g.E;
    plan.row_groups = (g.N + 128 * RT - 1) / (128 * RT);
    plan.units = (g.K + kUnit - 1) / kUnit;
    plan.items = static_cast<uint32_t>(first_tile[g.E]) * plan.row_groups;
    {
        const uint32_t ctas = gridDim.x, waves = (plan.items + ctas - 1) / ctas;
        // whole items when the last wave wastes less than a tenth of the time (always from
        // eleven waves on, so items * units below stays within 32 bits)
        plan.whole = plan.items > 0 && static_cast<uint64_t>(waves) * ctas * 10 <= static_cast<uint64_t>(plan.items) * 11;
        if (plan.whole) {
            plan.ctas = ctas;
            plan.at = blockIdx.x;
            plan.end = plan.items;
        } else {
            plan.ctas = max(1u, min(ctas, plan.items * plan.units));
            plan.at = plan.end = 0;
            if (blockIdx.x < plan.ctas) {
                plan.at = plan.begin_of(blockIdx.x);
                plan.end = plan.begin_of(blockIdx.x + 1);
            }
        }
    }

    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(g.status, 1u);
    };
    // bounded wait; false (and the abort flag) on expiry or when another role gave up
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try(bar, parity)) return true;
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

    if (warp == 0) {
        // ------------------------------------------------------------ codes
        if (lane == 0) {
            Ring<S::kCodeStages> r;
            int64_t issued = 0;
            MoeSegment s;
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
            // (on abort) every copy in flight lands before the CTA may exit
            if (*abort_flag)
                for (int64_t j = issued > S::kCodeStages ? issued - S::kCodeStages : 0; j < issued; ++j)
                    mbar_wait(code_full(static_cast<int>(j % S::kCodeStages)),
                              static_cast<uint32_t>(j / S::kCodeStages) & 1u, 50ull * 1000 * 1000);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        Ring<S::kXStages> rx;
        Ring<S::kSlots> ra;
        Ring<S::kAccs> rd;
        MoeSegment s;
        bool ok = true;
        const uint64_t x_desc = umma_desc(smem_addr(x_ring));
        while (ok && next_segment<NT>(plan, s)) {
            const int n16 = (s.rows + 15) / 16 * 16;
            const uint32_t idesc = idesc_f16(false, 128, PARTS * n16), idesc_lo = idesc_f16(false, 128, n16);
            bool fresh = true;   // the accumulators hold nothing of this segment
            const int half_unit = g.K % kUnit != 0 && g.K % kUnit <= kHalf ? g.K / kUnit : -1;   // the unit of one half
            for (int u = s.k0; ok && u < s.k1; ++u) {
                const uint32_t acc = tmem + static_cast<uint32_t>(rd.s * S::kAccCols);
                const uint64_t xd = x_desc + static_cast<uint32_t>(rx.s) * (S::kXBytes / 16);
                const bool both = u != half_unit;
                const bool drain = u + 1 == s.k1 || (PARTS == 2 && (u + 1 - s.k0) % kDrain == 0);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {   // weights: rounded, then the remainder
                        // all the barriers of the step are looked at together: one after
                        // another, each costs the latency of its own round trip
                        const bool need_x = t == 0 && p == 0, need_d = fresh && p == 0;
                        const bool ra_ok = mbar_test(a_full(ra.s), ra.ph);
                        const bool rx_ok = !need_x || mbar_test(x_full(rx.s), rx.ph);
                        const bool rd_ok = !need_d || mbar_test(d_empty(rd.s * RT + t), rd.ph ^ 1u);
                        if (!__all_sync(~0u, ra_ok && rx_ok && rd_ok)) {
                            if (need_d && !wait(d_empty(rd.s * RT + t), rd.ph ^ 1u)) ok = false;
                            if (need_x && !wait(x_full(rx.s), rx.ph)) ok = false;
                            if (!wait(a_full(ra.s), ra.ph)) ok = false;
                            ok = __all_sync(~0u, ok);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        const uint32_t a = tmem + S::kAccs * S::kAccCols + ra.s * kSlotCols;
                        const uint32_t d = acc + t * NT + (p == 1 ? n16 : 0);
                        const uint32_t id = p == 1 ? idesc_lo : idesc;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)   // 16 k: 32 bytes of a row of x, 8 columns of weights
                                umma_f16_ts(d, a + kk * 8, xd + kk * 2, id, p > 0 || kk > 0 || !fresh ? 1u : 0u);
                            if (both) {
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_f16_ts(d, a + 32 + kk * 8, xd + S::kXHalf / 16 + kk * 2, id, 1u);
                            }
                            umma_commit(a_empty(ra.s));
                            if (t == RT - 1 && p == PARTS - 1) umma_commit(x_empty(rx.s));
                            if (drain && p == PARTS - 1) umma_commit(d_full(rd.s * RT + t));
                        }
                        __syncwarp();
                        ra.step();
                    }
                    if (!ok) break;
                }
                rx.step();
                fresh = drain;
                if (drain) rd.step();
            }
        }
        if (elect_one()) umma_commit(done_bar);   // every MMA issued (waited for before tensor memory is freed)
        __syncwarp();
    } else if (warp >= S::kXWarp && warp < S::kDqWarp) {
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
        MoeSegment s;
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
                if constexpr (S::kXStages == 4) r.ph ^= 1u;
                else r.step(4);
            }
            before += units;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (full >= 0) hand_over();
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales and zero points
        Ring<S::kScaleBufs> r;
        MoeSegment s;
        bool ok = true;
        while (ok && next_segment<NT>(plan, s)) {
            for (int c = s.k0 >> (g.gshift - 3); c <= (s.k1 - 1) >> (g.gshift - 3); ++c) {   // 2^(gshift - 3) units each
                if (!wait(sc_empty(r.s), r.ph ^ 1u)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                uint32_t *buf = scale_ring + r.s * (S::kScaleBytes / 4);
                const int g0 = c * kChunk;
#pragma unroll 1
                for (int b = (warp & 1) * 2; b < RT * 4; b += 4) {
                    uint4 sc[2][2];
                    uint2 zz[2];
                    // two rows per lane and warp at a time, all loads in flight together
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = s.group * (128 * RT) + (b + i) * 32 + lane;
                        sc[i][0] = sc[i][1] = make_uint4(0, 0, 0, 0);
                        zz[i] = g.zeros != nullptr ? make_uint2(0, 0) : make_uint2(0x88888888u, 0x88888888u);
                        if (n < g.N) {
                            const int64_t row = static_cast<int64_t>(s.expert) * g.N + n;
                            const uint16_t *sp = g.scales + row * g.nb + g0;
                            if (g.wide_scales) {
                                if (g0 < g.nb) sc[i][0] = *reinterpret_cast<const uint4 *>(sp);
                                if (g0 + 8 < g.nb) sc[i][1] = *reinterpret_cast<const uint4 *>(sp + 8);
                            } else {
                                uint32_t w[8] = {};
#pragma unroll
                                for (int j = 0; j < kChunk; ++j)
                                    if (g0 + j < g.nb) w[j >> 1] |= ldg_u16(sp + j) << (16 * (j & 1));
                                sc[i][0] = make_uint4(w[0], w[1], w[2], w[3]);
                                sc[i][1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                            if (g.zeros != nullptr) {
                                const uint8_t *zp = g.zeros + row * g.zrow + g0 / 2;
                                if (g.wide_zeros) {
                                    zz[i] = *reinterpret_cast<const uint2 *>(zp);
                                } else {
                                    uint32_t w[2] = {};
#pragma unroll
                                    for (int j = 0; j < 8; ++j)
                                        if (g0 / 2 + j < g.zrow) w[j >> 2] |= ldg_u8(zp + j) << (8 * (j & 3));
                                    zz[i] = make_uint2(w[0], w[1]);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w[8] = {sc[i][0].x, sc[i][0].y, sc[i][0].z, sc[i][0].w,
                                               sc[i][1].x, sc[i][1].y, sc[i][1].z, sc[i][1].w};
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) {
                            const uint32_t sv = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
                            const uint32_t zv = ((j < 8 ? zz[i].x : zz[i].y) >> (4 * (j & 7))) & 15u;
                            buf[j * (128 * RT) + (b + i) * 32 + lane] = sv | (zv << 16);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full(r.s));
                r.step();
            }
        }
    } else if (warp >= 4 && warp < S::kXWarp) {
        // ------------------------------------------------------------ epilogue
        const int rt = (warp - 4) >> 2;           // weight tile: four warps each
        const int t = threadIdx.x - 128 * (1 + rt);   // lane of tensor memory: weight row of the tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int cols = g.swiglu ? g.N >> 1 : g.N;
        using Out = typename std::conditional<PARTS == 1, __nv_bfloat16, float>::type;
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
            if constexpr (PARTS == 1) *p = __float2bfloat16_rn(v);
            else *p = v;
        };
        Ring<S::kAccs> rd;
        MoeSegment s;
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
                    // bfloat16 outputs: the fast exponential and division are off by 2^-20, the rounding by 2^-8
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
                        if (j0 + j < s.rows) mine[(j0 + j) * 128] = v[j];
                }
            };
            const uint32_t acc0 = tmem + lane_base + static_cast<uint32_t>(rt * NT);
            bool ok = true;
            if constexpr (PARTS == 1) {
                ok = all4(wait(d_full(rd.s * RT + rt), rd.ph));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = acc0 + static_cast<uint32_t>(rd.s * S::kAccCols);
#pragma unroll 1
                for (int j0 = 0; j0 < s.rows; j0 += 16) {
                    float v[16];
                    tmem_ld16(acc + j0, v);
                    emit(j0, v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(d_empty(rd.s * RT + rt));
                rd.step();
            } else {
                const int n16 = (s.rows + 15) / 16 * 16;
                float sum[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[j] = 0.0f;
                for (int u = s.k0; u < s.k1; u += kDrain) {
                    ok = all4(wait(d_full(rd.s), rd.ph));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = acc0 + static_cast<uint32_t>(rd.s * S::kAccCols);
#pragma unroll
                    for (int j0 = 0; j0 < NT; j0 += 16)
                        if (j0 < s.rows) {
                            float v[16];
                            tmem_ld16(acc + j0, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[j0 + j] += v[j];
                            tmem_ld16(acc + n16 + j0, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[j0 + j] += v[j];
                        }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(d_empty(rd.s));
                    rd.step();
                }
                if (!ok) break;
#pragma unroll
                for (int j0 = 0; j0 < NT; j0 += 16)
                    if (j0 < s.rows) emit(j0, sum + j0);
            }
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
    } else if (warp >= S::kDqWarp) {
        // ------------------------------------------------------------ dequantisers
        const int group_id = (warp - S::kDqWarp) >> 2;
        const int row = (warp & 3) * 32 + lane;   // weight row of the tile = lane of tensor memory
        const uint32_t slots = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + S::kAccs * S::kAccCols;
        // Jobs are (unit, weight tile) in the order the MMAs take them; this group takes every
        // kGroups-th, whatever segment it falls into.
        constexpr int G = S::kGroups;
        Ring<S::kCodeStages> rc;
        Ring<S::kScaleBufs> rs;
        Ring<S::kSlots> ra;
        ra.step(group_id * PARTS);
        uint32_t next = static_cast<uint32_t>(group_id), before = 0;   // the next job; jobs of earlier segments
        uint32_t chunk = 0, held = 0;                                  // chunks of earlier segments; chunks taken so far
        uint32_t unit_at = 0;                                          // unit whose codes are at rc
        MoeSegment s;
        bool ok = true;
        const int chunk_shift = g.gshift - 3;
        const int half_unit = g.K % kUnit != 0 && g.K % kUnit <= kHalf ? g.K / kUnit : -1;   // the unit of one half
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
                const int t = RT == 1 ? 0 : static_cast<int>((next - before) % RT);
                const int u = s.k0 + static_cast<int>((next - before) / RT);
                // the chunk of scales: every group passes through every chunk
                const uint32_t want = chunk + static_cast<uint32_t>((u >> chunk_shift) - first_chunk) + 1;
                while (ok && held < want) take_chunk();
                if (!ok) break;
                const uint32_t unit = next / RT;
                rc.step(static_cast<int>(unit - unit_at));
                unit_at = unit;
                // slots of this job: the rounded weights, then their remainders
                const int sa = ra.s, sb = ra.s + 1;   // kSlots is a multiple of PARTS
                if (!wait(a_empty(sa), ra.ph ^ 1u)) ok = false;   // before code_full: see MoeShape
                if (PARTS == 2 && !wait(a_empty(sb), ra.ph ^ 1u)) ok = false;
                if (!wait(code_full(rc.s), rc.ph)) ok = false;
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                ra.step(G * PARTS);
                const uint32_t *sbuf = scale_ring + rs.s * (S::kScaleBytes / 4) + row;
                const bool both = u != half_unit;
                tc_fence_after();
                const unsigned char *codes = code_ring + rc.s * S::kCodeBytes + t * (128 * kUnit / 2) + row * 64;
                uint4 c4[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    c4[q] = *reinterpret_cast<const uint4 *>(codes + ((q ^ swz) << 4));
                uint32_t sz[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sz[q] = sbuf[((u * kUnit + q * 32) >> g.gshift) % kChunk * (128 * RT) + t * 128];
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // 32 codes of one group
                    if (q >= 2 && !both) break;
                    const uint32_t w4[4] = {c4[q].x, c4[q].y, c4[q].z, c4[q].w};
                    const __half2 sc = as_half2(__byte_perm(sz[q], 0, 0x1010));
                    const uint32_t z = sz[q] >> 16;
                    const __half2 z0 = as_half2(0x64006400u + z * 0x00010001u);   // 1024 + z
                    const __half2 z1 = as_half2(0xD400D400u + z * 0x00100010u);   // -(64 + z)
                    const __half2 sixteenth = as_half2(0x2C002C00u);              // 1 / 16
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a = w4[w], b = a >> 8;
                        __half2 d[4];
                        d[0] = __hsub2(as_half2(and_or(a, 0x000F000Fu, 0x64006400u)), z0);
                        d[1] = __hfma2(as_half2(and_or(a, 0x00F000F0u, 0x64006400u)), sixteenth, z1);
                        d[2] = __hsub2(as_half2(and_or(b, 0x000F000Fu, 0x64006400u)), z0);
                        d[3] = __hfma2(as_half2(and_or(b, 0x00F000F0u, 0x64006400u)), sixteenth, z1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __half2 v = __hmul2(d[i], sc);
                            hi[4 * w + i] = as_u32(v);
                            if (PARTS == 2) lo[4 * w + i] = as_u32(__hfma2(d[i], sc, __hneg2(v)));
                        }
                    }
                    tmem_st16(slots + sa * kSlotCols + q * 16, hi);
                    if (PARTS == 2) tmem_st16(slots + sb * kSlotCols + q * 16, lo);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(code_empty(rc.s));
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(a_full(sa));
                    if (PARTS == 2) mbar_arrive(a_full(sb));
                }
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
