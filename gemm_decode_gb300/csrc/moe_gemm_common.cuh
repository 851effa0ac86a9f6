// moe_gemm_common.cuh -- what the two kernels of the matrix product grouped by expert share:
// arguments, the division of the work, the preparation of x, the loading of scales, and
// tensor-memory helpers.
//
//   y[r] = W_e x[rows[r]],  r in [offsets[e], offsets[e+1]),  w = (q - z) s
//
// The weights are the MMA's operand A (128 weight rows are the 128 lanes of tensor memory)
// and the rows of x its operand B, so a group of any size pads to 16 rows, not to 128.
// Dequantisers write the weights into tensor memory, where the MMA reads them, without a
// trip through shared memory.
//
// x.  A first kernel (moe_prepare_kernel) writes each row of x as binary16 parts of x 2^e
// with 2^14 <= max |x| 2^e < 2^15: one part carries bfloat16 exactly, two carry binary32 to
// 22 bits, as long as the parts stay above binary16's last step, 2^-24; half of that step,
// 2^-39 of the row's largest element, is lost of anything smaller.  (A power of two per unit
// of k would follow outliers closer, at a multiplication per sum and unit in the epilogue.)
// (q - z) is exact in binary16.
//
// Codes.  A word of eight codes in natural order yields the pairs (0,4), (1,5), (2,6), (3,7)
// with one logic operation each; the prepared x has its elements in that order.
//
// Work.  An item is 128 or 256 weight rows by up to NT rows of one expert; its K is cut into
// units of 128.  When items are many each CTA takes whole items; when the last wave of
// items would leave SMs idle, the units of all items are laid end to end and every CTA
// takes the same number of them.  A CTA that does not hold an item's whole K stores its
// partial sums; the CTA that arrives last adds them in the order of K (so the result does
// not depend on who is last) and finishes the item.  Nobody waits for another CTA.
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
constexpr int kTmemCols = 512;
constexpr int kScaleRow = 40;  // bytes of a row's chunk: 16 scales, 8 bytes of zero points
constexpr int kJoin = 28;      // units that joining partial sums takes as long as (measured: see make_plan)

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
    int copy_scales;               // rows of both allow 8-byte copies
    unsigned long long timeout_ns;
    unsigned int *status;
    unsigned int *bounds;
};

// 16 bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool have) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(have ? 8 : 0) : "memory");
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
__device__ __forceinline__ void tmem_ld16x2(uint32_t a0, uint32_t a1, float *f, float *h) {
    uint32_t v[16], w[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(w[0]),
          "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]), "=r"(w[8]), "=r"(w[9]),
          "=r"(w[10]), "=r"(w[11]), "=r"(w[12]), "=r"(w[13]), "=r"(w[14]), "=r"(w[15])
        : "r"(a0), "r"(a1)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        f[i] = __uint_as_float(v[i]);
        h[i] = __uint_as_float(w[i]);
    }
}
__device__ __forceinline__ void tmem_ld8x4(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, float *f0, float *f1,
                                           float *f2, float *f3) {
    uint32_t v[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%33];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%34];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24,%25,%26,%27,%28,%29,%30,%31}, [%35];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f0[i] = __uint_as_float(v[i]);
        f1[i] = __uint_as_float(v[8 + i]);
        f2[i] = __uint_as_float(v[16 + i]);
        f3[i] = __uint_as_float(v[24 + i]);
    }
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
        const uint32_t all = items * units, each = all / ctas;
        return each * c + (all - each * ctas) * c / ctas;   // floor(all * c / ctas) in 32 bits
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

// First row and first tile (of NT rows) of each expert, by one warp: offsets clamped to
// [0, R] and to no less than the one before.
template <int NT>
__device__ __forceinline__ void expert_tables(const MoeKernelArgs &g, int lane, int *first_row, int *first_tile) {
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

// This CTA's share; RT: weight tiles of 128 rows per item.
template <int RT>
__device__ __forceinline__ MoePlan make_plan(const MoeKernelArgs &g, const int *first_row, const int *first_tile) {
    MoePlan plan;
    plan.first_row = first_row;
    plan.first_tile = first_tile;
    plan.E = g.E;
    plan.row_groups = (g.N + 128 * RT - 1) / (128 * RT);
    plan.units = (g.K + kUnit - 1) / kUnit;
    plan.items = static_cast<uint32_t>(first_tile[g.E]) * plan.row_groups;
    {
        const uint32_t ctas = gridDim.x, waves = (plan.items + ctas - 1) / ctas;
        // whole items when sharing their units would save no more time than joining the parts
        // takes (always from sixteen waves on, so items * units below fits 32 bits).  With
        // kJoin = 7 / 14 / 28: a block of 2048 tokens 231 / 211 / 203 us, one of 8 tokens 85 /
        // 79 / 81 us, 1024 binary32 tokens 116 / 112 / 112 us, the other sizes alike.  One
        // number, whatever the parts hold (512 bytes to 128 KB per CTA): where they are small
        // it keeps SMs idle that a cheaper join would use
        plan.whole = plan.items > 0 && (waves >= 16 || static_cast<uint64_t>(waves) * ctas * plan.units <=
                                                           static_cast<uint64_t>(plan.items) * plan.units + kJoin * ctas);
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
    return plan;
}

// A chunk of scales and zero points of 128 RT weight rows from row n0 of the expert on, into
// shared memory, kScaleRow bytes per row; by two warps, each two rows per lane at a time with
// all their loads in flight together.  Rows and groups that do not exist: zero scales.
template <int RT>
__device__ __forceinline__ void load_scales(const MoeKernelArgs &g, int expert, int n0, int c, int pair, int lane,
                                            unsigned char *buf) {
    const int g0 = c * kChunk;
#pragma unroll 1
    for (int b = pair * 2; b < RT * 4; b += 4) {
        uint4 sc[2][2];
        uint2 zz[2];
        // two rows per lane and warp at a time, all loads in flight together
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = n0 + (b + i) * 32 + lane;
            sc[i][0] = sc[i][1] = make_uint4(0, 0, 0, 0);
            zz[i] = g.zeros != nullptr ? make_uint2(0, 0) : make_uint2(0x88888888u, 0x88888888u);
            if (n < g.N) {
                const int64_t row = static_cast<int64_t>(expert) * g.N + n;
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
            unsigned char *to = buf + ((b + i) * 32 + lane) * kScaleRow;
            *reinterpret_cast<uint2 *>(to) = make_uint2(sc[i][0].x, sc[i][0].y);
            *reinterpret_cast<uint2 *>(to + 8) = make_uint2(sc[i][0].z, sc[i][0].w);
            *reinterpret_cast<uint2 *>(to + 16) = make_uint2(sc[i][1].x, sc[i][1].y);
            *reinterpret_cast<uint2 *>(to + 24) = make_uint2(sc[i][1].z, sc[i][1].w);
            *reinterpret_cast<uint2 *>(to + 32) = zz[i];
        }
    }
}

// The (q - z) of 32 codes of one group, times s unless WHOLE, in the order of the prepared x.
template <bool WHOLE>
__device__ __forceinline__ void decode32(const uint4 &codes, uint32_t z, __half2 s, uint32_t *out) {
    const __half2 z0 = as_half2(0x64006400u + z * 0x00010001u);   // 1024 + z
    const __half2 z1 = as_half2(0xD400D400u + z * 0x00100010u);   // -(64 + z)
    const __half2 sixteenth = as_half2(0x2C002C00u);              // 1 / 16
    const uint32_t w4[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t a = w4[w], b = a >> 8;
        __half2 d[4];
        d[0] = __hsub2(as_half2(and_or(a, 0x000F000Fu, 0x64006400u)), z0);
        d[1] = __hfma2(as_half2(and_or(a, 0x00F000F0u, 0x64006400u)), sixteenth, z1);
        d[2] = __hsub2(as_half2(and_or(b, 0x000F000Fu, 0x64006400u)), z0);
        d[3] = __hfma2(as_half2(and_or(b, 0x00F000F0u, 0x64006400u)), sixteenth, z1);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[4 * w + i] = as_u32(WHOLE ? d[i] : __hmul2(d[i], s));
    }
}

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

}  // namespace q4
