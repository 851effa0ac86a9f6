// attn_many.cuh -- attention of many rows by the keys of a shared segment, on the tensor cores.
//
// A segment is up to 256 rows (queries times the query heads of one kv head, in two tiles of
// 128) by the keys, in tiles of 128 keys:
//   S = Q K^T      operands in shared memory (128-byte swizzle), sums in tensor memory
//   P = exp2(scale2 S - m)   a thread has a row: 128 scores from tensor memory to registers,
//                  their maximum, then the weights, rounded to 16 bits back over the scores' columns
//   O += P V       operand A in tensor memory, the values as they lie (their features side by
//                  side: the operand is read transposed)
// The maximum that a row's weights are relative to is renewed only when it has grown by more
// than a factor of 2^8: weights up to 2^8 round as well as ones below 1, sums are binary32, and
// the sums in tensor memory hardly ever have to be scaled.
// Both operands of a product are of one type, so a weight is rounded once to the cache's (the sums
// that divide are of the unrounded ones): outputs are off by 1.8-2.4e-3 (bf16) and 2.7e-4 (f16), 2-norm,
// where their own rounding alone is 1.7e-3 and 2.1e-4.  What the rounding takes off could be a second
// operand, for half as many MMAs again.
//
// One CTA per SM, twelve warps:
//   warp 0      bulk tensor copies: queries of a segment, tiles of keys and values in turn into
//               one ring of stages (a box per page, or 64 rows of one; a lane each)
//   warp 1      the MMAs: the warp walks the loop, one elected lane issues.  The scores of one
//               tile of rows are formed while the weights of the other are computed.
//   warps 4-7, 8-11  weights of the first and second tile of rows, and the results
// (warps 2 and 3 do nothing: registers are handed from the first four warps to the others by
// groups of four)
//
// What bounds it: a unit (256 rows by 128 keys of 128 features) takes 3100 cycles, of which the
// tensor core needs 2048 at its rate.  Without any waiting for weights its products take 2540:
// the operands of S, both in shared memory, are read at the 128 bytes a cycle that it gives, and
// the copies of keys and values write there too.  The other 560 are the hand-overs between the
// MMAs and the weights (weights without exponentials: 3050).  A segment's beginning and end cost
// about 2.4 units: the first scores and weights, and the results out of tensor memory.
// Measured (graphs): 256 queries x 32 heads by 27900 keys of 8 heads 94 us, 1.25 PFLOP/s (0.65 of
// measured bf16); a causal prompt of 4096 tokens 141-147 us with plan and join, 0.93-0.97 PFLOP/s.
// Results stored 16 bytes a lane instead of whole sectors: 26 us more for the prompt.
#pragma once

#include "attn_common.cuh"

namespace q4 {

// The weights of a tile are handed over in two parts: those of the first keys, whose products
// take as long as the other weights do.  Causal prompt of 4096 and 256 sequences (graphs): 141 and
// 160 us with 96 keys first, 145 and 163 with 64, 144 and 162 with all at once.
constexpr int kFirstKeys = 96;

template <int D>
struct ManyAttn {
    static constexpr int kThreads = 384;
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = kManyKeys * 128;            // 128 rows of 64 features
    static constexpr int kTileBytes = kHalves * kHalfBytes;       // queries of a tile, keys or values of one
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kBars = 2 * kStages + 14;   // (an even number: what follows is aligned to 16 bytes)
    static constexpr int kTmemCols = 512;
    // Registers that the roles have after the hand-over: a block launched with fewer would wait for
    // them without end, so the launch is refused where the kernel was not compiled to have them.
    static constexpr int kRegisters = 128 * 88 + 256 * 208;
    static constexpr size_t smem() {
        return 1024 + static_cast<size_t>(kManyTiles + kStages) * kTileBytes + 8 * kBars + sizeof(AttnHeld) + 16;
    }
};

// Shared-memory matrix descriptor of an operand whose rows are k and lie with 64 of its N
// elements side by side (128-byte swizzle): `next` bytes from one 64 N to the next, 1024 from
// one 8 k to the next.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t addr, uint32_t next) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(next >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// N columns of the warp's lanes.  The load and its wait are one statement: between two, the
// compiler may move or spill registers that the load has not filled yet.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float *f);
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t addr, float *f) {
    uint32_t *v = reinterpret_cast<uint32_t *>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld<64>(uint32_t addr, float *f) {
    uint32_t *v = reinterpret_cast<uint32_t *>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
          "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
          "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld<128>(uint32_t addr, float *f) {
    uint32_t *v = reinterpret_cast<uint32_t *>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
          "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
          "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63]),
          "=r"(v[64]), "=r"(v[65]), "=r"(v[66]), "=r"(v[67]), "=r"(v[68]), "=r"(v[69]), "=r"(v[70]), "=r"(v[71]),
          "=r"(v[72]), "=r"(v[73]), "=r"(v[74]), "=r"(v[75]), "=r"(v[76]), "=r"(v[77]), "=r"(v[78]), "=r"(v[79]),
          "=r"(v[80]), "=r"(v[81]), "=r"(v[82]), "=r"(v[83]), "=r"(v[84]), "=r"(v[85]), "=r"(v[86]), "=r"(v[87]),
          "=r"(v[88]), "=r"(v[89]), "=r"(v[90]), "=r"(v[91]), "=r"(v[92]), "=r"(v[93]), "=r"(v[94]), "=r"(v[95]),
          "=r"(v[96]), "=r"(v[97]), "=r"(v[98]), "=r"(v[99]), "=r"(v[100]), "=r"(v[101]), "=r"(v[102]), "=r"(v[103]),
          "=r"(v[104]), "=r"(v[105]), "=r"(v[106]), "=r"(v[107]), "=r"(v[108]), "=r"(v[109]), "=r"(v[110]), "=r"(v[111]),
          "=r"(v[112]), "=r"(v[113]), "=r"(v[114]), "=r"(v[115]), "=r"(v[116]), "=r"(v[117]), "=r"(v[118]), "=r"(v[119]),
          "=r"(v[120]), "=r"(v[121]), "=r"(v[122]), "=r"(v[123]), "=r"(v[124]), "=r"(v[125]), "=r"(v[126]), "=r"(v[127])
        : "r"(addr)
        : "memory");
}
// 32 bytes of a row, a sector in one go where it is aligned (each lane has a row of its own).
__device__ __forceinline__ void put32(void *to, const uint32_t *w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float *f) {
    tmem_st16(addr, reinterpret_cast<const uint32_t *>(f));
    tmem_st16(addr + 16, reinterpret_cast<const uint32_t *>(f) + 16);
}

template <typename C, int D>
__global__ void __launch_bounds__(ManyAttn<D>::kThreads, 1)
attn_many_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const AttnArgs g) {
    using M = ManyAttn<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *q_tiles = smem, *ring = smem + kManyTiles * M::kTileBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + M::kStages * M::kTileBytes);
    AttnHeld *held = reinterpret_cast<AttnHeld *>(bars + M::kBars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(held + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const unsigned long long limit_ns = g.timeout_ns;
    auto ib = [&](bool ok) { return q4_in_bounds(ok, g.bounds); };
    const uint32_t bar0 = smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (M::kStages + s); };
    auto other = [&](int i) { return bar0 + 8u * (2 * M::kStages + i); };
    const uint32_t q_full = other(0), q_empty = other(1), done = other(2);
    auto s_full = [&](int t) { return other(3 + t); };    // scores of a tile of rows are there
    auto p_full = [&](int t, int part) { return other(5 + 2 * t + part); };   // the weights of its first keys are, of all
    auto o_full = [&](int t) { return other(9 + t); };    // its results are
    auto o_empty = [&](int t) { return other(11 + t); };  // its results have been read
    if (threadIdx.x == 0) {
        for (int s = 0; s < M::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(done, 1);
        for (int t = 0; t < kManyTiles; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t, 0), 4);
            mbar_init(p_full(t, 1), 4);
            mbar_init(o_full(t), 1);
            mbar_init(o_empty(t), 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(M::kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
    wait_prior_grid();
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
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool { return __all_sync(~0u, wait(bar, parity)) != 0; };
    AttnWalk<kManyKeys, kManyCost, false> walk;
    {
        const AttnCounts many = counts_at(g.many), few = counts_at(g.few);
        walk.begin(many, g.many_entries, g.many_start, many_ctas_of(g, many.units, few.units), lane);
    }
    walk.hold(held);
    __syncthreads();
    AttnSegment s;
    auto next = [&]() { return walk.next(s, g.Hkv, g.G); };
    const uint32_t s_cols = 0, o_cols = kManyTiles * kManyKeys;   // tensor memory: scores, results

    // registers: 384 x 168 at the launch, 128 x 88 + 256 x 208 from here on
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
        // ------------------------------------------------------------ copies
        Ring<M::kStages> r;
        uint32_t q_ph = 0;
        int64_t issued = 0, queries = 0;
        const int boxes = kManyKeys >> g.box_shift, copies = M::kHalves * boxes;
        const int box = lane % boxes, half = lane / boxes;
        const uint32_t to = smem_addr(ring) + half * M::kHalfBytes + (box << g.box_shift) * 128;
        bool ok = true;
        while (ok && next()) {
            const int tiles = s.e.queries > g.tile_queries ? 2 : 1;
            const int *table = g.shared_pages + static_cast<int64_t>(s.e.group) * g.max_shared;
            auto page_of = [&](int u) {   // the lane's page of a tile of keys; one outside the pool reads as zeros
                const int key = u * kManyKeys + (box << g.box_shift);
                int id = g.pages;
                if (lane < copies && key < s.e.keys && ib((key >> g.page_shift) < g.max_shared))
                    id = table[key >> g.page_shift];
                return id < 0 || id > g.pages ? g.pages : id;
            };
            int page = page_of(s.u0);
            for (int u = s.u0; ok && u < s.u1; ++u) {
                const int after = u + 1 < s.u1 ? page_of(u + 1) : 0;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!ok || !wait_all(empty(r.s), r.ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_expect_tx(full(r.s), M::kTileBytes);
                    __syncwarp();
                    if (lane < copies)
                        tma_load_4d(to + r.s * M::kTileBytes, kv == 0 ? &map_k : &map_v, full(r.s), half * 64,
                                    (u * kManyKeys + (box << g.box_shift)) & (g.page - 1), s.head, page);
                    r.step();
                    ++issued;
                    if (u == s.u0 && kv == 0) {   // the queries, as soon as the segment before needs its own no more
                        if (!wait_all(q_empty, q_ph ^ 1u)) {
                            ok = false;
                            break;
                        }
                        q_ph ^= 1u;
                        if (lane == 0)
                            mbar_expect_tx(q_full, static_cast<uint32_t>(tiles * M::kHalves * g.tile_queries * g.G * 128));
                        __syncwarp();
                        if (lane < tiles * M::kHalves) {
                            const int t = lane / M::kHalves, h = lane - t * M::kHalves;
                            tma_load_3d(smem_addr(q_tiles) + t * M::kTileBytes + h * M::kHalfBytes, &map_q, q_full,
                                        h * 64, s.head * g.G, s.e.first + t * g.tile_queries);
                        }
                        ++queries;
                    }
                }
                page = after;
            }
        }
        // every copy lands before the CTA may exit, whichever role gives up
        for (int64_t j = issued > M::kStages ? issued - M::kStages : 0; j < issued; ++j)
            mbar_wait(full(static_cast<int>(j % M::kStages)), static_cast<uint32_t>(j / M::kStages) & 1u,
                      50ull * 1000 * 1000);
        if (queries > 0) mbar_wait(q_full, static_cast<uint32_t>(queries - 1) & 1u, 50ull * 1000 * 1000);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        Ring<M::kStages> r;
        uint32_t q_ph = 0, p_ph[2] = {0, 0}, oe_ph[2] = {0, 0};
        const uint32_t bf16 = std::is_same<C, __nv_bfloat16>::value;
        // a scale below zero: the products of the queries' negatives (bit 13)
        const uint32_t idesc_s = idesc_f16(bf16 != 0, 128, kManyKeys) | (g.scale2 < 0.0f ? 1u << 13 : 0u);
        const uint32_t idesc_o = idesc_f16(bf16 != 0, 128, D) | (1u << 16);   // operand B read transposed
        const uint64_t q_desc = umma_desc(smem_addr(q_tiles)), k_desc = umma_desc(smem_addr(ring));
        const uint64_t v_desc = umma_desc_mn(smem_addr(ring), M::kHalfBytes);
        auto scores = [&](int t, int stage) {   // by one lane
            const uint64_t a = q_desc + static_cast<uint32_t>(t) * (M::kTileBytes / 16);
            const uint64_t b = k_desc + static_cast<uint32_t>(stage) * (M::kTileBytes / 16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = (k / 4) * (M::kHalfBytes / 16) + (k % 4) * 2;
                umma_f16(tmem + s_cols + t * kManyKeys, a + at, b + at, idesc_s, k > 0 ? 1u : 0u);
            }
            umma_commit(s_full(t));
        };
        bool ok = true;
        while (ok && next()) {
            const int tiles = s.e.queries > g.tile_queries ? 2 : 1;
            if (!wait_all(q_full, q_ph)) break;
            q_ph ^= 1u;
            int ks = r.s;
            if (!wait_all(full(ks), r.ph)) break;
            r.step();
            tc_fence_after();
            if (elect_one()) {
                for (int t = 0; t < tiles; ++t) scores(t, ks);
                umma_commit(empty(ks));
                if (s.u1 - s.u0 == 1) umma_commit(q_empty);
            }
            __syncwarp();
            for (int u = s.u0; ok && u < s.u1; ++u) {
                const int vs = r.s;
                const uint32_t v_ph = r.ph;
                r.step();
                const bool more = u + 1 < s.u1;
                uint32_t k_ph = 0;
                if (more) {
                    ks = r.s;
                    k_ph = r.ph;
                    r.step();
                }
                for (int t = 0; t < tiles; ++t) {
                    if (t == 0) {
                        if (!wait_all(full(vs), v_ph)) {
                            ok = false;
                            break;
                        }
                        const int end = s.e.keys - u * kManyKeys;   // keys of the tile that are the segment's
                        if (end < kManyKeys) {
                            // the rows behind them, in the box that holds the last, are not: zeros, whatever they are
                            unsigned char *rows = ring + vs * M::kTileBytes;
                            const int from = end * 128, until = ((end + g.box - 1) >> g.box_shift << g.box_shift) * 128;
#pragma unroll
                            for (int h = 0; h < M::kHalves; ++h)
                                for (int b = from + lane * 16; b < until; b += 512)
                                    *reinterpret_cast<uint4 *>(rows + h * M::kHalfBytes + b) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async();
                            __syncwarp();
                        }
                    }
                    if (!wait_all(p_full(t, 0), p_ph[t]) || (u == s.u0 && !wait_all(o_empty(t), oe_ph[t] ^ 1u))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t b = v_desc + static_cast<uint32_t>(vs) * (M::kTileBytes / 16);
                    const uint32_t a = tmem + s_cols + t * kManyKeys, d = tmem + o_cols + t * D;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kFirstKeys / 16; ++k)
                            umma_f16_ts(d, a + k * 8, b + k * (2048 / 16), idesc_o, k > 0 || u > s.u0 ? 1u : 0u);
                    }
                    __syncwarp();
                    if (!wait_all(p_full(t, 1), p_ph[t]) || (more && t == 0 && !wait_all(full(ks), k_ph))) {
                        ok = false;
                        break;
                    }
                    p_ph[t] ^= 1u;
                    if (u == s.u0) oe_ph[t] ^= 1u;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = kFirstKeys / 16; k < kManyKeys / 16; ++k)
                            umma_f16_ts(d, a + k * 8, b + k * (2048 / 16), idesc_o, 1u);
                        if (!more) umma_commit(o_full(t));
                        else scores(t, ks);
                        if (t == tiles - 1) {
                            umma_commit(empty(vs));
                            if (more) umma_commit(empty(ks));
                            if (u + 2 == s.u1) umma_commit(q_empty);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (elect_one()) umma_commit(done);   // every MMA issued (waited for before tensor memory is freed)
        __syncwarp();
    }
    } else {
        // ------------------------------------------------------------ weights and results
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = (warp >> 2) - 1;                        // tile of rows
        const int row = (warp & 3) * 32 + lane;               // lane of tensor memory
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + s_cols + t * kManyKeys, o_at = tmem + lanes + o_cols + t * D;
        const float scale2 = fabsf(g.scale2);   // (a sign below zero is in the scores already)
        uint32_t s_ph = 0, o_ph = 0;
        bool ok = true;
        while (ok && next()) {
            const int tiles = s.e.queries > g.tile_queries ? 2 : 1;
            if (t >= tiles) continue;
            const int held = min(g.tile_queries, s.e.queries - t * g.tile_queries) * g.G;   // rows in use
            const bool have = row < held;
            int query, head;
            row_of(g, s, t * g.tile_queries * g.G + min(row, held - 1), query, head);
            const int limit = have && ib(query < g.S) ? limit_of(g, s, query) : 0;
            float m = neg_inf(), l = 0.0f;
            for (int u = s.u0; u < s.u1; ++u) {
                if (!wait_all(s_full(t), s_ph)) {
                    ok = false;
                    break;
                }
                s_ph ^= 1u;
                tc_fence_after();
                float x[kManyKeys];
                tmem_ld<kManyKeys>(s_at, x);
                const int seen = limit - u * kManyKeys;
                if (!__all_sync(~0u, seen >= kManyKeys || !have)) {
#pragma unroll
                    for (int c = 0; c < kManyKeys; ++c)
                        if (c >= seen) x[c] = neg_inf();
                }
                float top = max3(x[0], x[1], x[2]), top1 = max3(x[3], x[4], x[5]);
#pragma unroll
                for (int c = 6; c + 3 < kManyKeys; c += 4) {
                    top = max3(top, x[c], x[c + 1]);
                    top1 = max3(top1, x[c + 2], x[c + 3]);
                }
                top = scale2 * max3(top, top1, fmaxf(x[kManyKeys - 2], x[kManyKeys - 1]));
                const bool renew = have && (top > m + 8.0f || (m == neg_inf() && top > m));
                if (__any_sync(~0u, renew)) {
                    float f = 1.0f;
                    if (renew) {
                        f = exp2_fast(m - top);
                        m = top;
                        l *= f;
                    }
                    if (u > s.u0) {   // the sums so far (the scores are there, so the products before them are done)
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float v[32];
                            tmem_ld<32>(o_at + c, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= f;
                            tmem_st32(o_at + c, v);
                        }
                    }
                }
                // (the code of a tile's weights stands here once: fetching it is what a short call waits for)
                uint32_t p[kManyKeys / 2];
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                const float b = m == neg_inf() ? 0.0f : -m;
                const float2 base = make_float2(b, b), scale = make_float2(scale2, scale2);
                auto weigh = [&](int from, int until) {
#pragma unroll
                    for (int i = from; i < until; i += 2) {
                        const float2 y = __ffma2_rn(make_float2(x[i], x[i + 1]), scale, base);
                        const float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                        sum[(i / 2) % 2] = __fadd2_rn(sum[(i / 2) % 2], e);
                        p[i / 2] = pack2<C>(e.x, e.y);
                    }
                };
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (part == 0) weigh(0, kFirstKeys);
                    else weigh(kFirstKeys, kManyKeys);
#pragma unroll
                    for (int c = part == 0 ? 0 : kFirstKeys; c < (part == 0 ? kFirstKeys : kManyKeys); c += 32)
                        tmem_st16(s_at + c / 2, p + c / 2);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(t, part));   // the products of these keys may begin
                }
                sum[0] = __fadd2_rn(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!ok || !wait_all(o_full(t), o_ph)) break;
            o_ph ^= 1u;
            tc_fence_after();
            const int64_t at = static_cast<int64_t>(query) * g.Hq + head;
            const bool final = s.whole && g.alone;
            const int64_t part = s.whole ? at : static_cast<int64_t>(s.slot) * (128 * kManyTiles) + t * 128 + row;
            const bool write = have && ib(query >= 0 && query < g.S && head < g.Hq && s.slot < 2 * g.many_ctas);
            const float f = final ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
            const bool wide = !final || reinterpret_cast<uintptr_t>(g.out) % 32 == 0;   // (rows are multiples of 32 bytes)
            // all of the row at once, so that the next segment's products may begin
            float v[D];
            tmem_ld<D>(o_at, v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty(t));
            if (write) {
                if (final && !g.out_f32) {
                    C *to = static_cast<C *>(g.out) + at * D;
#pragma unroll
                    for (int c = 0; c < D; c += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = pack2<C>(v[c + 2 * i] * f, v[c + 2 * i + 1] * f);
                        put32(to + c, w, wide);
                    }
                } else {
                    float *to = final ? static_cast<float *>(g.out) + at * D : (s.whole ? g.whole[0] : g.many_part) + part * D;
#pragma unroll
                    for (int c = 0; c < D; c += 8) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[c + i] * f);
                        put32(to + c, w, wide);
                    }
                }
            }
            __syncwarp();
            if (write) {
                if (!final) (s.whole ? g.whole_stats[0] : g.many_stats)[part] = make_float2(m, l);
                else if (g.lse != nullptr) g.lse[at] = lse_of(m, l);
            }
        }
    }
    // ---- every role is done; MMAs complete before tensor memory is freed ----
    __syncthreads();
    if (warp == 1) {
        mbar_wait(done, 0, 50ull * 1000 * 1000);
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(M::kTmemCols));
    }
}

}  // namespace q4
