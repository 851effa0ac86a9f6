// beam_reorder.cu -- after a beam step: page tables and unfinished pages follow the parents.
//
// Full pages are shared by the sequences whose tables name them, so a beam that continues
// another's text takes over the table's entries and copies only the rows of the page being
// written, in every plane (keys and values of each layer), into its spare page.  Nothing that
// is read is written by the same call, so sequences need no order among themselves.
//
// One CTA per sequence and run of planes copies; one more per sequence writes its table.
// Bound: the bytes of the copied rows, read and written: 16 groups of 8 beams, 64 planes of 8
// heads of 128 features, 7.5 rows on average (220 MB) 41 us, 5.4 TB/s, 0.79 of measured.
#include "q4_decode.cuh"

namespace q4 {

namespace {

constexpr int kReorderThreads = 256;

struct Moved {
    int parent;      // sequence whose pages are taken over
    int full, rest;  // full pages, tokens in the page being written
    bool copies;     // whether rows are copied
};
__device__ __forceinline__ Moved moved(const q4_beam_reorder_t &g, int i) {
    const int group = i / g.W, w = i - group * g.W;
    const int64_t most = static_cast<int64_t>(g.max_pages) * g.page;
    int64_t n = g.lens[group];
    n = n < 0 ? 0 : n > most ? most : n;
    int p = g.parents[i];
    if (p < 0 || p >= g.W) p = w;
    Moved m;
    m.parent = group * g.W + p;
    m.full = static_cast<int>(n / g.page);
    m.rest = static_cast<int>(n - static_cast<int64_t>(m.full) * g.page);
    m.copies = m.rest > 0 && p != w;
    return m;
}

}  // namespace

// V: the unit of a copy.
template <typename V>
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const q4_beam_reorder_t g, int runs,
                                                                       unsigned int *bounds) {
    wait_prior_grid();
    allow_next_grid();
    const int i = blockIdx.x;
    const Moved m = moved(g, i);
    const int64_t table = static_cast<int64_t>(i) * g.max_pages, from = static_cast<int64_t>(m.parent) * g.max_pages;
    if (blockIdx.y == runs) {
        for (int j = threadIdx.x; j < g.max_pages; j += kReorderThreads)
            g.out_tables[table + j] = j < m.full             ? g.tables[from + j]
                                      : j == m.full && m.copies ? g.spare[i]
                                                                : g.tables[table + j];
        if (threadIdx.x == 0) g.out_spare[i] = m.copies ? g.tables[table + m.full] : g.spare[i];
        return;
    }
    if (!m.copies) return;
    const int64_t src = g.tables[from + m.full], dst = g.spare[i];
    if (src < 0 || src >= g.pages || dst < 0 || dst >= g.pages) return;
    const int each = (g.planes + runs - 1) / runs, p0 = blockIdx.y * each, p1 = min(p0 + each, g.planes);
    const int per_row = static_cast<int>(g.row_bytes / sizeof(V)), per_head = per_row * m.rest;
    const int per_plane = per_head * g.heads;
    char *pool = static_cast<char *>(g.pool);
    for (int p = p0; p < p1; ++p) {
        const char *a = pool + p * g.plane_stride + src * g.page_stride;
        char *b = pool + p * g.plane_stride + dst * g.page_stride;
        constexpr int U = 4;   // units in flight a thread
        for (int e0 = threadIdx.x; e0 < per_plane; e0 += U * kReorderThreads) {
            V v[U];
            int64_t at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * kReorderThreads;
                if (e < per_plane) {
                    const int h = e / per_head, r = (e - h * per_head) / per_row, c = e - h * per_head - r * per_row;
                    at[u] = h * g.head_stride + r * g.row_stride + c * static_cast<int64_t>(sizeof(V));
                    if (q4_in_bounds(h < g.heads && r < g.page && (c + 1) * static_cast<int64_t>(sizeof(V)) <= g.row_bytes &&
                                         reinterpret_cast<uintptr_t>(a + at[u]) % sizeof(V) == 0, bounds))
                        v[u] = *reinterpret_cast<const V *>(a + at[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e0 + u * kReorderThreads < per_plane) *reinterpret_cast<V *>(b + at[u]) = v[u];
        }
    }
}

int launch_beam_reorder(const q4_beam_reorder_t &a, cudaStream_t stream) {
    const int n = a.groups * a.W;
    // a CTA per plane, up to the 65535 places of the grid's second dimension
    const int most = a.planes < 65534 ? a.planes : 65534;
    const int each = most > 0 ? (a.planes + most - 1) / most : 1, runs = (a.planes + each - 1) / each;
    const bool wide = aligned(a.pool, 16) && a.row_bytes % 16 == 0 && a.row_stride % 16 == 0 &&
                      a.head_stride % 16 == 0 && a.page_stride % 16 == 0 && a.plane_stride % 16 == 0;
    const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(runs + 1));
    const bool overlap = call_options().overlap;
    return wide ? launch_overlappable(beam_reorder_kernel<uint4>, grid, dim3(kReorderThreads), 0, stream, overlap, a,
                                      runs, bounds_counter())
                : launch_overlappable(beam_reorder_kernel<uint16_t>, grid, dim3(kReorderThreads), 0, stream, overlap, a,
                                      runs, bounds_counter());
}

}  // namespace q4
