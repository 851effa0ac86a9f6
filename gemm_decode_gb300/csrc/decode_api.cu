// decode_api.cu -- C ABI of the calls for several continuations of one prompt: argument
// checks and workspaces.  Every check runs on the host before any launch.
#include <cmath>

#include "q4_checks.cuh"
#include "q4_decode.cuh"

namespace q4 {

namespace {

constexpr uint32_t kDecodeFlags = Q4_RUN_OVERLAPPED | Q4_RUN_WAIT_TIMEOUT;

bool finite(float v) { return v >= -3.0e38f && v <= 3.0e38f; }   // NaN fails too
int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

bool outputs_clash(const Span *out, int nout, const Span *in, int nin) {
    for (int i = 0; i < nout; ++i) {
        if (overlaps_any(out[i], in, nin)) return true;
        if (overlaps_any(out[i], out, i)) return true;
    }
    return false;
}

// Sizes and strides whose products stay far from 2^63.
bool small(int64_t v) { return v >= 0 && v < (1ll << 44); }
// Rows whose last one lies as near.
bool small_rows(int64_t n, int64_t stride) { return n <= 1 || stride < (1ll << 44) / (n - 1); }

// The pools of a cache: sizes that make sense, and the elements from the first to the last.
int cache_shape(const q4_kv_cache_t &c) {
    if ((c.dtype != Q4_BF16 && c.dtype != Q4_F16) || c.heads < 1 || c.D < 1 || c.page < 1 || c.pages < 0)
        return Q4_ERR_INVALID_ARG;
    if (!small(c.page_stride) || !small(c.head_stride) || !small(c.row_stride)) return Q4_ERR_INVALID_ARG;
    // no two elements at the same place: the strides, in some order, each pass over what lies within
    const int64_t stride[3] = {c.page_stride, c.head_stride, c.row_stride}, count[3] = {c.pages, c.heads, c.page};
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[order[j]] < stride[order[i]]) {
                const int t = order[i];
                order[i] = order[j], order[j] = t;
            }
    int64_t within = c.D;
    for (int i : order) {
        if (count[i] <= 1) continue;
        if (stride[i] < within) return Q4_ERR_INVALID_ARG;
        if (stride[i] > (1ll << 44) / count[i]) return Q4_ERR_UNSUPPORTED;
        within += stride[i] * (count[i] - 1);
        if (!small(within)) return Q4_ERR_UNSUPPORTED;
    }
    return Q4_OK;
}
int64_t cache_bytes(const q4_kv_cache_t &c) {
    if (c.pages == 0) return 0;
    return 2 * ((c.pages - 1) * c.page_stride + (c.heads - 1) * c.head_stride + (c.page - 1) * c.row_stride + c.D);
}
// bytes of n rows `stride` elements apart
int64_t rows_bytes(int64_t n, int64_t stride, int64_t row, int64_t esize) {
    return n > 0 ? esize * ((n - 1) * stride + row) : 0;
}

int attn_shape(int64_t S, int64_t groups, int64_t Hq, int64_t Hkv, int64_t D) {
    if (S < 0 || groups < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return Q4_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || Hq / Hkv > kMaxShare || S > kMaxQueries || S * Hq > 0x7fffffffLL || groups > (S > 1 ? S : 1))
        return Q4_ERR_UNSUPPORTED;
    return Q4_OK;
}

int beam_shape(int64_t groups, int64_t W, int64_t K, int64_t V) {
    if (groups < 0 || W < 1 || K < 1 || V < 1) return Q4_ERR_INVALID_ARG;
    if (W > kMaxBeams || K > kMaxBeams || V >= 0x7fffffffLL || groups * W > 0x7fffffffLL) return Q4_ERR_UNSUPPORTED;
    return Q4_OK;
}

}  // namespace

}  // namespace q4

using namespace q4;

extern "C" {

int q4_rope_append_run(const q4_rope_append_t *args, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    int st = options_from(opts, kDecodeFlags, co);
    if (st != Q4_OK) return st;
    if (args == nullptr) return Q4_ERR_INVALID_ARG;
    const q4_rope_append_t &g = *args;
    const q4_kv_cache_t &c = g.cache;
    const bool keys = g.k != nullptr;
    if (g.T < 0 || g.Hq < 1 || c.D < 1 || g.rot < 0 || g.rot % 2 != 0 || g.rot > c.D ||
        (g.dtype != Q4_F32 && g.dtype != Q4_BF16) || (g.layout != Q4_ROPE_HALF && g.layout != Q4_ROPE_INTERLEAVED) ||
        !finite(g.scale) || !(g.eps >= 0.0f) || !finite(g.eps) || (c.dtype != Q4_BF16 && c.dtype != Q4_F16))
        return Q4_ERR_INVALID_ARG;
    if (keys != (g.v != nullptr)) return Q4_ERR_INVALID_ARG;
    if (keys && (st = cache_shape(c)) != Q4_OK) return st;
    const int64_t qrow = static_cast<int64_t>(g.Hq) * c.D, krow = keys ? static_cast<int64_t>(c.heads) * c.D : 0;
    if (!small(g.q_stride) || g.q_stride < (g.T > 1 ? qrow : 0)) return Q4_ERR_INVALID_ARG;
    if (keys && (!small(g.k_stride) || !small(g.v_stride) || (g.T > 1 && (g.k_stride < krow || g.v_stride < krow))))
        return Q4_ERR_INVALID_ARG;
    if (c.D > kMaxHeadD || qrow + 2 * krow > 0x7fffffLL || !small_rows(g.T, g.q_stride) ||
        (keys && (!small_rows(g.T, g.k_stride) || !small_rows(g.T, g.v_stride))))
        return Q4_ERR_UNSUPPORTED;
    if (g.T == 0) return Q4_OK;
    if (g.q == nullptr || g.q_out == nullptr || (g.rot > 0 && (g.positions == nullptr || g.inv_freq == nullptr)) ||
        (keys && c.pages > 0 && (c.k == nullptr || c.v == nullptr)))
        return Q4_ERR_INVALID_ARG;
    const uintptr_t b = g.dtype == Q4_F32 ? 4 : 2;
    if (!aligned(g.q, b) || !aligned(g.k, b) || !aligned(g.v, b) || !aligned(g.q_out, 2) || !aligned(c.k, 2) ||
        !aligned(c.v, 2) || !aligned(g.q_gamma, 4) || !aligned(g.k_gamma, 4) || !aligned(g.positions, 4) ||
        !aligned(g.inv_freq, 4) || !aligned(g.slots, 4))
        return Q4_ERR_MISALIGNED;
    {
        const int64_t e = static_cast<int64_t>(b);
        const Span in[8] = {span(g.q, rows_bytes(g.T, g.q_stride, qrow, e)),
                            span(g.k, rows_bytes(g.T, g.k_stride, krow, e)),
                            span(g.v, rows_bytes(g.T, g.v_stride, krow, e)),
                            span(g.q_gamma, 4ll * c.D), span(g.k_gamma, 4ll * c.D), span(g.positions, 4ll * g.T),
                            span(g.inv_freq, 2ll * g.rot), span(g.slots, 4ll * g.T)};
        // the pools may lie between one another (pages of keys, then of values), but not be the same
        const Span out[2] = {span(g.q_out, 2 * g.T * qrow), span(keys ? c.k : nullptr, keys ? cache_bytes(c) : 0)};
        const Span values = span(keys ? c.v : nullptr, keys ? cache_bytes(c) : 0);
        if (outputs_clash(out, 2, in, 8) || overlaps_any(values, in, 8) || overlap(values, out[0]) ||
            (keys && c.k == c.v && c.pages > 0))
            return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    return launch_rope_append(g, static_cast<cudaStream_t>(stream));
}

int q4_rope_frequencies(float *inv_freq, int32_t rot, double base, int32_t kind, double factor, double trained,
                        double low, double high) {
    if (inv_freq == nullptr || rot < 0 || rot % 2 != 0 || !(base > 0.0) || !std::isfinite(base) ||
        (kind != Q4_ROPE_PLAIN && kind != Q4_ROPE_LINEAR && kind != Q4_ROPE_BANDS))
        return Q4_ERR_INVALID_ARG;
    if (kind != Q4_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return Q4_ERR_INVALID_ARG;
    if (kind == Q4_ROPE_BANDS && (!(trained > 0.0) || !std::isfinite(trained) || !(low < high) ||
                                  !std::isfinite(low) || !std::isfinite(high)))
        return Q4_ERR_INVALID_ARG;
    const double two_pi = 2.0 * std::acos(-1.0);
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (kind == Q4_ROPE_LINEAR) f /= factor;
        if (kind == Q4_ROPE_BANDS) {
            double keep = (trained * f / two_pi - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * (f / factor);
        }
        inv_freq[i] = static_cast<float>(f);
    }
    return Q4_OK;
}

int64_t q4_prefix_attn_workspace(int32_t S, int32_t groups, int32_t Hq, int32_t Hkv, int32_t D) {
    if (attn_shape(S, groups, Hq, Hkv, D) != Q4_OK) return -1;
    return align256(prefix_attn_workspace_bytes(S, groups, Hq, Hkv, D)) + 256;
}

int q4_prefix_attn_run(const q4_prefix_attn_t *args, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    int st = options_from(opts, kDecodeFlags, co);
    if (st != Q4_OK) return st;
    if (args == nullptr) return Q4_ERR_INVALID_ARG;
    const q4_prefix_attn_t &g = *args;
    const q4_kv_cache_t &c = g.cache;
    if ((st = cache_shape(c)) != Q4_OK) return st;
    if ((st = attn_shape(g.S, g.groups, g.Hq, c.heads, c.D)) != Q4_OK) return st;
    if ((g.out_dtype != c.dtype && g.out_dtype != Q4_F32) || !(std::fabs(g.scale) <= 1e38f) || g.max_shared_pages < 0 ||
        g.max_own_pages < 0)
        return Q4_ERR_INVALID_ARG;
    const bool own = g.own_pages != nullptr || g.own_lens != nullptr;
    if (g.groups == 0 && !own) return Q4_ERR_INVALID_ARG;
    const int64_t qrow = static_cast<int64_t>(g.Hq) * c.D;
    if (!small(g.q_stride) || (g.S > 1 && g.q_stride < qrow)) return Q4_ERR_INVALID_ARG;
    if (c.page < 16 || (c.page & (c.page - 1)) != 0 || c.pages > 0x7fffffffLL || !small_rows(g.S, g.q_stride) ||
        static_cast<int64_t>(g.max_shared_pages) * c.page > 0x7fffffffLL ||
        static_cast<int64_t>(g.max_own_pages) * c.page > 0x7fffffffLL)
        return Q4_ERR_UNSUPPORTED;
    if (g.S == 0) return Q4_OK;
    if (g.q == nullptr || g.out == nullptr || g.workspace == nullptr || c.k == nullptr || c.v == nullptr || c.pages < 1)
        return Q4_ERR_INVALID_ARG;
    if (g.groups > 0 && (g.shared_lens == nullptr || (g.shared_pages == nullptr && g.max_shared_pages > 0) ||
                         (g.group_offsets == nullptr && g.groups != 1)))
        return Q4_ERR_INVALID_ARG;
    if (own && (g.own_lens == nullptr || (g.own_pages == nullptr && g.max_own_pages > 0))) return Q4_ERR_INVALID_ARG;
    if (g.workspace_bytes < q4_prefix_attn_workspace(g.S, g.groups, g.Hq, c.heads, c.D)) return Q4_ERR_INVALID_ARG;
    if (!aligned(g.q, 16) || !aligned(g.out, 16) || !aligned(c.k, 16) || !aligned(c.v, 16) ||
        g.q_stride % 8 != 0 || c.page_stride % 8 != 0 || c.head_stride % 8 != 0 || c.row_stride % 8 != 0 ||
        !aligned(g.group_offsets, 4) || !aligned(g.shared_pages, 4) || !aligned(g.shared_lens, 4) ||
        !aligned(g.limits, 4) || !aligned(g.own_pages, 4) || !aligned(g.own_lens, 4) || !aligned(g.lse, 4) ||
        !aligned(g.workspace, 256))
        return Q4_ERR_MISALIGNED;
    {
        const Span in[9] = {span(g.q, rows_bytes(g.S, g.q_stride, qrow, 2)),
                            span(c.k, cache_bytes(c)),
                            span(c.v, cache_bytes(c)),
                            span(g.group_offsets, g.groups > 0 ? 4ll * (g.groups + 1) : 0),
                            span(g.shared_pages, 4ll * g.groups * g.max_shared_pages),
                            span(g.shared_lens, 4ll * g.groups),
                            span(g.limits, 4ll * g.S),
                            span(g.own_pages, 4ll * g.S * g.max_own_pages),
                            span(g.own_lens, 4ll * g.S)};
        const Span out[3] = {span(g.out, (g.out_dtype == Q4_F32 ? 4 : 2) * g.S * qrow),
                             span(g.lse, 4ll * g.S * g.Hq), span(g.workspace, g.workspace_bytes)};
        if (outputs_clash(out, 3, in, 9)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    return launch_prefix_attn(g, static_cast<cudaStream_t>(stream));
}

int64_t q4_beam_step_workspace(int32_t groups, int32_t W, int32_t K, int64_t V) {
    if (beam_shape(groups, W, K, V) != Q4_OK) return -1;
    return align256(beam_workspace_bytes(groups, W, K, V)) + 256;
}

int q4_beam_step_run(const float *logits, int64_t row_stride, const float *scores, const uint8_t *finished_or_null,
                     int32_t groups, int32_t W, int32_t K, int64_t V, int32_t eos, int32_t *tokens, int32_t *parents,
                     float *out_scores, uint8_t *out_finished_or_null, void *workspace, int64_t workspace_bytes,
                     const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    int st = options_from(opts, kDecodeFlags, co);
    if (st != Q4_OK) return st;
    if ((st = beam_shape(groups, W, K, V)) != Q4_OK) return st;
    const int64_t rows = static_cast<int64_t>(groups) * W, out_n = static_cast<int64_t>(groups) * K;
    if (!small(row_stride) || (rows > 1 && row_stride < V) || eos < -1 || eos >= V ||
        (finished_or_null != nullptr && eos < 0))
        return Q4_ERR_INVALID_ARG;
    if (!small_rows(rows, row_stride)) return Q4_ERR_UNSUPPORTED;
    if (groups == 0) return Q4_OK;
    if (logits == nullptr || scores == nullptr || tokens == nullptr || parents == nullptr || out_scores == nullptr ||
        workspace == nullptr || workspace_bytes < q4_beam_step_workspace(groups, W, K, V))
        return Q4_ERR_INVALID_ARG;
    if (!aligned(logits, 4) || !aligned(scores, 4) || !aligned(tokens, 4) || !aligned(parents, 4) ||
        !aligned(out_scores, 4) || !aligned(workspace, 256))
        return Q4_ERR_MISALIGNED;
    {
        const Span in[3] = {span(logits, rows_bytes(rows, row_stride, V, 4)), span(scores, 4 * rows),
                            span(finished_or_null, rows)};
        const Span out[5] = {span(tokens, 4 * out_n), span(parents, 4 * out_n), span(out_scores, 4 * out_n),
                             span(out_finished_or_null, out_n), span(workspace, workspace_bytes)};
        if (outputs_clash(out, 5, in, 3)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    const BeamArgs a = {logits, row_stride, scores, finished_or_null, groups, W, K, V, eos, tokens, parents, out_scores,
                        out_finished_or_null, workspace, bounds_counter()};
    return launch_beam_step(a, static_cast<cudaStream_t>(stream));
}

int q4_beam_reorder_run(const q4_beam_reorder_t *args, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    const int st = options_from(opts, kDecodeFlags, co);
    if (st != Q4_OK) return st;
    if (args == nullptr) return Q4_ERR_INVALID_ARG;
    const q4_beam_reorder_t &g = *args;
    if (g.groups < 0 || g.W < 1 || g.max_pages < 0 || g.planes < 0 || g.heads < 1 || g.page < 1 || g.pages < 0 ||
        g.row_bytes < 2 || g.row_bytes % 2 != 0 || !small(g.row_bytes) || !small(g.plane_stride) ||
        !small(g.page_stride) || !small(g.head_stride) || !small(g.row_stride))
        return Q4_ERR_INVALID_ARG;
    const int64_t n = static_cast<int64_t>(g.groups) * g.W;
    if (g.W > kMaxReorderW || n > 0x7fffffffLL || g.pages > 0x7fffffffLL || !small_rows(n + 1, g.max_pages) ||
        static_cast<int64_t>(g.heads) * g.page > 0x7fffffffLL / g.row_bytes)
        return Q4_ERR_UNSUPPORTED;
    int64_t bytes = 0;
    if (g.planes > 0 && g.pages > 0) {
        const int64_t stride[4] = {g.plane_stride, g.page_stride, g.head_stride, g.row_stride};
        const int64_t count[4] = {g.planes, g.pages, g.heads, g.page};
        int order[4] = {0, 1, 2, 3};
        for (int i = 0; i < 4; ++i)
            for (int j = i + 1; j < 4; ++j)
                if (stride[order[j]] < stride[order[i]]) {
                    const int t = order[i];
                    order[i] = order[j], order[j] = t;
                }
        bytes = g.row_bytes;
        for (int i : order) {
            if (count[i] <= 1) continue;
            if (stride[i] < bytes) return Q4_ERR_INVALID_ARG;
            if (stride[i] > (1ll << 44) / count[i]) return Q4_ERR_UNSUPPORTED;
            bytes += stride[i] * (count[i] - 1);
        }
    }
    if (n == 0) return Q4_OK;
    if (g.lens == nullptr || g.parents == nullptr || g.spare == nullptr || g.out_spare == nullptr ||
        (g.max_pages > 0 && (g.tables == nullptr || g.out_tables == nullptr)) || (bytes > 0 && g.pool == nullptr))
        return Q4_ERR_INVALID_ARG;
    if (!aligned(g.tables, 4) || !aligned(g.lens, 4) || !aligned(g.parents, 4) || !aligned(g.spare, 4) ||
        !aligned(g.out_tables, 4) || !aligned(g.out_spare, 4) || !aligned(g.pool, 2) || g.plane_stride % 2 != 0 ||
        g.page_stride % 2 != 0 || g.head_stride % 2 != 0 || g.row_stride % 2 != 0)
        return Q4_ERR_MISALIGNED;
    {
        const Span in[4] = {span(g.tables, 4 * n * g.max_pages), span(g.lens, 4ll * g.groups), span(g.parents, 4 * n),
                            span(g.spare, 4 * n)};
        const Span out[3] = {span(g.out_tables, 4 * n * g.max_pages), span(g.out_spare, 4 * n), span(g.pool, bytes)};
        if (outputs_clash(out, 3, in, 4)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    return launch_beam_reorder(g, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
