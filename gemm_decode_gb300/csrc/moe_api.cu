// moe_api.cu -- C ABI of the mixture-of-experts calls: argument checks, workspaces, and
// the block that runs them together.  Every check runs on the host before any launch.
#include <initializer_list>

#include "q4_checks.cuh"
#include "q4_moe.cuh"

namespace q4 {

namespace {

constexpr uint32_t kMoeFlags = Q4_RUN_OVERLAPPED | Q4_RUN_WAIT_TIMEOUT;

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
bool valid_dtype(int32_t d) { return d == Q4_F32 || d == Q4_BF16; }
int64_t size_of(int32_t d) { return d == Q4_BF16 ? 2 : 4; }
bool finite_nonneg(float v) { return v >= 0.0f && v <= 3.0e38f; }   // NaN fails too

bool is_sigmoid(int32_t score) { return (score & ~Q4_ROUTE_SCORE_BIAS) == Q4_ROUTE_SIGMOID; }
bool is_score_bias(int32_t score) { return (score & Q4_ROUTE_SCORE_BIAS) != 0; }

// Outputs against inputs and against one another.
bool outputs_clash(const Span *out, int nout, const Span *in, int nin) {
    for (int i = 0; i < nout; ++i) {
        if (overlaps_any(out[i], in, nin)) return true;
        if (overlaps_any(out[i], out, i)) return true;
    }
    return false;
}

int route_shape(int64_t T, int64_t E, int64_t k, int32_t score) {
    if (T < 0 || E < 1 || k < 1 || k > E) return Q4_ERR_INVALID_ARG;
    const int32_t kind = score & ~Q4_ROUTE_SCORE_BIAS;
    if (kind != Q4_ROUTE_SOFTMAX && kind != Q4_ROUTE_SIGMOID) return Q4_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > kMaxTopK || T * k > 0x7fffffffLL) return Q4_ERR_UNSUPPORTED;
    return Q4_OK;
}

int gemm_shape(int64_t R, int64_t Tx, int64_t E, int64_t N, int64_t K, int32_t group, int32_t dtype,
               int32_t epilogue) {
    const int st = check_shape(R, N, K, group);
    if (st != Q4_OK) return st;
    if (Tx < 0 || E < 1 || !valid_dtype(dtype)) return Q4_ERR_INVALID_ARG;
    if (epilogue != Q4_EPILOGUE_NONE && epilogue != Q4_EPILOGUE_SWIGLU) return Q4_ERR_INVALID_ARG;
    if (epilogue == Q4_EPILOGUE_SWIGLU && N % 2 != 0) return Q4_ERR_INVALID_ARG;
    if (E > kMaxExperts || R > 0x7fffffffLL || Tx >= 0x7fffffffLL || E * N > 0x7fffffffLL || K > kMaxMoeK)
        return Q4_ERR_UNSUPPORTED;
    // the kernels count items in 32 bits; no y that fits a device has as many
    if (!moe_gemm_countable(R, static_cast<int>(E), N, group, dtype == Q4_BF16)) return Q4_ERR_UNSUPPORTED;
    return Q4_OK;
}

// Places of the block's intermediates in its workspace.  h and y, between the products and
// the norm, are of the call's type, as when the four calls are made one after another: in
// bfloat16 half the bytes, for two more roundings (2.0e-3 off the exact value in the 2-norm,
// where rounding that value alone is 1.7e-3).
struct BlockLayout {
    int64_t offsets, rows, pos, h, y, scratch, scratch_bytes, total;
};
BlockLayout block_layout(int64_t T, int64_t E, int64_t k, int64_t H, int64_t inner, int32_t dtype) {
    const int64_t R = T * k, b = size_of(dtype);
    BlockLayout l;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t p = at;
        at += align256(bytes);
        return p;
    };
    l.offsets = take(4 * (E + 1));
    l.rows = take(4 * R);
    l.pos = take(4 * R);
    l.h = take(b * R * inner);
    l.y = take(b * R * H);
    // one scratch area serves the three calls in turn
    const bool bf16 = dtype == Q4_BF16;
    l.scratch_bytes = route_workspace_bytes(static_cast<int>(T), static_cast<int>(E), static_cast<int>(k));
    for (int64_t n : {moe_gemm_workspace_bytes(R, T, 2 * inner, H, static_cast<int>(E), bf16),
                      moe_gemm_workspace_bytes(R, R, H, inner, static_cast<int>(E), bf16)})
        if (n > l.scratch_bytes) l.scratch_bytes = n;
    l.scratch = take(l.scratch_bytes);
    l.total = at;
    return l;
}

// Overlapped launches for the calls inside a block that follow its first kernel.
class OverlapInside {
public:
    OverlapInside() : scope_(options()) {}

private:
    static CallOptions options() {
        CallOptions o = call_options();
        o.overlap = true;
        return o;
    }
    CallScope scope_;
};

}  // namespace

}  // namespace q4

using namespace q4;

extern "C" {

int64_t q4moe_route_workspace(int32_t T, int32_t E, int32_t top_k) {
    if (route_shape(T, E, top_k, Q4_ROUTE_SOFTMAX) != Q4_OK) return -1;
    return align256(route_workspace_bytes(T, E, top_k)) + 256;
}

int q4moe_route_run(const float *logits, const float *bias_or_null, const uint8_t *token_mask_or_null, int32_t T,
                    int32_t E, int32_t top_k, int32_t score, int32_t renormalize, float scale, int32_t *ids,
                    float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                    int64_t workspace_bytes, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    int st = options_from(opts, kMoeFlags, co);
    if (st != Q4_OK) return st;
    if ((st = route_shape(T, E, top_k, score)) != Q4_OK) return st;
    if (T == 0) return Q4_OK;
    if (logits == nullptr || ids == nullptr || weights == nullptr || offsets == nullptr || rows == nullptr ||
        pos == nullptr || workspace == nullptr)
        return Q4_ERR_INVALID_ARG;
    const int64_t R = static_cast<int64_t>(T) * top_k;
    if (workspace_bytes < q4moe_route_workspace(T, E, top_k)) return Q4_ERR_INVALID_ARG;
    if (!aligned(logits, 4) || !aligned(bias_or_null, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4) || !aligned(workspace, 256))
        return Q4_ERR_MISALIGNED;
    {
        const Span in[3] = {span(logits, 4ll * T * E), span(bias_or_null, 4ll * E), span(token_mask_or_null, T)};
        const Span out[6] = {span(ids, 4 * R),         span(weights, 4 * R), span(offsets, 4 * (E + 1ll)),
                             span(rows, 4 * R),        span(pos, 4 * R),     span(workspace, workspace_bytes)};
        if (outputs_clash(out, 6, in, 3)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    RouteArgs a = {logits, bias_or_null, token_mask_or_null, T, E, top_k, is_sigmoid(score), renormalize != 0,
                   is_score_bias(score), scale, ids, weights, offsets, rows, pos, static_cast<int *>(workspace),
                   bounds_counter()};
    return launch_route(a, static_cast<cudaStream_t>(stream));
}

int64_t q4moe_gemm_workspace(int64_t R, int64_t Tx, int64_t N, int64_t K, int32_t E, int32_t dtype) {
    if (gemm_shape(R, Tx, E, N, K, 32, dtype, Q4_EPILOGUE_NONE) != Q4_OK) return -1;
    return align256(moe_gemm_workspace_bytes(R, Tx, N, K, E, dtype == Q4_BF16)) + 256;
}

int q4moe_gemm_run(const void *codes, const void *scales_f16, const void *zeros_u4_or_null, const void *x,
                   const int32_t *rows_or_null, const int32_t *offsets, void *y, int32_t E, int64_t R, int64_t Tx,
                   int64_t N, int64_t K, int32_t group, int32_t dtype, int32_t epilogue, void *workspace,
                   int64_t workspace_bytes, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    int st = options_from(opts, kMoeFlags, co);
    if (st != Q4_OK) return st;
    if ((st = gemm_shape(R, Tx, E, N, K, group, dtype, epilogue)) != Q4_OK) return st;
    if (rows_or_null == nullptr && Tx < R) return Q4_ERR_INVALID_ARG;
    if (R == 0 || N == 0) return Q4_OK;
    if ((st = check_q4_args(codes, scales_f16, N, K, group)) != Q4_OK) return st;
    if ((x == nullptr && Tx > 0) || offsets == nullptr || y == nullptr || workspace == nullptr)
        return Q4_ERR_INVALID_ARG;
    if (workspace_bytes < q4moe_gemm_workspace(R, Tx, N, K, E, dtype)) return Q4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(rows_or_null, 4) || !aligned(offsets, 4) ||
        !aligned(y, static_cast<uintptr_t>(size_of(dtype))) || !aligned(workspace, 256))
        return Q4_ERR_MISALIGNED;
    {
        Span in[6];
        weight_spans(codes, scales_f16, zeros_u4_or_null, static_cast<int64_t>(E) * N, K, group, in);
        in[3] = span(x, size_of(dtype) * Tx * K);
        in[4] = span(rows_or_null, 4 * R);
        in[5] = span(offsets, 4 * (E + 1ll));
        const int64_t cols = epilogue == Q4_EPILOGUE_SWIGLU ? N / 2 : N;
        const Span out[2] = {span(y, size_of(dtype) * R * cols), span(workspace, workspace_bytes)};
        if (outputs_clash(out, 2, in, 6)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    MoeGemmArgs a = {static_cast<const uint8_t *>(codes), static_cast<const uint16_t *>(scales_f16),
                     static_cast<const uint8_t *>(zeros_u4_or_null), x, rows_or_null, offsets, y, E,
                     static_cast<int>(R), static_cast<int>(Tx), static_cast<int>(N), static_cast<int>(K), group,
                     dtype == Q4_BF16, epilogue == Q4_EPILOGUE_SWIGLU, workspace};
    return launch_moe_gemm(a, static_cast<cudaStream_t>(stream));
}

int q4_block_norm_run(const q4_block_norm_t *args, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    const int st = options_from(opts, kMoeFlags, co);
    if (st != Q4_OK) return st;
    if (args == nullptr) return Q4_ERR_INVALID_ARG;
    const q4_block_norm_t &g = *args;
    if (g.T < 0 || g.H < 1 || g.top_k < 0 || g.R < 0 || !valid_dtype(g.dtype) || !finite_nonneg(g.eps))
        return Q4_ERR_INVALID_ARG;
    if (g.H > kMaxNormH || g.top_k > kMaxTopK) return Q4_ERR_UNSUPPORTED;
    if (g.gate != nullptr && g.gate_stride != 0 && g.gate_stride != g.H) return Q4_ERR_INVALID_ARG;
    if (g.top_k == 0 && g.R != g.T) return Q4_ERR_INVALID_ARG;
    if (g.T == 0) return Q4_OK;
    if ((g.y == nullptr && g.R > 0) || g.x == nullptr || g.out == nullptr) return Q4_ERR_INVALID_ARG;
    if (g.top_k > 0 && (g.pos == nullptr || g.weights == nullptr)) return Q4_ERR_INVALID_ARG;
    if ((g.pre_gamma == nullptr) != (g.out_norm == nullptr)) return Q4_ERR_INVALID_ARG;
    const int64_t b = size_of(g.dtype), n = static_cast<int64_t>(g.T) * g.H;
    if (!aligned(g.y, 16) || !aligned(g.x, 16) || !aligned(g.out, 16) || !aligned(g.out_norm, 16) ||
        !aligned(g.gate, static_cast<uintptr_t>(b)) || !aligned(g.post_gamma, 4) || !aligned(g.pre_gamma, 4) ||
        !aligned(g.pos, 4) || !aligned(g.weights, 4))
        return Q4_ERR_MISALIGNED;
    {
        const int64_t c = 4ll * g.T * g.top_k;
        const Span in[7] = {span(g.y, b * g.R * g.H),  span(g.x, b * n), span(g.pos, c),
                            span(g.weights, c),        span(g.post_gamma, 4ll * g.H),
                            span(g.pre_gamma, 4ll * g.H), span(g.gate, b * (g.gate_stride != 0 ? n : g.H))};
        const Span out[2] = {span(g.out, b * n), span(g.out_norm, b * n)};
        if (outputs_clash(out, 2, in, 7)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    return launch_block_norm(g, static_cast<cudaStream_t>(stream));
}

int64_t q4moe_block_workspace(int32_t T, int32_t E, int32_t top_k, int32_t H, int32_t inner, int32_t dtype) {
    if (route_shape(T, E, top_k, Q4_ROUTE_SOFTMAX) != Q4_OK || inner < 1 || H < 1) return -1;
    const int64_t R = static_cast<int64_t>(T) * top_k;
    if (gemm_shape(R, T, E, 2ll * inner, H, 32, dtype, Q4_EPILOGUE_SWIGLU) != Q4_OK ||
        gemm_shape(R, R, E, H, inner, 32, dtype, Q4_EPILOGUE_NONE) != Q4_OK)
        return -1;
    return block_layout(T, E, top_k, H, inner, dtype).total + 256;
}

int q4moe_block_run(const q4moe_block_t *args, const q4_run_options_t *opts, void *stream) {
    CallOptions co;
    int st = options_from(opts, kMoeFlags, co);
    if (st != Q4_OK) return st;
    if (args == nullptr) return Q4_ERR_INVALID_ARG;
    const q4moe_block_t &g = *args;
    if ((st = route_shape(g.T, g.E, g.top_k, g.score)) != Q4_OK) return st;
    if (g.H < 1 || g.inner < 1 || !valid_dtype(g.dtype) || !finite_nonneg(g.eps)) return Q4_ERR_INVALID_ARG;
    const int64_t R = static_cast<int64_t>(g.T) * g.top_k;
    if ((st = gemm_shape(R, g.T, g.E, 2ll * g.inner, g.H, g.group, g.dtype, Q4_EPILOGUE_SWIGLU)) != Q4_OK) return st;
    if ((st = gemm_shape(R, R, g.E, g.H, g.inner, g.group, g.dtype, Q4_EPILOGUE_NONE)) != Q4_OK) return st;
    if (g.H > kMaxNormH) return Q4_ERR_UNSUPPORTED;
    if (g.gate != nullptr && g.gate_stride != 0 && g.gate_stride != g.H) return Q4_ERR_INVALID_ARG;
    if ((g.pre_gamma == nullptr) != (g.out_norm == nullptr)) return Q4_ERR_INVALID_ARG;
    if (g.T == 0) return Q4_OK;
    if (g.up_codes == nullptr || g.up_scales_f16 == nullptr || g.down_codes == nullptr ||
        g.down_scales_f16 == nullptr || g.logits == nullptr || g.a == nullptr || g.x == nullptr || g.ids == nullptr ||
        g.route_weights == nullptr || g.out == nullptr || g.workspace == nullptr)
        return Q4_ERR_INVALID_ARG;
    const BlockLayout l = block_layout(g.T, g.E, g.top_k, g.H, g.inner, g.dtype);
    if (g.workspace_bytes < l.total + 256) return Q4_ERR_INVALID_ARG;
    const int64_t b = size_of(g.dtype), n = b * g.T * g.H;
    if (!aligned(g.up_codes, 16) || !aligned(g.down_codes, 16) || !aligned(g.up_scales_f16, 2) ||
        !aligned(g.down_scales_f16, 2) || !aligned(g.a, 16) || !aligned(g.x, 16) || !aligned(g.out, 16) ||
        !aligned(g.out_norm, 16) || !aligned(g.workspace, 256) || !aligned(g.logits, 4) || !aligned(g.bias_or_null, 4) ||
        !aligned(g.ids, 4) || !aligned(g.route_weights, 4) || !aligned(g.post_gamma, 4) || !aligned(g.pre_gamma, 4) ||
        !aligned(g.gate, static_cast<uintptr_t>(b)))
        return Q4_ERR_MISALIGNED;
    {
        Span in[14];
        weight_spans(g.up_codes, g.up_scales_f16, g.up_zeros_u4_or_null, 2ll * g.E * g.inner, g.H, g.group, in);
        weight_spans(g.down_codes, g.down_scales_f16, g.down_zeros_u4_or_null, static_cast<int64_t>(g.E) * g.H,
                     g.inner, g.group, in + 3);
        in[6] = span(g.logits, 4ll * g.T * g.E);
        in[7] = span(g.bias_or_null, 4ll * g.E);
        in[8] = span(g.token_mask_or_null, g.T);
        in[9] = span(g.a, n);
        in[10] = span(g.x, n);
        in[11] = span(g.post_gamma, 4ll * g.H);
        in[12] = span(g.pre_gamma, 4ll * g.H);
        in[13] = span(g.gate, g.gate_stride != 0 ? n : b * g.H);
        const Span out[5] = {span(g.ids, 4 * R), span(g.route_weights, 4 * R), span(g.out, n), span(g.out_norm, n),
                             span(g.workspace, g.workspace_bytes)};
        if (outputs_clash(out, 5, in, 14)) return Q4_ERR_INVALID_ARG;
    }
    CallScope scope(co);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    unsigned char *w = static_cast<unsigned char *>(g.workspace);
    int *offsets = reinterpret_cast<int *>(w + l.offsets), *rows = reinterpret_cast<int *>(w + l.rows),
        *pos = reinterpret_cast<int *>(w + l.pos);
    const RouteArgs r = {g.logits, g.bias_or_null, g.token_mask_or_null, g.T, g.E, g.top_k,
                         is_sigmoid(g.score), g.renormalize != 0, is_score_bias(g.score), g.route_scale, g.ids,
                         g.route_weights, offsets, rows, pos, reinterpret_cast<int *>(w + l.scratch), bounds_counter()};
    if ((st = launch_route(r, cs)) != Q4_OK) return st;
    OverlapInside inside;
    const int bf16 = g.dtype == Q4_BF16;
    const MoeGemmArgs up = {static_cast<const uint8_t *>(g.up_codes), static_cast<const uint16_t *>(g.up_scales_f16),
                            static_cast<const uint8_t *>(g.up_zeros_u4_or_null), g.a, rows, offsets, w + l.h, g.E,
                            static_cast<int>(R), g.T, 2 * g.inner, g.H, g.group, bf16, 1, w + l.scratch};
    if ((st = launch_moe_gemm(up, cs)) != Q4_OK) return st;
    const MoeGemmArgs down = {static_cast<const uint8_t *>(g.down_codes),
                              static_cast<const uint16_t *>(g.down_scales_f16),
                              static_cast<const uint8_t *>(g.down_zeros_u4_or_null), w + l.h, nullptr, offsets,
                              w + l.y, g.E, static_cast<int>(R), static_cast<int>(R), g.H, g.inner, g.group, bf16, 0,
                              w + l.scratch};
    if ((st = launch_moe_gemm(down, cs)) != Q4_OK) return st;
    q4_block_norm_t nm = {};
    nm.T = g.T;
    nm.H = g.H;
    nm.top_k = g.top_k;
    nm.dtype = g.dtype;
    nm.R = R;
    nm.y = w + l.y;
    nm.pos = pos;
    nm.weights = g.route_weights;
    nm.x = g.x;
    nm.post_gamma = g.post_gamma;
    nm.gate = g.gate;
    nm.gate_stride = g.gate_stride;
    nm.pre_gamma = g.pre_gamma;
    nm.out = g.out;
    nm.out_norm = g.out_norm;
    nm.residual_scale = g.residual_scale;
    nm.eps = g.eps;
    return launch_block_norm(nm, cs);
}

}  // extern "C"
