// moe_gemm.cu -- matrix product grouped by expert over int4 weights, ragged sizes.
//
//   y[r] = W_e x[rows[r]],  r in [offsets[e], offsets[e+1]),  w = (q - z) s
//
// A CTA computes 64 weight rows by 32 rows of x of one expert: weights are dequantised
// into shared memory 32 k at a time, sums are binary32.
#include <cuda_bf16.h>

#include "q4_moe.cuh"

namespace q4 {

namespace {
constexpr int TN = 64, TM = 32, TK = 32;

__device__ __forceinline__ float load_x(const MoeGemmArgs &g, int64_t row, int k) {
    const int64_t at = row * g.K + k;
    return g.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(g.x)[at]) : static_cast<const float *>(g.x)[at];
}
__device__ __forceinline__ void store_y(const MoeGemmArgs &g, int64_t at, float v) {
    if (g.bf16) static_cast<__nv_bfloat16 *>(g.y)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(g.y)[at] = v;
}
}  // namespace

__global__ void __launch_bounds__(256) moe_gemm_kernel(const MoeGemmArgs g) {
    __shared__ float ws[TK][TN + 1], xs[TK][TM + 1];
    __shared__ int tile_e, tile_r0, tile_rows;
    wait_prior_grid();
    allow_next_grid();
    if (threadIdx.x == 0) {
        int left = blockIdx.y, hi = min(max(g.offsets[0], 0), g.R);
        tile_e = -1;
        for (int e = 0; e < g.E; ++e) {
            const int lo = hi;
            hi = max(lo, min(g.offsets[e + 1], g.R));   // an offset that falls: an empty expert
            const int tiles = (hi - lo + TM - 1) / TM;
            if (left < tiles) {
                tile_e = e;
                tile_r0 = lo + left * TM;
                tile_rows = min(TM, hi - tile_r0);
                break;
            }
            left -= tiles;
        }
    }
    __syncthreads();
    if (tile_e < 0) return;
    const int n0 = blockIdx.x * TN;
    const int nb = g.K / g.group, zrow = (nb + 1) / 2;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;   // 4 weight rows, 2 rows of x per thread
    float acc[4][2] = {};
    for (int k0 = 0; k0 < g.K; k0 += TK) {
        for (int i = threadIdx.x; i < TN * TK; i += 256) {
            const int n = i / TK, k = i % TK;
            float w = 0.0f;
            if (n0 + n < g.N) {
                const int64_t row = static_cast<int64_t>(tile_e) * g.N + n0 + n;
                const int kk = k0 + k, grp = kk / g.group;
                const uint32_t byte = g.codes[row * (g.K / 2) + kk / 2];
                const int q = kk & 1 ? byte >> 4 : byte & 15;
                int z = 8;
                if (g.zeros != nullptr) {
                    const uint32_t zb = g.zeros[row * zrow + grp / 2];
                    z = grp & 1 ? zb >> 4 : zb & 15;
                }
                w = static_cast<float>(q - z) * half_bits_to_float(g.scales[row * nb + grp]);
            }
            ws[k][n] = w;
        }
        for (int i = threadIdx.x; i < TM * TK; i += 256) {
            const int m = i / TK, k = i % TK;
            float v = 0.0f;
            if (m < tile_rows) {
                const int64_t src = g.rows != nullptr ? g.rows[tile_r0 + m] : tile_r0 + m;
                if (src >= 0 && src < g.Tx) v = load_x(g, src, k0 + k);
            }
            xs[k][m] = v;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < TK; ++k) {
            const float x0 = xs[k][ty * 2], x1 = xs[k][ty * 2 + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = ws[k][tx * 4 + i];
                acc[i][0] = fmaf(w, x0, acc[i][0]);
                acc[i][1] = fmaf(w, x1, acc[i][1]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (ty * 2 + j >= tile_rows) continue;
        const int64_t r = tile_r0 + ty * 2 + j;
        const int n = n0 + tx * 4;
        if (g.swiglu) {
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                if (n + i < g.N) {
                    const float v = acc[i][j];
                    store_y(g, r * (g.N / 2) + (n + i) / 2, v / (1.0f + expf(-v)) * acc[i + 1][j]);
                }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < g.N) store_y(g, r * g.N + n + i, acc[i][j]);
        }
    }
}

int64_t moe_gemm_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int, bool) { return 0; }

int launch_moe_gemm(const MoeGemmArgs &a, cudaStream_t stream) {
    const int64_t tiles = a.R / TM + (a.E < a.R ? a.E : a.R);   // at most: full tiles, and a partial one per expert
    if (tiles > 65535) return Q4_ERR_UNSUPPORTED;
    return launch_overlappable(moe_gemm_kernel, dim3((a.N + TN - 1) / TN, static_cast<unsigned>(tiles)), dim3(256), 0,
                               stream, call_options().overlap, a);
}

}  // namespace q4
