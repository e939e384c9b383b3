// Norm of each head's queries and keys with the position rotation in the same
// pass, forward and backward, and the table of the rotation's angles.
//
//   r = 1 / sqrt(mean(x^2) + eps), n = x r w            (or n = x: no norm)
//   y: the first `rotary` elements of n in pairs (a, b), turned by the angle of the
//      token's position: a cos - b sin, a sin + b cos; the others unchanged
//   dn = dy turned back, dw = sum dn x r, g = dn w, dx = r (g - x r mean(g x r))
//
// HBM-bound: a row is read once, held in registers as fp32 and written once.  One
// warp per row; the row goes through shared memory once so that any pairing can
// be formed.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "checks.h"

namespace dmuon {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxDim = 256;
constexpr int kWarps = 8;
constexpr int kPer = kMaxDim / 32;  // elements of a lane
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int kMaxHeads = 1024;
constexpr int kMaxPartials = 608;   // blocks of the backward pass: rows of partial sums

struct Rows {
    const void* x;
    const void* dy;
    const void* w;
    void* out;
    int64_t x_token, x_head, dy_token, dy_head;
    int32_t heads;
};

struct RotArgs {
    Rows r[2];                 // queries, keys
    const int64_t* positions;
    const float* table;        // [positions][rotary]: cos, then sin; NULL: no rotation
    int64_t tokens, table_rows;
    int32_t dim, rotary, interleaved, norm;
    float eps;
    float* partial;            // backward: [blocks][2][dim], NULL: no weight gradients
};

template <typename E>
__device__ __forceinline__ float to_f(E v) {
    if constexpr (sizeof(E) == 2) return __bfloat162float(v);
    else return v;
}

template <typename E>
__device__ __forceinline__ E from_f(float v) {
    if constexpr (sizeof(E) == 2) return __float2bfloat16_rn(v);
    else return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(kFull, v, s);
    return v;
}

// Turns the row in `s` (shared memory) and returns element e; `sign` -1: back.
// cs: the position's cos and sin, NULL: the position is outside the table.
__device__ __forceinline__ float turned(const RotArgs& a, const float* s, const float* cs, int e, float sign) {
    if (e >= a.rotary || !a.table) return s[e];
    const int half = a.rotary / 2;
    const int pair = a.interleaved ? e / 2 : e < half ? e : e - half;
    const bool second = a.interleaved ? (e & 1) != 0 : e >= half;
    const int other = a.interleaved ? e ^ 1 : second ? e - half : e + half;
    const float c = cs ? cs[pair] : __int_as_float(0x7fffffff), n = cs ? cs[half + pair] : c;
    return fmaf(s[e], c, (second ? sign : -sign) * s[other] * n);
}

template <typename E, bool kBack>
__global__ void __launch_bounds__(32 * kWarps) rows_kernel(const __grid_constant__ RotArgs a) {
    __shared__ float rows[kWarps][kMaxDim];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float* s = rows[warp];
    for (int part = 0; part < 2; ++part) {
        const Rows& R = a.r[part];
        float dw[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) dw[i] = 0.0f;
        const int64_t n = a.tokens * R.heads;
        for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp; row < n; row += gridDim.x * kWarps) {
            const int64_t token = row / R.heads, head = row - token * R.heads;
            const float* cs = nullptr;
            if (a.table) {
                const int64_t p = a.positions[token];
                if (p >= 0 && p < a.table_rows) cs = a.table + p * a.rotary;
            }
            const E* px = static_cast<const E*>(R.x) + token * R.x_token + head * R.x_head;
            const E* w = static_cast<const E*>(R.w);
            E* out = static_cast<E*>(R.out) + row * a.dim;
            float x[kPer], r = 1.0f;
            if (!kBack || a.norm) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[i] = lane + 32 * i < a.dim ? to_f<E>(px[lane + 32 * i]) : 0.0f;
            }
            if (a.norm) {
                float q = 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) q = fmaf(x[i], x[i], q);
                r = 1.0f / sqrtf(warp_sum(q) / static_cast<float>(a.dim) + a.eps);
            }
            if constexpr (!kBack) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.dim) s[e] = a.norm ? x[i] * r * (w ? to_f<E>(w[e]) : 1.0f) : x[i];
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.dim) out[e] = from_f<E>(turned(a, s, cs, e, 1.0f));
                }
            } else {
                const E* pd = static_cast<const E*>(R.dy) + token * R.dy_token + head * R.dy_head;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.dim) s[e] = to_f<E>(pd[e]);
                }
                __syncwarp();
                float g[kPer], dot = 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int e = lane + 32 * i;
                    g[i] = e < a.dim ? turned(a, s, cs, e, -1.0f) : 0.0f;
                    if (a.norm && e < a.dim) {
                        x[i] *= r;
                        dw[i] = fmaf(g[i], x[i], dw[i]);
                        if (w) g[i] *= to_f<E>(w[e]);
                        dot = fmaf(g[i], x[i], dot);
                    }
                }
                if (a.norm) dot = warp_sum(dot) / static_cast<float>(a.dim);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.dim) out[e] = from_f<E>(a.norm ? r * (g[i] - x[i] * dot) : g[i]);
                }
            }
            __syncwarp();
        }
        if constexpr (kBack) {
            if (!a.partial) continue;
            // the block's sums, warp after warp
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kPer; ++i) s[lane + 32 * i] = dw[i];
            __syncthreads();
            for (int e = threadIdx.x; e < a.dim; e += 32 * kWarps) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) sum += rows[k][e];
                a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + part) * a.dim + e] = sum;
            }
            __syncthreads();
        }
    }
}

// Weight gradients from the partial sums [n][2][dim], always in the same order: 32
// columns per block, 32 threads each.
template <typename E>
__global__ void __launch_bounds__(1024) reduce_kernel(const float* partial, int n, int dim, void* dq, void* dk) {
    __shared__ float sums[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x % 32, group = threadIdx.x / 32;
    float sum = 0.0f;
    if (col < 2 * dim)
        for (int i = group; i < n; i += 32) sum += partial[static_cast<int64_t>(i) * 2 * dim + col];
    sums[group][threadIdx.x % 32] = sum;
    __syncthreads();
    if (group != 0 || col >= 2 * dim) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sums[i][threadIdx.x];
    void* out = col < dim ? dq : dk;
    if (out) static_cast<E*>(out)[col < dim ? col : col - dim] = from_f<E>(sum);
}

// cos and sin of position * base^(-2 i / rotary), in 64 bits until they are rounded:
// far positions are many turns, of which 32 bits lose the fraction.
__global__ void __launch_bounds__(256) table_kernel(float* table, int64_t positions, int rotary, double log2_base) {
    const int half = rotary / 2;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < positions * half;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t p = i / half, k = i - p * half;
        double s, c;
        sincos(static_cast<double>(p) * exp2(-2.0 * static_cast<double>(k) / rotary * log2_base), &s, &c);
        table[p * rotary + k] = static_cast<float>(c);
        table[p * rotary + half + k] = static_cast<float>(s);
    }
}

int check_heads(const dmuon_heads_t* t, int64_t tokens, int64_t heads, int64_t dim, int es, const char* name,
                const char* where) {
    if (!t) return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": " + name + " is NULL");
    OPS_TRY(check_ptr(t->p, name, where, static_cast<size_t>(es)));
    const int64_t most = int64_t(1) << 36;
    if ((tokens > 1 && !in_range(t->token_stride, dim, most)) || (heads > 1 && !in_range(t->head_stride, dim, most)))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": strides of " + name + " must be at least dim, and at most 2^36");
    return DMUON_OK;
}

bool sizes_ok(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim) {
    return in_range(tokens, 0, kMaxTokens) && in_range(heads, 1, kMaxHeads) && in_range(kv_heads, 1, kMaxHeads) &&
           in_range(dim, 1, kMaxDim);
}

int blocks_of(int64_t tokens, int heads, int kv_heads) {
    return static_cast<int>(
        std::min<int64_t>(std::max<int64_t>(1, ceil_div(tokens * std::max(heads, kv_heads), kWarps)), kMaxPartials));
}

// What both directions check, and the arguments they share.
int common(RotArgs& a, const int64_t* positions, const float* table, int64_t table_rows, int32_t rotary,
           int32_t interleaved, const void* q_weight, const void* k_weight, int32_t norm, float eps, int64_t tokens,
           int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype, const char* where) {
    if (!sizes_ok(tokens, heads, kv_heads, dim))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": tokens must be in [0, 2^24], heads and kv_heads in "
                                                                "[1, 1024], dim in [1, 256]");
    OPS_TRY(check_dtype(dtype, where));
    if (table) {
        if (rotary % 2 != 0 || !in_range(rotary, 2, dim))
            return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": rotary must be even and in [2, dim]");
        if (!in_range(table_rows, 1, kMaxTokens))
            return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": table_rows must be in [1, 2^24]");
        OPS_TRY(check_ptr(table, "table", where));
        if (tokens > 0) OPS_TRY(check_ptr(positions, "positions", where, 8));
    }
    if (!norm && (q_weight || k_weight))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": weights without the norm");
    if (norm && !(eps >= 0.0f && std::isfinite(eps)))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": eps must be finite and >= 0");
    if (q_weight) OPS_TRY(check_ptr(q_weight, "q_weight", where));
    if (k_weight) OPS_TRY(check_ptr(k_weight, "k_weight", where));
    a.positions = positions;
    a.table = table;
    a.tokens = tokens;
    a.table_rows = table_rows;
    a.dim = dim;
    a.rotary = table ? rotary : 0;
    a.interleaved = interleaved != 0;
    a.norm = norm != 0;
    a.eps = eps;
    a.r[0].w = q_weight;
    a.r[1].w = k_weight;
    a.r[0].heads = heads;
    a.r[1].heads = kv_heads;
    return DMUON_OK;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" int dmuon_rotary_table(float* table, int64_t positions, int32_t rotary, double base, void* stream) {
    const char* where = "dmuon_rotary_table";
    if (!in_range(positions, 0, kMaxTokens) || rotary % 2 != 0 || !in_range(rotary, 2, kMaxDim))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": positions must be in [0, 2^24], rotary even and in [2, 256]");
    if (!(base > 0.0) || !std::isfinite(base))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": base must be finite and > 0");
    if (positions == 0) return DMUON_OK;
    OPS_TRY(check_ptr(table, "table", where));
    OPS_TRY(check_device(where));
    const int64_t blocks = std::min<int64_t>(ceil_div(positions * (rotary / 2), 256), 2432);
    table_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(table, positions, rotary,
                                                                                             std::log2(base));
    OPS_CUDA(cudaGetLastError());
    return DMUON_OK;
}

extern "C" size_t dmuon_qk_norm_rotary_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim,
                                                       int32_t dtype) {
    if (!sizes_ok(tokens, heads, kv_heads, dim) ||
        check_dtype(dtype, "dmuon_qk_norm_rotary_workspace_bytes") != DMUON_OK)
        return 0;
    return static_cast<size_t>(blocks_of(tokens, heads, kv_heads)) * 2 * dim * sizeof(float);
}

extern "C" int dmuon_qk_norm_rotary_forward(const dmuon_heads_t* q, const dmuon_heads_t* k, const int64_t* positions,
                                            const float* table, int64_t table_rows, int32_t rotary,
                                            int32_t interleaved, const void* q_weight, const void* k_weight,
                                            int32_t norm, float eps, void* q_out, void* k_out, int64_t tokens,
                                            int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype, void* stream) {
    const char* where = "dmuon_qk_norm_rotary_forward";
    RotArgs a = {};
    OPS_TRY(common(a, positions, table, table_rows, rotary, interleaved, q_weight, k_weight, norm, eps, tokens, heads,
                   kv_heads, dim, dtype, where));
    if (tokens == 0) return DMUON_OK;
    const int es = dtype == DMUON_FP32 ? 4 : 2;
    OPS_TRY(check_heads(q, tokens, heads, dim, es, "q", where));
    OPS_TRY(check_heads(k, tokens, kv_heads, dim, es, "k", where));
    OPS_TRY(check_ptr(q_out, "q_out", where));
    OPS_TRY(check_ptr(k_out, "k_out", where));
    OPS_TRY(check_device(where));
    const dmuon_heads_t* in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        a.r[i].x = in[i]->p;
        a.r[i].x_token = in[i]->token_stride;
        a.r[i].x_head = in[i]->head_stride;
    }
    a.r[0].out = q_out;
    a.r[1].out = k_out;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid =
        static_cast<unsigned>(std::min<int64_t>(ceil_div(tokens * std::max(heads, kv_heads), kWarps), 152 * 8 * 4));
    if (dtype == DMUON_FP32) rows_kernel<float, false><<<grid, 32 * kWarps, 0, s>>>(a);
    else rows_kernel<__nv_bfloat16, false><<<grid, 32 * kWarps, 0, s>>>(a);
    OPS_CUDA(cudaGetLastError());
    return DMUON_OK;
}

extern "C" int dmuon_qk_norm_rotary_backward(const dmuon_heads_t* dq_out, const dmuon_heads_t* dk_out,
                                             const dmuon_heads_t* q, const dmuon_heads_t* k, const int64_t* positions,
                                             const float* table, int64_t table_rows, int32_t rotary,
                                             int32_t interleaved, const void* q_weight, const void* k_weight,
                                             int32_t norm, float eps, void* dq, void* dk, void* dq_weight,
                                             void* dk_weight, int64_t tokens, int32_t heads, int32_t kv_heads,
                                             int32_t dim, int32_t dtype, void* workspace, size_t workspace_bytes,
                                             void* stream) {
    const char* where = "dmuon_qk_norm_rotary_backward";
    RotArgs a = {};
    OPS_TRY(common(a, positions, table, table_rows, rotary, interleaved, q_weight, k_weight, norm, eps, tokens, heads,
                   kv_heads, dim, dtype, where));
    if (!norm && (dq_weight || dk_weight))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": weights' gradients without the norm");
    const bool sums = dq_weight || dk_weight;
    if (dq_weight) OPS_TRY(check_ptr(dq_weight, "dq_weight", where));
    if (dk_weight) OPS_TRY(check_ptr(dk_weight, "dk_weight", where));
    const int es = dtype == DMUON_FP32 ? 4 : 2;
    if (tokens > 0) {
        const dmuon_heads_t *x[2] = {q, k}, *dy[2] = {dq_out, dk_out};
        const char *xn[2] = {"q", "k"}, *dn[2] = {"dq_out", "dk_out"};
        void* out[2] = {dq, dk};
        for (int i = 0; i < 2; ++i) {
            const int h = i ? kv_heads : heads;
            OPS_TRY(check_heads(dy[i], tokens, h, dim, es, dn[i], where));
            if (norm) {
                OPS_TRY(check_heads(x[i], tokens, h, dim, es, xn[i], where));
                a.r[i].x = x[i]->p;
                a.r[i].x_token = x[i]->token_stride;
                a.r[i].x_head = x[i]->head_stride;
            }
            OPS_TRY(check_ptr(out[i], i ? "dk" : "dq", where));
            a.r[i].dy = dy[i]->p;
            a.r[i].dy_token = dy[i]->token_stride;
            a.r[i].dy_head = dy[i]->head_stride;
            a.r[i].out = out[i];
        }
    }
    if (sums)
        OPS_TRY(check_workspace(workspace, workspace_bytes,
                                dmuon_qk_norm_rotary_workspace_bytes(tokens, heads, kv_heads, dim, dtype), where));
    if (tokens == 0 && !sums) return DMUON_OK;
    OPS_TRY(check_device(where));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = dtype == DMUON_FP32;
    const int blocks = tokens > 0 ? blocks_of(tokens, heads, kv_heads) : 0;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    if (blocks > 0) {
        if (f32) rows_kernel<float, true><<<blocks, 32 * kWarps, 0, s>>>(a);
        else rows_kernel<__nv_bfloat16, true><<<blocks, 32 * kWarps, 0, s>>>(a);
        OPS_CUDA(cudaGetLastError());
    }
    if (sums) {
        const unsigned grid = static_cast<unsigned>(ceil_div(2 * dim, 32));
        if (f32) reduce_kernel<float><<<grid, 1024, 0, s>>>(a.partial, blocks, dim, dq_weight, dk_weight);
        else reduce_kernel<__nv_bfloat16><<<grid, 1024, 0, s>>>(a.partial, blocks, dim, dq_weight, dk_weight);
        OPS_CUDA(cudaGetLastError());
    }
    return DMUON_OK;
}
