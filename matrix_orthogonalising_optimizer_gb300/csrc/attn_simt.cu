// Attention in fp32 FFMA arithmetic, forward and backward: fp32 tensors, and bf16
// ones whose rows begin off 16-byte boundaries although their length is a multiple of 16 bytes.
//
//   s_ij = scale q_i k_j over the keys j that i sees,  lse_i = log sum_j exp s_ij
//   p = exp(s - lse),  o_i = sum_j p_ij v_j
//   ds_ij = p_ij (do_i v_j - delta_i),  delta_i = do_i o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// One pass over the keys per 64 (or 32) queries with the running maximum and sum of the
// softmax; the backward pass takes p from lse, once per 64 queries for dq and once
// per 64 keys for dk and dv (summed over the query heads that share the key head), so
// every sum has one owner and a fixed order.  A block of 256 threads forms 64 x 64
// products, 4 x 4 per thread; all tiles lie row by row in shared memory as fp32,
// dim + 4 floats apart: 16-byte reads of eight rows then cover all banks.
//
// Bound: FFMA (about half of its rate) and shared-memory loads (4 x 4 products take 8 loads of
// 2 cycles each per 32 FMA instructions); a second block per SM adds nothing.  Measured in
// fp32: 2048 tokens, 16 heads of 64, causal: forward 231 us (19 TFLOP/s), backward 720 us (30);
// 777 tokens, 6 / 2 heads of 80: 36 and 70 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "act.cuh"
#include "attn.h"
#include "internal.h"
#include "ops.h"
#include "tc.cuh"

namespace dmuon {
namespace {

constexpr int T = 64;           // keys of a tile (side of the keys: and queries)
constexpr int kThreads = 256;   // 16 x 16: thread (ty, tx) holds rows ty + 16 r, columns tx + 16 c
constexpr int LP = T + 16;      // row stride of a T x T tile: a warp's two rows on different banks
constexpr unsigned kFull = 0xffffffffu;

// A warp holds two rows of threads, in alternate lanes: neighbours then read the same
// 16 bytes of a column's operand, and the load takes two cycles of the shared memory; with a
// half warp per row it takes four (777 tokens: forward 45 -> 37 us, backward 82 -> 68).
__device__ __forceinline__ int row_of() { return threadIdx.x / 32 * 2 + threadIdx.x % 2; }
__device__ __forceinline__ int col_of() { return threadIdx.x % 32 / 2; }

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

// N rows of a head on their way into shared memory, zero behind `rows` and `dim`.  fetch()
// has all loads in flight at once and may run well before put(), so that a tile's
// latency falls under the products of the one before.  `vec`: rows start on 16-byte
// boundaries and dim is a multiple of 4; else put() loads element by element.
template <typename E, int DP, int N = T>
struct Tile {
    static constexpr int LD = DP + 4, kEach = N * (DP / 4) / kThreads;
    using Word = typename std::conditional<sizeof(E) == 4, float4, uint2>::type;
    Word v[kEach];

    __device__ __forceinline__ void fetch(const AttnHeads& h, int64_t row0, int rows, int head, int dim, bool vec) {
        if (!vec) return;
        const E* base = static_cast<const E*>(h.p) + row0 * h.token + head * h.head;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads, r = i / (DP / 4), c = i % (DP / 4) * 4;
            v[k] = Word{};
            if (r < rows && c < dim) v[k] = *reinterpret_cast<const Word*>(base + r * h.token + c);
        }
    }
    __device__ __forceinline__ void put(float* dst, const AttnHeads& h, int64_t row0, int rows, int head, int dim,
                                        bool vec) const {
        if (vec) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x + k * kThreads, r = i / (DP / 4), c = i % (DP / 4) * 4;
                float4 x;
                if constexpr (sizeof(E) == 4) {
                    x = v[k];
                } else {
                    const float2 a = tc::unpack_bf16x2(v[k].x), b = tc::unpack_bf16x2(v[k].y);
                    x = make_float4(a.x, a.y, b.x, b.y);
                }
                *reinterpret_cast<float4*>(dst + r * LD + c) = x;
            }
            return;
        }
        const E* base = static_cast<const E*>(h.p) + row0 * h.token + head * h.head;
#pragma unroll 4
        for (int i = threadIdx.x; i < N * DP; i += kThreads) {
            const int r = i / DP, c = i % DP;
            dst[r * LD + c] = r < rows && c < dim ? to_f<E>(base[r * h.token + c]) : 0.0f;
        }
    }
};

template <typename E, int DP, int N = T>
__device__ __forceinline__ void load_tile(float* dst, const AttnHeads& h, int64_t row0, int rows, int head, int dim,
                                          bool vec) {
    Tile<E, DP, N> t;
    t.fetch(h, row0, rows, head, dim, vec);
    t.put(dst, h, row0, rows, head, dim, vec);
}

// Two tiles of the same rows.
template <typename E, int DP>
struct Pair {
    Tile<E, DP> a, b;
    __device__ __forceinline__ void fetch(const AttnHeads& ha, const AttnHeads& hb, int64_t row0, int rows, int head,
                                          int dim, bool va, bool vb) {
        a.fetch(ha, row0, rows, head, dim, va);
        b.fetch(hb, row0, rows, head, dim, vb);
    }
    __device__ __forceinline__ void put(float* da, float* db, const AttnHeads& ha, const AttnHeads& hb, int64_t row0,
                                        int rows, int head, int dim, bool va, bool vb) const {
        a.put(da, ha, row0, rows, head, dim, va);
        b.put(db, hb, row0, rows, head, dim, vb);
    }
};

// acc[r][c] = sum_d A[ty + 16 r][d] B[tx + 16 c][d].  Packed arithmetic (two products an
// instruction, the same rate) leaves the issue slots that the loads need.
template <int DP, int R>
__device__ __forceinline__ void product_nt(float (&acc)[R][4], const float* A, const float* B, int dim4) {
    constexpr int LD = DP + 4;
    const float* a0 = A + row_of() * LD;
    const float* b0 = B + col_of() * LD;
    float2 sum[R][4];  // even and odd d
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[r][c] = tc::both(0.0f);
#pragma unroll 4
    for (int d = 0; d < dim4; d += 4) {
        float4 a[R], b[4];
#pragma unroll
        for (int r = 0; r < R; ++r) a[r] = *reinterpret_cast<const float4*>(a0 + 16 * r * LD + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4*>(b0 + 16 * c * LD + d);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sum[r][c] = tc::fma2(make_float2(a[r].x, a[r].y), make_float2(b[c].x, b[c].y), sum[r][c]);
                sum[r][c] = tc::fma2(make_float2(a[r].z, a[r].w), make_float2(b[c].z, b[c].w), sum[r][c]);
            }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = sum[r][c].x + sum[r][c].y;
}

// acc[r][k] += sum_j P[ty + 16 r][j] V[j][4 tx + 64 (k / 2) + 2 (k % 2) ..]
template <int DP, int R>
__device__ __forceinline__ void product_nn(float2 (&acc)[R][DP / 32], const float* P, const float* V) {
    constexpr int LD = DP + 4;
    const float* p0 = P + row_of() * LP;
    const float* v0 = V + 4 * col_of();
#pragma unroll 4
    for (int j = 0; j < T; j += 4) {
        float4 p[R];
#pragma unroll
        for (int r = 0; r < R; ++r) p[r] = *reinterpret_cast<const float4*>(p0 + 16 * r * LP + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(v0 + (j + jj) * LD + 64 * c);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 w = tc::both(jj == 0 ? p[r].x : jj == 1 ? p[r].y : jj == 2 ? p[r].z : p[r].w);
                    acc[r][2 * c] = tc::fma2(w, make_float2(v.x, v.y), acc[r][2 * c]);
                    acc[r][2 * c + 1] = tc::fma2(w, make_float2(v.z, v.w), acc[r][2 * c + 1]);
                }
            }
    }
}

// Rows ty + 16 r < rows of a contiguous tokens x heads x dim tensor, times f[r].
template <typename E, int DP, int R>
__device__ __forceinline__ void store_rows(void* out, const float2 (&acc)[R][DP / 32], const float (&f)[R],
                                           int64_t row0, int rows, int heads, int head, int dim) {
    const int ty = row_of(), tx = col_of();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = ty + 16 * r;
        if (i >= rows) continue;
        E* p = static_cast<E*>(out) + ((row0 + i) * heads + head) * static_cast<int64_t>(dim);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            const int d = 4 * tx + 64 * (k / 4) + k % 4;
            if (d < dim) p[d] = from_f<E>((k % 2 ? acc[r][k / 2].y : acc[r][k / 2].x) * f[r]);
        }
    }
}

// Sum and maximum over the 16 lanes that share a row.
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int s = 16; s >= 2; s >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, s));
    return v;
}

__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int s = 16; s >= 2; s >>= 1) v += __shfl_xor_sync(kFull, v, s);
    return v;
}

// Whether row i of a sequence sees one key only: p is 1 then and ds exactly 0, not what the
// roundings of dp and delta leave of it.
__device__ __forceinline__ bool single(const AttnTile& t, const AttnArgs& a, int i) {
    return a.causal ? i == 0 : t.len == 1;
}

struct Block {
    AttnTile t;
    int head, row0, rows, tiles;
};

// The share of the rows of no sequence that a block behind the tiles' clears; else negative.
__device__ __forceinline__ int clear_share(const AttnArgs& a, unsigned block, unsigned tiles) {
    return block < tiles * static_cast<unsigned>(a.slots) ? -1 : static_cast<int>(block - tiles * a.slots);
}

// The block's tile: heads run fastest, tiles of a sequence from its end where the
// last ones have most to do (`last_first`).  False: the slot holds none.
template <int N>
__device__ __forceinline__ bool take_block(const AttnArgs& a, unsigned block, int heads, bool last_first, Block& b) {
    const int slot = static_cast<int>(block / static_cast<unsigned>(heads));
    b.head = static_cast<int>(block - static_cast<unsigned>(slot) * heads);
    if (!attn_find(a, slot, N, b.t)) return false;
    b.tiles = (b.t.len + N - 1) / N;
    const int tile = last_first ? b.tiles - 1 - b.t.tile : b.t.tile;
    b.row0 = tile * N;
    b.rows = min(N, b.t.len - b.row0);
    return true;
}

template <typename E>
__device__ __forceinline__ bool vec_rows(const AttnHeads& h, int dim) {
    constexpr int n = 16 / sizeof(E);
    return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.token % n == 0 && h.head % n == 0 && dim % 4 == 0;
}

template <typename E, int DP, int R>
__global__ void __launch_bounds__(kThreads, 1) forward_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int LD = DP + 4;
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + 16 * R * LD, *V = K + T * LD, *P = V + T * LD;
    Block b;
    const int share = clear_share(a, blockIdx.x, a.heads);
    if (share >= 0) {
        attn_clear(a, static_cast<E*>(a.out), a.lse, a.heads, share, threadIdx.x, kThreads);
        return;
    }
    if (!take_block<16 * R>(a, blockIdx.x, a.heads, a.causal != 0, b)) return;
    const int kv = b.head / a.group, dim4 = (a.dim + 3) / 4 * 4;
    const int ty = row_of(), tx = col_of();
    const bool vk = vec_rows<E>(a.k, a.dim), vv = vec_rows<E>(a.v, a.dim);
    load_tile<E, DP, 16 * R>(Q, a.q, b.t.begin + b.row0, b.rows, b.head, a.dim, vec_rows<E>(a.q, a.dim));
    float2 acc[R][DP / 32];
    float top[R], base[R], sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        top[r] = __int_as_float(0xff800000);
        base[r] = 0.0f;
        sum[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < DP / 32; ++k) acc[r][k] = tc::both(0.0f);
    }
    const int end = a.causal ? b.row0 + b.rows : b.t.len;  // keys that any of the rows sees
    Pair<E, DP> next;
    next.fetch(a.k, a.v, b.t.begin, min(T, b.t.len), kv, a.dim, vk, vv);
    for (int j0 = 0; j0 < end; j0 += T) {
        const int keys = min(T, b.t.len - j0);
        __syncthreads();
        next.put(K, V, a.k, a.v, b.t.begin + j0, keys, kv, a.dim, vk, vv);
        __syncthreads();
        if (j0 + T < end) next.fetch(a.k, a.v, b.t.begin + j0 + T, min(T, b.t.len - j0 - T), kv, a.dim, vk, vv);
        float s[R][4];
        product_nt<DP>(s, Q, K, dim4);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = b.row0 + ty + 16 * r;
            const int seen = a.causal ? min(i + 1 - j0, keys) : keys;
            float m = top[r];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (tx + 16 * c >= seen) s[r][c] = __int_as_float(0xff800000);
                m = fmaxf(m, s[r][c]);
            }
            m = row_max(m);
            // what is subtracted is rounded, the same for all of a row's exponentials: the
            // factor between two maxima comes from the rounded values, and is exactly 1 where
            // the maximum stays
            const float fresh = exp_shift(m) * a.scale_log2;
            const float old = top[r] == __int_as_float(0xff800000) ? 0.0f : ex2(base[r] - fresh);
            top[r] = m;
            base[r] = fresh;
            float part = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float e = ex2(fmaf(s[r][c], a.scale_log2, -fresh));
                part += e;
                P[(ty + 16 * r) * LP + tx + 16 * c] = e;
            }
            sum[r] = fmaf(sum[r], old, row_sum(part));
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) acc[r][k] = tc::mul2(acc[r][k], tc::both(old));
        }
        __syncwarp();  // a row of P is written and read by one warp
        product_nn<DP>(acc, P, V);
    }
    float f[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        f[r] = 1.0f / sum[r];
        const int i = ty + 16 * r;
        if (tx == 0 && i < b.rows)
            a.lse[b.head * a.tokens + b.t.begin + b.row0 + i] =
                (base[r] + log2f(sum[r])) * 0.6931471805599453f;
    }
    store_rows<E, DP>(a.out, acc, f, b.t.begin + b.row0, b.rows, a.heads, b.head, a.dim);
}

template <typename E, int DP, int R>
__device__ __forceinline__ void dq_block(const AttnArgs& a, unsigned index, float* sm) {
    constexpr int LD = DP + 4;
    float *Q = sm, *O = Q + 16 * R * LD, *K = O + 16 * R * LD, *V = K + T * LD, *P = V + T * LD;
    Block b;
    const int share = clear_share(a, index, a.heads);
    if (share >= 0) {
        attn_clear(a, static_cast<E*>(a.out), nullptr, a.heads, share, threadIdx.x, kThreads);
        return;
    }
    if (!take_block<16 * R>(a, index, a.heads, a.causal != 0, b)) return;
    const int kv = b.head / a.group, dim4 = (a.dim + 3) / 4 * 4;
    const int ty = row_of(), tx = col_of();
    const bool vk = vec_rows<E>(a.k, a.dim), vv = vec_rows<E>(a.v, a.dim);
    const int64_t row = b.t.begin + b.row0;
    load_tile<E, DP, 16 * R>(Q, a.q, row, b.rows, b.head, a.dim, vec_rows<E>(a.q, a.dim));
    load_tile<E, DP, 16 * R>(O, a.d_o, row, b.rows, b.head, a.dim, vec_rows<E>(a.d_o, a.dim));
    float2 acc[R][DP / 32];
    float lse[R], delta[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = ty + 16 * r;
        const bool in = i < b.rows;
        lse[r] = in ? a.lse[b.head * a.tokens + row + i] * kLog2e : 0.0f;
        delta[r] = in && sizeof(E) == 4 && !single(b.t, a, b.row0 + i) ? a.delta[b.head * a.tokens + row + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < DP / 32; ++k) acc[r][k] = tc::both(0.0f);
    }
    const int end = a.causal ? b.row0 + b.rows : b.t.len;
    Pair<E, DP> next;
    const auto fetch = [&](int j0) {
        next.fetch(a.k, a.v, b.t.begin + j0, min(T, b.t.len - j0), kv, a.dim, vk, vv);
    };
    // p and dp of the keys from j0 on, 0 where a row sees none
    const auto form = [&](int j0, float (&p)[R][4], float (&g)[R][4]) {
        const int keys = min(T, b.t.len - j0);
        __syncthreads();
        next.put(K, V, a.k, a.v, b.t.begin + j0, keys, kv, a.dim, vk, vv);
        __syncthreads();
        if (j0 + T < end) fetch(j0 + T);
        product_nt<DP>(p, Q, K, dim4);
        product_nt<DP>(g, O, V, dim4);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = b.row0 + ty + 16 * r;
            const int seen = a.causal ? min(i + 1 - j0, keys) : keys;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool in = tx + 16 * c < seen;
                p[r][c] = in ? ex2(fmaf(p[r][c], a.scale_log2, -lse[r])) : 0.0f;
                g[r][c] = in && !single(b.t, a, i) ? g[r][c] : 0.0f;
            }
        }
    };
    if constexpr (sizeof(E) == 2) {
        // delta = sum p dp, in a pass of its own: do . o would hold the rounding of o to
        // bf16, which shows where few keys count (dp - delta is then small beside dp)
#pragma unroll
        for (int r = 0; r < R; ++r) delta[r] = 0.0f;
        fetch(0);
        for (int j0 = 0; j0 < end; j0 += T) {
            float p[R][4], g[R][4];
            form(j0, p, g);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) delta[r] = fmaf(p[r][c], g[r][c], delta[r]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            delta[r] = row_sum(delta[r]);
            const int i = ty + 16 * r;
            if (tx == 0 && i < b.rows) a.delta[b.head * a.tokens + row + i] = delta[r];
        }
    }
    fetch(0);
    for (int j0 = 0; j0 < end; j0 += T) {
        float p[R][4], g[R][4];
        form(j0, p, g);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) P[(ty + 16 * r) * LP + tx + 16 * c] = p[r][c] * (g[r][c] - delta[r]);
        __syncwarp();
        product_nn<DP>(acc, P, K);
    }
    float f[R];
#pragma unroll
    for (int r = 0; r < R; ++r) f[r] = a.scale;
    store_rows<E, DP>(a.out, acc, f, row, b.rows, a.heads, b.head, a.dim);
}

template <typename E, int DP>
__device__ __forceinline__ void dkv_block(const AttnArgs& a, unsigned index, float* sm) {
    constexpr int LD = DP + 4;
    float *K = sm, *V = K + T * LD, *Q = V + T * LD, *O = Q + T * LD, *P = O + T * LD, *G = P + T * LP;
    Block b;
    const int share = clear_share(a, index, a.kv_heads * a.parts);
    if (share >= 0) {
        const auto clear = [&](auto* x) { attn_clear(a, x, nullptr, a.kv_heads, share, threadIdx.x, kThreads); };
        if (a.parts > 1) {
            for (int k = 0; k < 2 * a.parts; ++k) clear(attn_partial(a, 0, k));
        } else {
            clear(static_cast<E*>(a.dk));
            clear(static_cast<E*>(a.dv));
        }
        return;
    }
    const int part = static_cast<int>(index % static_cast<unsigned>(a.parts));
    if (!take_block<T>(a, index / static_cast<unsigned>(a.parts), a.kv_heads, false, b)) return;
    const int dim4 = (a.dim + 3) / 4 * 4, ty = row_of(), tx = col_of();
    const bool vq = vec_rows<E>(a.q, a.dim), vo = vec_rows<E>(a.d_o, a.dim);
    const int64_t row = b.t.begin + b.row0;
    load_tile<E, DP>(K, a.k, row, b.rows, b.head, a.dim, vec_rows<E>(a.k, a.dim));
    load_tile<E, DP>(V, a.v, row, b.rows, b.head, a.dim, vec_rows<E>(a.v, a.dim));
    float2 dk[4][DP / 32], dv[4][DP / 32];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < DP / 32; ++k) dk[r][k] = dv[r][k] = tc::both(0.0f);
    const int first = a.causal ? b.row0 : 0;  // the first query that sees any of the keys
    const int per_head = (b.t.len - first + T - 1) / T, steps = per_head * a.group;
    const int end = attn_part(steps, part + 1, a.parts);
    for (int step = attn_part(steps, part, a.parts); step < end; ++step) {
        const int h = step / per_head, head = b.head * a.group + h, i0 = first + (step - h * per_head) * T;
        const int queries = min(T, b.t.len - i0);
        Pair<E, DP> tiles;
        tiles.fetch(a.q, a.d_o, b.t.begin + i0, queries, head, a.dim, vq, vo);
        __syncthreads();
        tiles.put(Q, O, a.q, a.d_o, b.t.begin + i0, queries, head, a.dim, vq, vo);
        __syncthreads();
        float s[4][4], g[4][4];
        product_nt<DP>(s, K, Q, dim4);
        product_nt<DP>(g, V, O, dim4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = tx + 16 * c;
            const int64_t at = head * a.tokens + b.t.begin + i0 + i;
            const bool in = i < queries;
            const float lse = in ? a.lse[at] * kLog2e : 0.0f, delta = in ? a.delta[at] : 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = ty + 16 * r;
                const bool seen = in && (!a.causal || b.row0 + j <= i0 + i);
                const float p = seen ? ex2(fmaf(s[r][c], a.scale_log2, -lse)) : 0.0f;
                P[j * LP + i] = p;
                G[j * LP + i] = seen && !single(b.t, a, i0 + i) ? p * (g[r][c] - delta) : 0.0f;
            }
        }
        __syncwarp();
        product_nn<DP>(dv, P, O);
        product_nn<DP>(dk, G, Q);
    }
    const float one[4] = {1.0f, 1.0f, 1.0f, 1.0f}, f[4] = {a.scale, a.scale, a.scale, a.scale};
    if (a.parts > 1) {
        store_rows<float, DP>(attn_partial(a, 1, part), dv, one, row, b.rows, a.kv_heads, b.head, a.dim);
        store_rows<float, DP>(attn_partial(a, 0, part), dk, one, row, b.rows, a.kv_heads, b.head, a.dim);
        return;
    }
    store_rows<E, DP>(a.dv, dv, one, row, b.rows, a.kv_heads, b.head, a.dim);
    store_rows<E, DP>(a.dk, dk, f, row, b.rows, a.kv_heads, b.head, a.dim);
}

// `keys` blocks for dk and dv, and behind them those for dq, 16 R queries each.
template <typename E, int DP, int R>
__global__ void __launch_bounds__(kThreads, 1) backward_kernel(const __grid_constant__ AttnArgs a, unsigned keys) {
    extern __shared__ float sm[];
    if (blockIdx.x < keys) {
        dkv_block<E, DP>(a, blockIdx.x, sm);
        return;
    }
    AttnArgs q = a;
    q.slots = a.query_slots;
    dq_block<E, DP, R>(q, blockIdx.x - keys, sm);
}

// dk (y = 0) and dv (1) from the partial sums of a.parts blocks, N elements a thread.
template <typename E, int N>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    struct __align__(4 * N) In { float v[N]; };
    struct __align__(sizeof(E) * N) Out { E v[N]; };
    const int64_t n = a.tokens * a.kv_heads * a.dim;
    const bool v = blockIdx.y != 0;
    const float* p = attn_partial(a, v ? 1 : 0, 0);
    E* out = static_cast<E*>(v ? a.dv : a.dk);
    const float f = v ? 1.0f : a.scale;
    for (int64_t i = (blockIdx.x * 256ll + threadIdx.x) * N; i < n; i += gridDim.x * 256ll * N) {
        float sum[N] = {};
#pragma unroll 4
        for (int k = 0; k < a.parts; ++k) {
            const In x = *reinterpret_cast<const In*>(p + k * n + i);
#pragma unroll
            for (int c = 0; c < N; ++c) sum[c] += x.v[c];
        }
        Out y;
#pragma unroll
        for (int c = 0; c < N; ++c) y.v[c] = from_f<E>(sum[c] * f);
        *reinterpret_cast<Out*>(out + i) = y;
    }
}

// delta = do . o of the rows of all sequences, one warp per row.
template <typename E>
__global__ void __launch_bounds__(256) delta_kernel(const __grid_constant__ AttnArgs a) {
    const int64_t first = attn_offset(a, 0) * a.heads, rows = attn_offset(a, a.sequences) * a.heads;
    const int lane = threadIdx.x % 32;
    for (int64_t r = first + blockIdx.x * 8ll + threadIdx.x / 32; r < rows; r += gridDim.x * 8ll) {
        const int64_t token = r / a.heads;
        const int head = static_cast<int>(r - token * a.heads);
        const E* o = static_cast<const E*>(a.o) + r * a.dim;
        const E* d = static_cast<const E*>(a.d_o.p) + token * a.d_o.token + head * a.d_o.head;
        float sum = 0.0f;
        for (int c = lane; c < a.dim; c += 32) sum = fmaf(to_f<E>(o[c]), to_f<E>(d[c]), sum);
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
        if (lane == 0) a.delta[head * a.tokens + token] = sum;
    }
}

// The same where rows start on 16-byte boundaries: G lanes a row, 16 bytes each of o and
// do; a warp takes 32 / G * 4 tokens of one head, all their loads in flight, so that what it
// stores lies together (134 MB at 8192 tokens, 32 heads of 128: 22 us, 6.1 TB/s; with a token's
// heads in a row 33 us).
template <typename E, int G>
__global__ void __launch_bounds__(256) delta_vector_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int N = 16 / sizeof(E), R = 32 / G, U = 4;
    const int64_t first = attn_offset(a, 0), end = attn_offset(a, a.sequences);
    const int lane = threadIdx.x % 32, c = lane % G * N;
    // divided in 32 bits: o has fewer than 2^38 elements, a unit at least 2^7
    const uint32_t unit = blockIdx.x * 8u + threadIdx.x / 32, group = unit / static_cast<uint32_t>(a.heads);
    const int head = static_cast<int>(unit - group * static_cast<uint32_t>(a.heads));
    const int64_t token0 = first + static_cast<int64_t>(group) * (R * U) + lane / G;
    const E* po = static_cast<const E*>(a.o) + (token0 * a.heads + head) * a.dim + c;
    const E* pd = static_cast<const E*>(a.d_o.p) + token0 * a.d_o.token + head * a.d_o.head + c;
    uint4 o[U], d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        o[u] = d[u] = make_uint4(0, 0, 0, 0);
        if (c >= a.dim || token0 + u * R >= end) continue;
        o[u] = *reinterpret_cast<const uint4*>(po + static_cast<int64_t>(u * R) * a.heads * a.dim);
        d[u] = *reinterpret_cast<const uint4*>(pd + u * R * a.d_o.token);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t x[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, y[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 2) {
                const float2 p = tc::unpack_bf16x2(x[i]), q = tc::unpack_bf16x2(y[i]);
                sum = fmaf(p.x, q.x, fmaf(p.y, q.y, sum));
            } else {
                sum = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), sum);
            }
        }
#pragma unroll
        for (int s = G / 2; s >= 1; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
        if (lane % G == 0 && token0 + u * R < end) a.delta[head * a.tokens + token0 + u * R] = sum;
    }
}

// Rows of bf16 into padded ones, eight elements a thread; blockIdx.y: q, k, v, do.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnArgs b) {
    const int which = blockIdx.y;
    const AttnHeads& in = which == 0 ? a.q : which == 1 ? a.k : which == 2 ? a.v : a.d_o;
    const AttnHeads& out = which == 0 ? b.q : which == 1 ? b.k : which == 2 ? b.v : b.d_o;
    const uint32_t heads = which % 3 == 0 ? a.heads : a.kv_heads, pieces = static_cast<uint32_t>(b.dim) / 8;
    const int64_t rows = a.tokens * heads, count = rows * pieces;
    const bool small = count < (int64_t(1) << 32);  // divided in 32 bits
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) {
        const int64_t row = small ? static_cast<uint32_t>(i) / pieces : i / pieces;
        const int64_t token = small ? static_cast<uint32_t>(row) / heads : row / heads;
        const int c = static_cast<int>(i - row * pieces) * 8;
        const uint16_t* p = static_cast<const uint16_t*>(in.p) + token * in.token + (row - token * heads) * in.head + c;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = (c + 2 * k < a.dim ? p[2 * k] : 0u) | (c + 2 * k + 1 < a.dim ? p[2 * k + 1] : 0u) << 16;
        static_cast<uint4*>(const_cast<void*>(out.p))[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename E, int G>
void launch_delta_vector(const AttnArgs& a, cudaStream_t s) {
    constexpr int tokens = 32 / G * 4;  // of a warp
    const int64_t units = (a.tokens + tokens - 1) / tokens * a.heads;
    delta_vector_kernel<E, G><<<static_cast<unsigned>((units + 7) / 8), 256, 0, s>>>(a);
}

template <typename E>
cudaError_t run_delta(const AttnArgs& a, cudaStream_t s) {
    constexpr int n = 16 / sizeof(E);
    if (a.dim % n == 0 && reinterpret_cast<uintptr_t>(a.d_o.p) % 16 == 0 && a.d_o.token % n == 0 &&
        a.d_o.head % n == 0) {
        const int lanes = a.dim / n;
        if (lanes <= 4) launch_delta_vector<E, 4>(a, s);
        else if (lanes <= 8) launch_delta_vector<E, 8>(a, s);
        else if (lanes <= 16) launch_delta_vector<E, 16>(a, s);
        else launch_delta_vector<E, 32>(a, s);
    } else {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>((a.tokens * a.heads + 7) / 8, 1216));
        delta_kernel<E><<<grid, 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

// Shared memory: `rows` rows of queries (and of gradients), `tiles` tiles of T rows, and
// `squares` x T logits' rows of stride LP.
constexpr size_t tiles_bytes(int rows, int tiles, int squares, int dp) {
    return static_cast<size_t>((rows + tiles * T) * (dp + 4) + squares * LP) * sizeof(float);
}
template <int DP, int R>
constexpr size_t kForwardBytes = tiles_bytes(16 * R, 2, 16 * R, DP);
template <int DP>
constexpr size_t kBackwardBytes = tiles_bytes(0, 4, 2 * T, DP);  // of the keys' blocks; the queries' take less

template <typename K>
cudaError_t allow(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <typename E, int DP>
cudaError_t attributes() {
    cudaError_t e = allow(forward_kernel<E, DP, 4>, kForwardBytes<DP, 4>);
    if (e == cudaSuccess) e = allow(forward_kernel<E, DP, 2>, kForwardBytes<DP, 2>);
    if (e == cudaSuccess) e = allow(backward_kernel<E, DP, 4>, kBackwardBytes<DP>);
    if (e == cudaSuccess) e = allow(backward_kernel<E, DP, 2>, kBackwardBytes<DP>);
    return e;
}

// Shared-memory attributes of all instances, once per device.
cudaError_t prepare() {
    static PerDevice cache;
    int dev = 0, ok = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cache.get(dev, &ok, [](int* out) {
        *out = 1;
        cudaError_t r = attributes<float, 64>();
        if (r == cudaSuccess) r = attributes<float, 128>();
        if (r == cudaSuccess) r = attributes<__nv_bfloat16, 64>();
        if (r == cudaSuccess) r = attributes<__nv_bfloat16, 128>();
        return r;
    });
}

// Blocks of 32 queries where those of 64 leave SMs without one: each then takes less time,
// if not half.  Measured in fp32, 64 -> 32 queries, forward | backward: 777 tokens, 6 / 2
// heads of 80 (about 90 blocks of 64) 49 -> 36 us | 95 -> 70; 1024 tokens, 8 heads of 128 (136)
// 121 -> 84 | 295 -> 230; 12 heads of 64 (204) 68 -> 70 | 184 -> 184; 2048 tokens, 16 heads
// of 64 (528) 231 -> 299 | 703 -> 789.
bool half_blocks(const AttnArgs& a) { return (a.tokens / T + 1) * a.heads < 152; }

template <typename E, int DP, int R>
cudaError_t forward(AttnArgs a, cudaStream_t s) {
    a.slots = static_cast<int32_t>(attn_slots(a.tokens, a.sequences, 16 * R));
    const unsigned grid = static_cast<unsigned>(a.slots) * a.heads + a.fill;
    forward_kernel<E, DP, R><<<grid, kThreads, kForwardBytes<DP, R>, s>>>(a);
    return cudaGetLastError();
}

template <typename E, int DP>
cudaError_t forward(const AttnArgs& a, cudaStream_t s) {
    return half_blocks(a) ? forward<E, DP, 2>(a, s) : forward<E, DP, 4>(a, s);
}

template <typename E, int DP, int R>
cudaError_t backward(AttnArgs a, cudaStream_t s) {
    a.slots = static_cast<int32_t>(attn_slots(a.tokens, a.sequences, T));
    a.query_slots = static_cast<int32_t>(attn_slots(a.tokens, a.sequences, 16 * R));
    const unsigned keys = static_cast<unsigned>(a.slots) * a.kv_heads * a.parts + a.fill;
    const unsigned queries = static_cast<unsigned>(a.query_slots) * a.heads + a.fill;
    const auto run = [&](unsigned k, unsigned q) {
        backward_kernel<E, DP, R><<<k + q, kThreads, kBackwardBytes<DP>, s>>>(a, k);
        return cudaGetLastError();
    };
    if (sizeof(E) == 4) return run(keys, queries);
    const cudaError_t e = run(0, queries);  // makes the delta that the other reads
    return e == cudaSuccess ? run(keys, 0) : e;
}

template <typename E, int DP>
cudaError_t backward(const AttnArgs& a, cudaStream_t s) {
    return half_blocks(a) ? backward<E, DP, 2>(a, s) : backward<E, DP, 4>(a, s);
}

}  // namespace

cudaError_t attn_simt_forward(const AttnArgs& a, bool f32, cudaStream_t s) {
    const cudaError_t e = prepare();
    if (e != cudaSuccess) return e;
    if (f32) return a.dim <= 64 ? forward<float, 64>(a, s) : forward<float, 128>(a, s);
    return a.dim <= 64 ? forward<__nv_bfloat16, 64>(a, s) : forward<__nv_bfloat16, 128>(a, s);
}

cudaError_t attn_simt_backward(const AttnArgs& a, bool f32, cudaStream_t s) {
    const cudaError_t e = prepare();
    if (e != cudaSuccess) return e;
    if (f32) return a.dim <= 64 ? backward<float, 64>(a, s) : backward<float, 128>(a, s);
    return a.dim <= 64 ? backward<__nv_bfloat16, 64>(a, s) : backward<__nv_bfloat16, 128>(a, s);
}

cudaError_t attn_join(const AttnArgs& a, bool f32, cudaStream_t s) {
    const int64_t n = a.tokens * a.kv_heads * a.dim;
    const int each = a.dim % 4 == 0 ? 4 : 1;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((n / each + 255) / 256, 1216)), 2);
    if (each == 4)
        return launch_dependent(f32 ? join_kernel<float, 4> : join_kernel<__nv_bfloat16, 4>, grid, 256, s, a);
    return launch_dependent(f32 ? join_kernel<float, 1> : join_kernel<__nv_bfloat16, 1>, grid, 256, s, a);
}

cudaError_t attn_pack(const AttnArgs& a, const AttnArgs& b, cudaStream_t s) {
    const int64_t most = a.tokens * a.heads * (b.dim / 8);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((most + 255) / 256, 2432)), a.d_o.p ? 4 : 3);
    pack_kernel<<<grid, 256, 0, s>>>(a, b);
    return cudaGetLastError();
}

cudaError_t attn_delta(const AttnArgs& a, bool f32, cudaStream_t s) {
    return f32 ? run_delta<float>(a, s) : run_delta<__nv_bfloat16>(a, s);
}

}  // namespace dmuon
