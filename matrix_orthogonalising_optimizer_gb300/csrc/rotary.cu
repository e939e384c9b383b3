// Norm of each head's queries and keys with the position rotation in the same
// pass, forward and backward, and the table of the rotation's angles.
//
//   r = 1 / sqrt(mean(x^2) + eps), n = x r w            (or n = x: no norm)
//   y: the first `rotary` elements of n in pairs (a, b), turned by the angle of the
//      token's position: a cos - b sin, a sin + b cos; the others unchanged
//   dn = dy turned back, dw = sum dn x r, g = dn w, dx = r (g - x r mean(g x r))
//
// HBM-bound: a row is read once, held in registers as fp32 and written once.  Measured: 16384
// tokens, 32/8 heads of 128: forward 58 us (6.0 TB/s, 89 % of the copy rate), backward 84 us
// with the weights' gradients (6.1 TB/s); fp32 158 us (4.3 TB/s) and 264 us (3.8 TB/s), each call
// from a cold cache (bf16 so: 64 and 94 us).
//
// Vector kernels (rows on 16 bytes, dim and rotary multiples of 16): a lane holds 16
// elements of a row, and both elements of each of their pairs -- columns 8 t .. and
// rotary / 2 + 8 t .., or 16 t .. interleaved --, so the rotation needs no exchange.
// A warp goes over the heads of one token, 32 / (dim / 16) rows at a time, with the
// position's cos and sin in registers; a few tokens are shared out among more warps.
// The rows come through shared memory by cp.async, so that the bytes in flight do not
// cost registers.  The weights' gradients stay in the lanes'
// registers over all of a warp's rows; the block adds them up in a fixed order, and a
// second kernel the blocks' sums.
//
// Other rows: one warp per row, which goes through shared memory once so that any
// pairing can be formed.  A warp's rows follow one another, so that a token's cos and sin
// serve its heads and the next row is fetched ahead.  Measured, bf16, 16384 tokens, 32/8 heads of
// 120: forward 133 us (2.4 TB/s), backward 197 us; 764 and 830 us with rows dealt out one by
// one.  Bound: instructions, element by element.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "checks.h"
#include "tc.cuh"

namespace dmuon {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxDim = 256;
constexpr int kWarps = 8;
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int kMaxHeads = 1024;
constexpr int kVectorBlocks = 304;  // two per SM; backward: rows of partial sums
constexpr int kRowBlocks = 608;     // four per SM, of the kernel for any rows (a row in flight per warp)

struct Rows {
    const void* x;
    const void* dy;
    const void* w;
    void* out;
    int64_t x_token, x_head, dy_token, dy_head;
    int32_t heads;
    int32_t first, blocks;     // the blocks that work on them
    int32_t split, per;        // vector kernels: warps that share a token's heads, steps of each
};

struct RotArgs {
    Rows r[2];                 // queries, keys
    const int64_t* positions;
    const float* table;        // [positions][rotary]: cos, then sin; NULL: no rotation
    int64_t tokens, table_rows;
    int32_t dim, rotary, interleaved, norm;
    float eps;
    float* partial;            // backward: [blocks][dim], NULL: no weight gradients
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

// kPer: elements of a lane, 32 kPer >= dim.
template <typename E, bool kBack, int kPer>
__global__ void __launch_bounds__(32 * kWarps, kPer <= 4 ? 4 : 2) rows_kernel(const __grid_constant__ RotArgs a) {
    __shared__ float rows[kWarps][32 * kPer];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float* s = rows[warp];
    const Rows& R = a.r[blockIdx.x < static_cast<unsigned>(a.r[1].first) ? 0 : 1];
    // of this lane's elements: the place of the other one of the pair, of the pair's cos in a
    // row of the table (negative: not turned), the sign of its sine, the weight
    const int half = a.rotary / 2;
    int other[kPer], at[kPer];
    float sign[kPer], w[kPer], dw[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        const bool second = a.interleaved ? (e & 1) != 0 : e >= half;
        other[i] = a.interleaved ? e ^ 1 : second ? e - half : e + half;
        at[i] = e >= a.rotary ? -1 : a.interleaved ? e / 2 : second ? e - half : e;
        sign[i] = second != kBack ? 1.0f : -1.0f;
        w[i] = R.w && e < a.dim ? to_f<E>(static_cast<const E*>(R.w)[e]) : 1.0f;
        dw[i] = 0.0f;
    }
    const float inv = 1.0f / static_cast<float>(a.dim);
    // a warp's rows follow one another: a token's cos and sin serve all its heads, and the next
    // row is on its way while one is worked on
    const int64_t n = a.tokens * R.heads, unit = static_cast<int64_t>(blockIdx.x - R.first) * kWarps + warp;
    const int64_t units = static_cast<int64_t>(R.blocks) * kWarps, end = n * (unit + 1) / units;
    int64_t row = n * unit / units, token = row / R.heads;
    int head = static_cast<int>(row - token * R.heads);
    E xn[kPer], gn[kPer];
    const auto fetch = [&](int64_t token, int64_t head) {
        const E* px = static_cast<const E*>(R.x) + token * R.x_token + head * R.x_head;
        const E* pd = static_cast<const E*>(R.dy) + token * R.dy_token + head * R.dy_head;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            xn[i] = (!kBack || a.norm) && e < a.dim ? px[e] : E(0.0f);
            if constexpr (kBack) gn[i] = e < a.dim ? pd[e] : E(0.0f);
        }
    };
    if (row < end) fetch(token, head);
    bool fresh = true;
    float c[kPer], sn[kPer];
    for (; row < end; ++row) {
        E* out = static_cast<E*>(R.out) + row * a.dim;
        float x[kPer], g[kPer], r = 1.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            x[i] = to_f<E>(xn[i]);
            if constexpr (kBack) g[i] = to_f<E>(gn[i]);
        }
        if (fresh) {
            const int64_t position = a.table ? a.positions[token] : 0;
            const bool inside = position >= 0 && position < a.table_rows;
            const float* cs = a.table + (inside ? position : 0) * a.rotary;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                c[i] = 1.0f;
                sn[i] = 0.0f;
                if (at[i] >= 0) {
                    c[i] = inside ? cs[at[i]] : __int_as_float(0x7fffffff);
                    sn[i] = sign[i] * cs[half + at[i]];
                }
            }
        }
        fresh = ++head == R.heads;
        if (fresh) {
            head = 0;
            ++token;
        }
        if (row + 1 < end) fetch(token, head);
        if (a.norm) {
            float q = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) q = fmaf(x[i], x[i], q);
            r = rsqrtf(fmaf(warp_sum(q), inv, a.eps));
        }
        // y = n c + (the other one) sin
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if constexpr (!kBack) g[i] = a.norm ? x[i] * (r * w[i]) : x[i];
            s[lane + 32 * i] = g[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (at[i] >= 0) g[i] = fmaf(g[i], c[i], s[other[i]] * sn[i]);
        if (kBack && a.norm) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                x[i] *= r;
                dw[i] = fmaf(g[i], x[i], dw[i]);
                g[i] *= w[i];
                dot = fmaf(g[i], x[i], dot);
            }
            dot = warp_sum(dot) * inv;
#pragma unroll
            for (int i = 0; i < kPer; ++i) g[i] = r * (g[i] - x[i] * dot);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < a.dim) out[lane + 32 * i] = from_f<E>(g[i]);
        __syncwarp();
    }
    if constexpr (kBack) {
        if (!a.partial) return;
        // the block's sums, warp after warp
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) s[lane + 32 * i] = dw[i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.dim; e += 32 * kWarps) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) sum += rows[k][e];
            a.partial[static_cast<int64_t>(blockIdx.x) * a.dim + e] = sum;
        }
    }
}

// ---------------------------------------------------------------- vector kernels

// Eight elements that a lane holds as one or two 16-byte words, 32 lanes apart.
template <typename E>
__device__ __forceinline__ void unpack8(const uint4* d, int step, float (&v)[8]) {
    if constexpr (sizeof(E) == 2) {
        const uint4 w = *d;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = tc::unpack_bf16x2(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 w = d[i * step];
            v[4 * i] = __uint_as_float(w.x);
            v[4 * i + 1] = __uint_as_float(w.y);
            v[4 * i + 2] = __uint_as_float(w.z);
            v[4 * i + 3] = __uint_as_float(w.w);
        }
    }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, const float (&v)[8]) {
    if constexpr (sizeof(E) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(tc::pack_bf16x2(v[0], v[1]), tc::pack_bf16x2(v[2], v[3]),
                                                  tc::pack_bf16x2(v[4], v[5]), tc::pack_bf16x2(v[6], v[7]));
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::saddr(dst)), "l"(src) : "memory");
}

// Eight elements into the words of unpack8.
template <typename E>
__device__ __forceinline__ void copy8(uint4* dst, const E* src) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(E)) / 2; ++i) copy16(dst + 32 * i, src + 16 / sizeof(E) * i);
}

// Elements i and i + 1, for packed arithmetic.
__device__ __forceinline__ float2 pair(const float (&v)[8], int i) { return make_float2(v[i], v[i + 1]); }
__device__ __forceinline__ void set(float (&v)[8], int i, float2 x) {
    v[i] = x.x;
    v[i + 1] = x.y;
}
__device__ __forceinline__ float2 negated(float2 x) { return make_float2(-x.x, -x.y); }

// Two stored vectors as the elements a and b of eight pairs, and back.
template <bool kInter>
__device__ __forceinline__ void to_pairs(const float (&v0)[8], const float (&v1)[8], float (&a)[8], float (&b)[8]) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        a[p] = !kInter ? v0[p] : p < 4 ? v0[2 * (p % 4)] : v1[2 * (p % 4)];
        b[p] = !kInter ? v1[p] : p < 4 ? v0[2 * (p % 4) + 1] : v1[2 * (p % 4) + 1];
    }
}

template <bool kInter>
__device__ __forceinline__ void from_pairs(const float (&a)[8], const float (&b)[8], float (&v0)[8], float (&v1)[8]) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        v0[p] = !kInter ? a[p] : p % 2 ? b[p / 2] : a[p / 2];
        v1[p] = !kInter ? b[p] : p % 2 ? b[4 + p / 2] : a[4 + p / 2];
    }
}

// Stages of a warp's ring (8 KB of rows), and its shared memory.
template <typename E, bool kBack>
constexpr int kStages = (sizeof(E) == 2 ? 8 : 4) / (kBack ? 2 : 1);

template <typename E, int G, bool kBack>
struct WarpRing {
    static constexpr int kWords = static_cast<int>(sizeof(E)) * (kBack ? 2 : 1);  // 16-byte words of a lane and stage
    uint4 x[kStages<E, kBack>][kWords][32];
    float4 cs[kStages<E, kBack>][4][G];  // per token: cos of pairs 8 t .., their sines
    int64_t pos[kStages<E, kBack>];
};

// G: lanes of a row, a power of two with 16 G >= dim.  Steps of a warp: 32 / G heads of
// a token; the rows come through the lanes' own slots of a ring by cp.async, a whole
// ring ahead, and cos and sin with a token's first step.
template <typename E, int G, bool kBack, bool kInter>
__global__ void __launch_bounds__(32 * kWarps, 2) vector_kernel(const __grid_constant__ RotArgs a) {
    constexpr int R = 32 / G, S = kStages<E, kBack>, H = static_cast<int>(sizeof(E)) / 2;  // H words per eight elements
    extern __shared__ __align__(16) uint8_t raw[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, t = lane % G;
    WarpRing<E, G, kBack>& ring = reinterpret_cast<WarpRing<E, G, kBack>*>(raw)[warp];
    const bool in = 16 * t < a.dim;  // this lane holds elements
    const int half = a.rotary / 2;
    const bool turns = 8 * t < half;
    const int c0 = kInter ? 16 * t : turns ? 8 * t : a.rotary + 16 * (t - half / 8);
    const int c1 = kInter ? c0 + 8 : turns ? half + 8 * t : c0 + 8;
    const float inv = 1.0f / static_cast<float>(a.dim);
    const Rows& Q = a.r[blockIdx.x < static_cast<unsigned>(a.r[1].first) ? 0 : 1];
    const int heads = Q.heads, split = Q.split, per = Q.per;
    float wa[8], wb[8], dwa[8], dwb[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        wa[p] = wb[p] = 1.0f;
        dwa[p] = dwb[p] = 0.0f;
    }
    if (Q.w && in) {
        float v0[8], v1[8];
        unpack8<E>(reinterpret_cast<const uint4*>(static_cast<const E*>(Q.w) + c0), 1, v0);
        unpack8<E>(reinterpret_cast<const uint4*>(static_cast<const E*>(Q.w) + c1), 1, v1);
        to_pairs<kInter>(v0, v1, wa, wb);
    }
    // item = token * split + share; a warp's items are `stride` apart
    const int stride = Q.blocks * kWarps, first = static_cast<int>(blockIdx.x - Q.first) * kWarps + warp;
    const int step_token = stride / split, step_share = stride - step_token * split;
    const auto advance = [&](int& token, int& share) {
        token += step_token;
        share += step_share;
        if (share >= split) {
            share -= split;
            ++token;
        }
    };
    const int tokens = static_cast<int>(a.tokens);

    // the loads' place: item, step of it, ring slots
    int ld_token = first / split, ld_share = first - ld_token * split, ld_k = 0, ld_slot = 0, ld_tok = 0;
    // a position is fetched one item ahead of the copy of its cos and sin
    int64_t next = half > 0 && ld_token < tokens ? a.positions[ld_token] : 0;
    const auto issue = [&] {
        if (ld_token < tokens) {
            const int64_t token = ld_token;
            const int h = (ld_share + ld_k * split) * R + lane / G;
            if (in && h < heads) {
                uint4* d = &ring.x[ld_slot][0][lane];
                if (!kBack || a.norm) {
                    const E* p = static_cast<const E*>(Q.x) + token * Q.x_token + h * Q.x_head;
                    copy8(d, p + c0);
                    copy8(d + 32 * H, p + c1);
                }
                if constexpr (kBack) {
                    const E* p = static_cast<const E*>(Q.dy) + token * Q.dy_token + h * Q.dy_head;
                    copy8(d + 64 * H, p + c0);
                    copy8(d + 96 * H, p + c1);
                }
            }
            if (ld_k == 0 && half > 0) {
                if (lane < G && turns) {
                    const bool inside = next >= 0 && next < a.table_rows;
                    const float* p = a.table + (inside ? next : 0) * a.rotary + 8 * t;
                    copy16(&ring.cs[ld_tok][0][t], p);
                    copy16(&ring.cs[ld_tok][1][t], p + 4);
                    copy16(&ring.cs[ld_tok][2][t], p + half);
                    copy16(&ring.cs[ld_tok][3][t], p + half + 4);
                    if (lane == 0) ring.pos[ld_tok] = next;
                }
            }
            if (++ld_k == per) {
                ld_k = 0;
                advance(ld_token, ld_share);
                if (half > 0 && ld_token < tokens) next = a.positions[ld_token];
                if (++ld_tok == S) ld_tok = 0;
            }
            if (++ld_slot == S) ld_slot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i + 1 < S; ++i) issue();

    float cs[8], sn[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        cs[p] = 1.0f;
        sn[p] = 0.0f;
    }
    int token = first / split, share = first - token * split;
    int k = 0, slot = 0, tok = 0;
    while (token < tokens) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();
        if (k == 0 && turns) {
            const int64_t pos = ring.pos[tok];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 c = ring.cs[tok][i][t], s = ring.cs[tok][2 + i][t];
                cs[4 * i] = c.x, cs[4 * i + 1] = c.y, cs[4 * i + 2] = c.z, cs[4 * i + 3] = c.w;
                sn[4 * i] = s.x, sn[4 * i + 1] = s.y, sn[4 * i + 2] = s.z, sn[4 * i + 3] = s.w;
            }
            if (pos < 0 || pos >= a.table_rows) {
#pragma unroll
                for (int p = 0; p < 8; ++p) cs[p] = sn[p] = __int_as_float(0x7fffffff);
            }
        }
        issue();
        const int h = (share + k * split) * R + lane / G;
        const bool active = in && h < heads;
        const uint4* d = &ring.x[slot][0][lane];
        float v0[8], v1[8], p[8], q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v0[i] = v1[i] = 0.0f;
        if (active && (!kBack || a.norm)) {
            unpack8<E>(d, 32, v0);
            unpack8<E>(d + 32 * H, 32, v1);
        }
        to_pairs<kInter>(v0, v1, p, q);
        float r = 1.0f;
        if (a.norm) {
            float2 s2 = tc::both(0.0f);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                s2 = tc::fma2(pair(p, i), pair(p, i), s2);
                s2 = tc::fma2(pair(q, i), pair(q, i), s2);
            }
            float s = s2.x + s2.y;
#pragma unroll
            for (int x = G / 2; x >= 1; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
            r = rsqrtf(fmaf(s, inv, a.eps));
        }
        const float2 r2 = tc::both(r);
        if constexpr (!kBack) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float2 m = pair(p, i), n = pair(q, i);
                if (a.norm) {
                    m = tc::mul2(m, tc::mul2(r2, pair(wa, i)));
                    n = tc::mul2(n, tc::mul2(r2, pair(wb, i)));
                }
                set(p, i, tc::fma2(m, pair(cs, i), negated(tc::mul2(n, pair(sn, i)))));
                set(q, i, tc::fma2(m, pair(sn, i), tc::mul2(n, pair(cs, i))));
            }
            from_pairs<kInter>(p, q, v0, v1);
        } else {
            float g[8], u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v0[i] = v1[i] = 0.0f;
            if (active) {
                unpack8<E>(d + 64 * H, 32, v0);
                unpack8<E>(d + 96 * H, 32, v1);
            }
            to_pairs<kInter>(v0, v1, g, u);
            float2 dot2 = tc::both(0.0f);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float2 m = tc::fma2(pair(g, i), pair(cs, i), tc::mul2(pair(u, i), pair(sn, i)));
                float2 n = tc::fma2(pair(u, i), pair(cs, i), negated(tc::mul2(pair(g, i), pair(sn, i))));
                if (a.norm) {
                    const float2 x = tc::mul2(pair(p, i), r2), y = tc::mul2(pair(q, i), r2);
                    set(p, i, x);
                    set(q, i, y);
                    if (active) {
                        set(dwa, i, tc::fma2(m, x, pair(dwa, i)));
                        set(dwb, i, tc::fma2(n, y, pair(dwb, i)));
                    }
                    m = tc::mul2(m, pair(wa, i));
                    n = tc::mul2(n, pair(wb, i));
                    dot2 = tc::fma2(m, x, tc::fma2(n, y, dot2));
                }
                set(g, i, m);
                set(u, i, n);
            }
            if (a.norm) {
                float dot = dot2.x + dot2.y;
#pragma unroll
                for (int x = G / 2; x >= 1; x >>= 1) dot += __shfl_xor_sync(kFull, dot, x);
                const float2 off = tc::both(-dot * inv);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    set(g, i, tc::mul2(r2, tc::fma2(pair(p, i), off, pair(g, i))));
                    set(u, i, tc::mul2(r2, tc::fma2(pair(q, i), off, pair(u, i))));
                }
            }
            from_pairs<kInter>(g, u, v0, v1);
        }
        if (active) {
            E* out = static_cast<E*>(Q.out) + (static_cast<int64_t>(token) * heads + h) * a.dim;
            store8(out + c0, v0);
            store8(out + c1, v1);
        }
        if (++k == per) {
            k = 0;
            advance(token, share);
            if (++tok == S) tok = 0;
        }
        if (++slot == S) slot = 0;
    }
    if constexpr (kBack) {
        if (!a.partial) return;
        // the warp's row groups, then the block's warps
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        float(*sums)[16 * G] = reinterpret_cast<float(*)[16 * G]>(raw);
#pragma unroll
        for (int s = G; s < 32; s <<= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dwa[i] += __shfl_xor_sync(kFull, dwa[i], s);
                dwb[i] += __shfl_xor_sync(kFull, dwb[i], s);
            }
        if (in && lane < G) {
            float v0[8], v1[8];
            from_pairs<kInter>(dwa, dwb, v0, v1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[warp][c0 + i] = v0[i];
                sums[warp][c1 + i] = v1[i];
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.dim; e += 32 * kWarps) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += sums[w][e];
            a.partial[static_cast<int64_t>(blockIdx.x) * a.dim + e] = sum;
        }
    }
}

// Whether the vector kernels can take the call.
bool vectors(const RotArgs& a, int es, bool back) {
    const int64_t n = 16 / es;
    bool ok = a.dim % 16 == 0 && a.rotary % 16 == 0;
    for (const Rows& r : a.r) {
        if (!back || a.norm)
            ok = ok && reinterpret_cast<uintptr_t>(r.x) % 16 == 0 && r.x_token % n == 0 && r.x_head % n == 0;
        if (back) ok = ok && reinterpret_cast<uintptr_t>(r.dy) % 16 == 0 && r.dy_token % n == 0 && r.dy_head % n == 0;
    }
    return ok;
}

// The blocks of the queries and, behind them, of the keys: in proportion to their
// rows, no more than they can use, at least one each.
int set_blocks(Rows (&r)[2], int64_t tokens, int most) {
    const int64_t all = r[0].heads + r[1].heads;
    for (int i = 0; i < 2; ++i)
        r[i].blocks = static_cast<int32_t>(std::max<int64_t>(
            1, std::min<int64_t>(ceil_div(tokens * r[i].heads, kWarps), (most - 1) * r[i].heads / all)));
    r[0].first = 0;
    r[1].first = r[0].blocks;
    return r[0].blocks + r[1].blocks;
}

template <typename E, int G, bool kBack>
cudaError_t run_vector(RotArgs a, int blocks, cudaStream_t s) {
    constexpr int R = 32 / G;
    // a token's heads are shared among warps until each has 16 items or more, so that
    // their unequal counts cost a few percent at most
    for (Rows& r : a.r) {
        const int64_t chunks = ceil_div(r.heads, R);
        r.split = static_cast<int32_t>(std::min<int64_t>(chunks, ceil_div(16 * r.blocks * kWarps, a.tokens)));
        r.per = static_cast<int32_t>(ceil_div(chunks, r.split));
    }
    const auto kernel = a.interleaved ? vector_kernel<E, G, kBack, true> : vector_kernel<E, G, kBack, false>;
    constexpr int bytes = kWarps * static_cast<int>(sizeof(WarpRing<E, G, kBack>));
    static PerDevice cache[2];  // the shared-memory attribute, once per device
    int dev = 0, ok = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cache[a.interleaved].get(dev, &ok, [&](int* out) {
            *out = 1;
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename E, bool kBack>
cudaError_t run_rows(RotArgs& a, cudaStream_t s) {
    const bool vector = vectors(a, sizeof(E), kBack);
    const int blocks = set_blocks(a.r, a.tokens, vector ? kVectorBlocks : kRowBlocks);
    if (vector) {
        if (a.dim <= 16) return run_vector<E, 1, kBack>(a, blocks, s);
        if (a.dim <= 32) return run_vector<E, 2, kBack>(a, blocks, s);
        if (a.dim <= 64) return run_vector<E, 4, kBack>(a, blocks, s);
        if (a.dim <= 128) return run_vector<E, 8, kBack>(a, blocks, s);
        return run_vector<E, 16, kBack>(a, blocks, s);
    }
    const auto kernel = a.dim <= 64    ? rows_kernel<E, kBack, 2>
                        : a.dim <= 128 ? rows_kernel<E, kBack, 4>
                                       : rows_kernel<E, kBack, 8>;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), 32 * kWarps, s, a);
}

// Weight gradients from the partial sums [blocks][dim], always in the same order: 32
// columns per block, 32 threads each; blockIdx.y: queries, keys.
template <typename E>
__global__ void __launch_bounds__(1024) reduce_kernel(const float* partial, int nq, int nk, int dim, void* dq,
                                                      void* dk) {
    __shared__ float sums[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool keys = blockIdx.y != 0;
    const int col = blockIdx.x * 32 + threadIdx.x % 32, group = threadIdx.x / 32, n = keys ? nk : nq;
    if (keys) partial += static_cast<int64_t>(nq) * dim;
    float sum = 0.0f;
    if (col < dim)
        for (int i = group; i < n; i += 32) sum += partial[static_cast<int64_t>(i) * dim + col];
    sums[group][threadIdx.x % 32] = sum;
    __syncthreads();
    void* out = keys ? dk : dq;
    if (group != 0 || col >= dim || !out) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sums[i][threadIdx.x];
    static_cast<E*>(out)[col] = from_f<E>(sum);
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
    return static_cast<size_t>(kRowBlocks) * dim * sizeof(float);
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
    const bool f32 = dtype == DMUON_FP32;
    OPS_CUDA((f32 ? run_rows<float, false>(a, s) : run_rows<__nv_bfloat16, false>(a, s)));
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
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    if (tokens > 0) OPS_CUDA((f32 ? run_rows<float, true>(a, s) : run_rows<__nv_bfloat16, true>(a, s)));
    if (sums) {
        const dim3 grid(static_cast<unsigned>(ceil_div(dim, 32)), 2);
        OPS_CUDA(launch_dependent(f32 ? reduce_kernel<float> : reduce_kernel<__nv_bfloat16>, grid, 1024, s, a.partial,
                                  a.r[0].blocks, a.r[1].blocks, dim, dq_weight, dk_weight));
    }
    return DMUON_OK;
}
