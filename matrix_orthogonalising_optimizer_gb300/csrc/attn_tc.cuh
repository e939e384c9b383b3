// What the tensor-core kernels of attention share: tiles in shared memory, their
// descriptors, the products of one 128-row tile, and the end of a CTA.
//
// A tile is 128 rows of a head as TMA brings them: one or two boxes of 64 columns,
// rows of 128 bytes, 128-byte swizzle; columns behind `dim` and rows behind the tensor
// read as zero.  The same bytes serve as an operand whose contraction runs over the
// columns (K-major: s = q k^T) and over the rows (MN-major: o = p v).
#pragma once

#include "act.cuh"
#include "attn.h"
#include "tc.cuh"

namespace dmuon {
namespace attn {

using namespace tc;

constexpr int kRows = 128;
constexpr int kBox = kRows * 128;  // bytes of a box

template <int DP>
constexpr int kTile = DP / 64 * kBox;  // bytes of a tile

// M = 128; a_mn, b_mn: A's, B's contraction runs over its rows.
__device__ __forceinline__ constexpr uint32_t idesc_of(int n, bool b_mn, bool a_mn = false) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return smem_desc(addr, 0, 1024); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) { return smem_desc(addr, kBox, 1024); }

// D (128 x 128) = A B^T over the tiles' columns.
template <int DP>
__device__ __forceinline__ void product_cols(uint32_t e, uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
        const uint64_t step = static_cast<uint64_t>((k / 4 * kBox + k % 4 * 32) >> 4);
        umma_bf16(e, d, a + step, b + step, idesc_of(kRows, false), k != 0 ? 1u : 0u);
    }
}

// The same with A in TMEM.
template <int DP>
__device__ __forceinline__ void product_cols_ts(uint32_t e, uint32_t d, uint32_t a, uint64_t b) {
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
        umma_bf16_ts(e, d, a + static_cast<uint32_t>(8 * k),
                     b + static_cast<uint64_t>((k / 4 * kBox + k % 4 * 32) >> 4), idesc_of(kRows, false),
                     k != 0 ? 1u : 0u);
}

// D (128 x DP) (+)= P B over 16 n rows of B, from row 16 k0 on; P in TMEM.
template <int DP>
__device__ __forceinline__ void product_rows(uint32_t e, uint32_t d, uint32_t p, uint64_t b, int k0, int n, bool add) {
#pragma unroll
    for (int k = 0; k < n; ++k)
        umma_bf16_ts(e, d, p + static_cast<uint32_t>(8 * k), b + static_cast<uint64_t>(((k0 + k) * 2048) >> 4),
                     idesc_of(DP, true), add || k != 0 ? 1u : 0u);
}

// D (128 x DP) (+)= A B over B's 128 rows, A in shared memory: a 128 x 128 tile in two
// boxes, its columns against B's rows, or (kRowsOfA) its rows: D = A^T B.
template <int DP, bool kRowsOfA>
__device__ __forceinline__ void product_tile(uint32_t e, uint32_t d, uint64_t a, uint64_t b, bool add) {
#pragma unroll
    for (int k = 0; k < kRows / 16; ++k)
        umma_bf16(e, d, a + static_cast<uint64_t>((kRowsOfA ? k * 2048 : k / 4 * kBox + k % 4 * 32) >> 4),
                  b + static_cast<uint64_t>((k * 2048) >> 4), idesc_of(DP, true, kRowsOfA), add || k != 0 ? 1u : 0u);
}

// Loads the tile that begins at a token.
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t e, uint32_t dst, const CUtensorMap* map, uint32_t bar, int head,
                                          int token) {
#pragma unroll
    for (int b = 0; b < DP / 64; ++b) tma_load_3d(e, dst + b * kBox, map, bar, 64 * b, head, token);
}

// Until an item's copies have landed -- those of `first`, outside the ring, and the last of
// `issued` into `slots` -- by the warp that issued them, which is idle then: none is under way
// when the CTA leaves, also after a wait of any warp that gave up (these are waited for once more,
// with the same limit).
__device__ __forceinline__ void await_copies(uint64_t* first, uint64_t* full, int issued, int slots, int32_t* bad) {
    mbar_wait<false>(first, 0, bad);
#pragma unroll 1
    for (int i = max(issued - slots, 0); i < issued; ++i) mbar_wait<false>(&full[i % slots], (i / slots) & 1, bad);
    __syncwarp();
}

// Rows [first, 128) of a tile, which belong to another sequence or to none, become
// zero: their weight in a product over the rows is 0, but 0 times an infinity or NaN
// is not.  By `threads` threads; visible to the tensor cores after a barrier.
template <int DP>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int first, int thread, int threads) {
    const int pieces = (kRows - first) * 8;
    for (int b = 0; b < DP / 64; ++b)
        for (int i = thread; i < pieces; i += threads)
            *reinterpret_cast<uint4*>(tile + b * kBox + first * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// A CTA that has come to its end takes the place of a block that has not started yet
// (cluster launch control): shared memory, TMEM and barriers are set up once, and the
// order stays that of the grid.  By one warp: false if all blocks have started; `asked`
// counts the requests on `claimed` (one arrival), and none may follow one that failed.
__device__ __forceinline__ bool claim_block(uint4* claim, uint64_t* claimed, uint32_t& asked, uint32_t& block,
                                            int32_t* bad, int lane) {
    if (lane == 0) {
        mbar_expect_tx(claimed, 16);
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                saddr(claim)),
            "r"(saddr(claimed))
            : "memory");
    }
    __syncwarp();
    const bool there = __all_sync(kFullMask, mbar_wait<false>(claimed, asked & 1, bad));
    if (!there) mbar_wait<false>(claimed, asked & 1, bad);  // once more: no answer after the CTA has left
    ++asked;
    uint32_t got = 0, index = 0;
    if (there)
        asm volatile(
            "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
            "ld.shared.b128 h, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
            : "=r"(got), "=r"(index)
            : "r"(saddr(claim))
            : "memory");
    // the answer is read before the next one may come
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    block = __shfl_sync(kFullMask, index, 0);
    return __shfl_sync(kFullMask, got, 0) != 0;
}

template <int kCols>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(slot)), "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

template <int kCols>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(kCols) : "memory");
}

// A warp's 32 rows of an accumulator (64 kBoxes columns at TMEM address t, this lane's
// row) times f, as bf16, to `rows` rows of `dim` elements, `ld` apart (one by one where dim is
// no multiple of 8).  They pass through the warp's 4 KB slices of a finished tile's boxes in shared memory,
// so that an instruction stores whole 128-byte pieces: row by row from the lanes it
// touches 32 lines, and a tile took 1 us.
template <int kBoxes>
__device__ __forceinline__ void store_rows(uint8_t* stage, uint32_t t, float f, __nv_bfloat16* out, int64_t ld,
                                           int rows, int dim, int lane) {
    const int chunk = lane % 8;
#pragma unroll 1
    for (int b = 0; b < kBoxes; ++b, stage += kBox) {
        uint4* mine = reinterpret_cast<uint4*>(stage + lane * 128);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[32];
            tmem_ld32(t + 64 * b + 32 * h, v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mine[(4 * h + k) ^ chunk] =
                    make_uint4(pack_bf16x2(v[8 * k] * f, v[8 * k + 1] * f),
                               pack_bf16x2(v[8 * k + 2] * f, v[8 * k + 3] * f),
                               pack_bf16x2(v[8 * k + 4] * f, v[8 * k + 5] * f),
                               pack_bf16x2(v[8 * k + 6] * f, v[8 * k + 7] * f));
        }
        __syncwarp();
        const int c = 64 * b + 8 * chunk;
        if (dim % 8 != 0) {
#pragma unroll 1
            for (int r = 0; r < min(rows, 32); ++r)
                for (int x = lane; x < min(64, dim - 64 * b); x += 32)
                    out[r * ld + 64 * b + x] =
                        reinterpret_cast<const __nv_bfloat16*>(stage + r * 128)[((x / 8) ^ (r % 8)) * 8 + x % 8];
            __syncwarp();
            continue;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + lane / 8;
            const uint4 w = reinterpret_cast<const uint4*>(stage + r * 128)[chunk ^ (r % 8)];
            if (r < rows && c < dim) *reinterpret_cast<uint4*>(out + r * ld + c) = w;
        }
        __syncwarp();
    }
}

// The same in fp32, unscaled, 32 columns at a time.
template <int kBoxes>
__device__ __forceinline__ void store_rows_f32(uint8_t* stage, uint32_t t, float* out, int64_t ld, int rows, int dim,
                                               int lane) {
    const int chunk = lane % 8;
    float4* mine = reinterpret_cast<float4*>(stage + lane * 128);
#pragma unroll 1
    for (int b = 0; b < 2 * kBoxes; ++b) {
        float v[32];
        tmem_ld32(t + 32 * b, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mine[k ^ chunk] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        __syncwarp();
        const int c = 32 * b + 4 * chunk;
        if (dim % 8 != 0) {
#pragma unroll 1
            for (int r = 0; r < min(rows, 32); ++r)
                if (32 * b + lane < dim)
                    out[r * ld + 32 * b + lane] =
                        reinterpret_cast<const float*>(stage + r * 128)[((lane / 4) ^ (r % 8)) * 4 + lane % 4];
            __syncwarp();
            continue;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + lane / 8;
            const float4 w = reinterpret_cast<const float4*>(stage + r * 128)[chunk ^ (r % 8)];
            if (r < rows && c < dim) *reinterpret_cast<float4*>(out + r * ld + c) = w;
        }
        __syncwarp();
    }
}

}  // namespace attn
}  // namespace dmuon
