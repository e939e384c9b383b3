// Attention: the arguments its kernels share, and how a block finds its rows in
// a packed batch.  Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace dmuon {

// One tensor of tokens x heads x dim: strides in elements, a head's row contiguous.
struct AttnHeads {
    const void* p;
    int64_t token, head;
};

struct AttnArgs {
    AttnHeads q, k, v, d_o;    // queries, keys, values, gradient of the outputs
    const void* o;             // tokens x heads x dim, contiguous like the outputs
    void* out;                 // forward: o | backward: dq
    void* dk;
    void* dv;
    float* lse;                // [heads][tokens]
    float* delta;              // [heads][tokens]: do . o
    const int64_t* offsets;    // sequences + 1, or NULL: equal sequences of `length` tokens
    int64_t tokens, length;
    int32_t sequences;
    int32_t heads, kv_heads, group, dim;
    int32_t causal;
    int32_t slots;             // row tiles of a head (an upper bound: see attn_slots)
    int32_t query_slots;       // FFMA backward: the same of the queries' blocks
    int32_t fill;              // blocks behind all heads' that clear the rows of no sequence
    int32_t whole;             // backward, tensor cores: sequences, where those of one tile have their own launch
    int32_t parts;             // backward: blocks that share the queries of a key tile
    float* partial;            // parts > 1: [2][parts][tokens][kv_heads][dim] sums of dk (unscaled) and dv
    float scale, scale_log2;   // scale_log2 = scale * log2(e)
};

// A tile of `T` rows of one sequence.  Which tiles exist is only known on the
// device, so the grid has room for every split of the tokens into n sequences:
// sequence s, which begins at token b, owns the slots from b / T + s on.  Up to the
// next sequence's first slot that is at least one slot per T rows or part of T rows;
// the slots that are too many find nothing and return.
__host__ __device__ inline int64_t attn_slots(int64_t tokens, int64_t sequences, int tile) {
    return tokens / tile + sequences;
}

struct AttnTile {
    int64_t begin;  // the sequence's first token
    int32_t len;    // its tokens
    int32_t tile;   // index of the tile in the sequence
};

__device__ __forceinline__ int64_t attn_offset(const AttnArgs& a, int64_t s) {
    if (!a.offsets) return s * a.length;
    const int64_t o = a.offsets[s];
    return o < 0 ? 0 : o > a.tokens ? a.tokens : o;  // no access outside, whatever the offsets say
}

// The tile at a slot, by all 32 lanes of a warp (each round splits the sequences
// left into 32; up to 31 sequences take one round of loads).  False: the slot holds none.
__device__ __forceinline__ bool attn_find(const AttnArgs& a, int32_t slot, int T, AttnTile& t) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0, count = a.sequences, b = 0, e = 0;  // tokens < 2^31
    do {
        const int32_t step = (count + 31) / 32, i = lo + lane * step;
        const bool there = lane * step <= count;  // also the end of the last one
        const int32_t o = there ? static_cast<int32_t>(attn_offset(a, i < a.sequences ? i : a.sequences)) : 0;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < count && o / T + i <= slot);
        const int c = m == 0 ? 0 : 31 - __clz(m);
        b = __shfl_sync(0xffffffffu, o, c);
        e = __shfl_sync(0xffffffffu, o, c + 1 < 32 ? c + 1 : c);
        const int32_t end = lo + count;
        lo += c * step;
        if (step == 1 && c == 31) e = static_cast<int32_t>(attn_offset(a, lo + 1));
        count = step < end - lo ? step : end - lo;
        if (step == 1) count = 0;
    } while (count > 0);
    const int32_t k = slot - (b / T + lo);
    // from one lane: the compiler then knows them to be the same in all, and keeps what
    // follows from them in uniform registers, where MMAs and copies take their operands
    t.begin = __shfl_sync(0xffffffffu, b, 0);
    t.len = __shfl_sync(0xffffffffu, e - b, 0);
    t.tile = __shfl_sync(0xffffffffu, k, 0);
    return __shfl_sync(0xffffffffu, k >= 0 && b + static_cast<int64_t>(k) * T < e ? 1 : 0, 0) != 0;
}

// Clears elements [from, to) of x: share f of a.fill, 16 bytes a store.
template <typename T>
__device__ __forceinline__ void attn_zero(const AttnArgs& a, T* x, int64_t from, int64_t to, int f, int thread,
                                          int threads) {
    constexpr int N = 16 / sizeof(T);
    const int64_t off = reinterpret_cast<uintptr_t>(x) / sizeof(T) % N;  // from here on, in whole words
    x -= off;
    from += off;
    to += off;
    const int64_t lo = (from + N - 1) / N, hi = to / N;
    for (int64_t i = lo + f * threads + thread; i < hi; i += a.fill * threads)
        reinterpret_cast<uint4*>(x)[i] = make_uint4(0, 0, 0, 0);
    if (f != 0) return;
    const int64_t head = lo * N < to ? lo * N : to, tail = hi * N > head ? hi * N : head;
    for (int64_t i = from + thread; i < head; i += threads) x[i] = T(0.0f);
    for (int64_t i = tail + thread; i < to; i += threads) x[i] = T(0.0f);
}

// Clears the rows of no sequence -- before the first and behind the last -- of a tensor
// tokens x heads x dim, and (lse given) sets their lse to -inf: share f of a.fill.
// (Row by row and head by head, 4096 of 8192 tokens, 32 heads of 128, took 166 us.)
template <typename T>
__device__ __forceinline__ void attn_clear(const AttnArgs& a, T* x, float* lse, int heads, int f, int thread,
                                           int threads) {
    const int64_t first = attn_offset(a, 0), end = attn_offset(a, a.sequences), last = end > first ? end : first;
    const int64_t width = static_cast<int64_t>(heads) * a.dim;
    attn_zero(a, x, 0, first * width, f, thread, threads);
    attn_zero(a, x, last * width, a.tokens * width, f, thread, threads);
    if (!lse) return;
    const int64_t outside = first + a.tokens - last;
    for (int h = 0; h < heads; ++h)
        for (int64_t i = f * threads + thread; i < outside; i += a.fill * threads)
            lse[h * a.tokens + (i < first ? i : i - first + last)] = __int_as_float(0xff800000);
}

// Tensor-core kernels: bf16, rows of 16-byte stride in the maps (the outputs' rows may have
// any length).
struct AttnMaps {
    CUtensorMap q, k, v, d_o;  // dim x heads x tokens, boxes of 64 x 1 x 128
};
cudaError_t attn_tc_forward(const AttnArgs& a, const AttnMaps& m, cudaStream_t s);
bool attn_tc_needs_delta(const AttnArgs& a);  // some sequence may be longer than one tile
cudaError_t attn_tc_backward(const AttnArgs& a, const AttnMaps& m, cudaStream_t s);
cudaError_t attn_fwd_status_word(void** p);  // the kernels' time-out flags on the current device
cudaError_t attn_bwd_status_word(void** p);

// The range of a key tile's steps (query tiles of all its heads) that part p takes.
__host__ __device__ inline int attn_part(int steps, int p, int parts) {
    return static_cast<int>(static_cast<int64_t>(steps) * p / parts);
}

__device__ __forceinline__ float* attn_partial(const AttnArgs& a, int which, int part) {
    return a.partial + (static_cast<int64_t>(which) * a.parts + part) * a.tokens * a.kv_heads * a.dim;
}

// FFMA kernels (attn_simt.cu): any strides, either type.
cudaError_t attn_simt_forward(const AttnArgs& a, bool f32, cudaStream_t s);
cudaError_t attn_simt_backward(const AttnArgs& a, bool f32, cudaStream_t s);
// dk and dv from their partial sums, in the order of the parts
cudaError_t attn_join(const AttnArgs& a, bool f32, cudaStream_t s);
// the rows of a.q, a.k, a.v, a.d_o (bf16) to those of b, contiguous, zeros behind a.dim
cudaError_t attn_pack(const AttnArgs& a, const AttnArgs& b, cudaStream_t s);
// delta, for both backward passes
cudaError_t attn_delta(const AttnArgs& a, bool f32, cudaStream_t s);

}  // namespace dmuon
