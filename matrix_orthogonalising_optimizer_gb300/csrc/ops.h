// Internal structures of the training operators (layer norm, gated
// feed-forward block, vocabulary loss): the grouped tcgen05 GEMM they share
// and its host-side builder.  Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>
#include <string>

#include "internal.h"

namespace dmuon {

void set_last_error(const std::string& msg);

// Launch of a kernel that begins with griddepcontrol.wait: it may be placed while
// the stream's previous kernel finishes (programmatic dependent launch), which
// takes 1 to 2 us off a chain of short kernels.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int kOpsMaxProblems = 4;
constexpr int kOpsMaxSegs = 12;

// An fp32 matrix enters the tensor cores as three bf16 parts, x = hi + mid +
// lo (8 + 8 + 8 significant bits), and a product of two such matrices as the
// six part products above 2^-24 of the whole, the smallest first.
constexpr int kF32Parts = 3;

enum OpsEpi : int32_t { OPS_STORE = 0, OPS_GATE = 1, OPS_DGATE = 2, OPS_LOGITS = 3, OPS_STORE_SCALED = 4 };
constexpr int kOpsKinds = 5;
enum OpsAct : int32_t { OPS_SILU = 0, OPS_GELU = 1 };

// A row-major matrix an epilogue reads or writes.
struct OpsMat {
    void* p;
    int64_t ld;      // elements
    int32_t type;    // ElemType
    int32_t vec;     // rows start on 16-byte boundaries: 16-byte accesses
    int64_t part;    // > 0: kF32Parts bf16 parts, `part` elements apart
};

// D (M x N) = sum over K segments of A-part (M x K) * B-part (K x N).  Segment s
// reads source, A part and B part from seg[s]; every segment is `slabs` 64-deep
// K slabs long (a ragged end is zero-filled by TMA).  A is K-major (stored
// M x K) or MN-major (stored K x M), B likewise (N x K or K x N).  `dual`: B is
// two matrices of N rows, source maps b[0] and b[1], and a pair tile is bn / 2
// columns of each (CTA rank r loads those of matrix r), so the lower half of the
// accumulator's columns belongs to the first and the upper half to the second.
struct OpsProblem {
    CUtensorMap a[2], b[2];
    int32_t maps_a, maps_b;     // tensor maps in use
    int32_t M, N;
    int32_t bn;                 // columns of a pair tile: 256, or 128 (not LOGITS)
    int32_t a_rows[2];          // rows of A that CTA rank 0 / 1 loads: 128, fewer if M is below one tile
    int32_t slabs, nseg;
    uint16_t seg[kOpsMaxSegs];  // source | A part << 4 | B part << 8
    int32_t a_mn, b_mn, dual;
    int32_t tiles_m, tiles_n;
    // work units: `whole` tiles of all K, then the other tiles in `split` K ranges each
    int32_t whole, split;
    int32_t unit_begin;  // first unit of this problem in the launch
    int32_t tail_begin;  // first split tile (counter index)
    int32_t slot_begin;  // first partial-sum slot
    // epilogue
    int32_t act;
    OpsMat out[4];  // STORE, STORE_SCALED: D | GATE: h, act, u act', h again | DGATE: da, du | LOGITS: exponentials
                    // (fp32, or 16-bit codes, rows padded to whole 16-column chunks)
    OpsMat in[2];   // STORE: in[0] = addend (fp32) | DGATE: u act', act
    float2* stats;            // LOGITS: [M][nblk] (max, sum of exp) of 128-column blocks
    int32_t nblk;
    float* target_logit;      // LOGITS: [M]
    const int64_t* targets;   // LOGITS: [M]
};

struct OpsLaunch {
    OpsProblem p[kOpsMaxProblems];
    int32_t n, total_units;
    int32_t chain;         // K slabs per chain of MMAs where sums are added up in registers
    int32_t* counter;      // unit counter, zero at launch
    int32_t* tail_count;   // arrivals per (split tile, CTA rank, epilogue warp), zero at launch
    float* partials;       // split tiles' partial sums
    const float* scale;    // STORE_SCALED: the sums' factor (the addend is not scaled)
};

// Product of a few rows x (tokens x K) with weight rows (N x K, twice for the
// gated block), bf16 or fp32, rows of 16-byte stride: the weights are streamed
// once through registers (ops_stream.cu).
struct OpsStream {
    const void* x;
    const void* w[2];           // [0]; GATE: gate and up
    int64_t ldx, ldw;           // elements, multiples of 16 bytes
    int32_t tokens, N, K;
    int32_t act;
    int32_t after;              // the launch directly follows the library's own kernel, which did not write w
    OpsMat out[4];              // as OpsProblem
    float2* stats;              // LOGITS: [tokens][nblk] of ops_stream_block() columns
    int32_t nblk;
    float* target_logit;
    const int64_t* targets;
};

// Most rows the streaming kernel takes: of the gated block, and of the loss in
// bf16 and fp32.  Where both sides are close the limit is one for all widths: 32
// rows of a large fp32 block lose 6 % by it and those of a small one gain 35 %, 16
// rows of a loss win 5 % or lose 2 % with the machine.  Measured, streaming ->
// tcgen05 kernel:
//   block  bf16, 4096 x 14336: 8 rows 57 -> 88 us, 16 rows 60 -> 88, 32 rows 74 -> 89;
//          1024 x 2816: 32 rows 12.8 -> 22.8
//          fp32, 4096 x 14336: 16 rows 365 -> 675 us, 32 rows 708 -> 664;
//          1024 x 2816: 32 rows 53 -> 81
//   loss   bf16, 4096 x 131072: 8 rows 157 -> 167 us, 16 rows 175 -> 167;
//          4096 x 32000: 8 rows 47 -> 53, 16 rows 52 -> 53;
//          1024 x 32000: 8 rows 18.0 -> 22.6, 16 rows 24.2 -> 22.6
//          fp32, 4096 x 32000: 16 rows 261 -> 450 us, 24 rows 403 -> 449;
//          1024 x 32000: 16 rows 95 -> 124, 24 rows 137 -> 124
constexpr int kStreamTokens = 32, kStreamLossTokens = 8, kStreamLossTokensF32 = 16;
int ops_stream_block(int64_t tokens, bool f32);  // LOGITS: columns per statistics block
cudaError_t launch_ops_stream(const OpsStream& a, int32_t kind, bool f32, cudaStream_t s);

constexpr int64_t kOpsSlotFloats = 256 * 256;  // one partial accumulator of a pair tile
constexpr int kOpsTailCounts = 16;             // counters per split tile

// What the schedule of a launch depends on, of one product: its K in slabs over
// all segments, and the columns per tile.
struct OpsShape {
    int64_t M, N;
    int32_t total, dual, bn;
};
// Chooses the columns per tile of a launch's products.  Host only.
void ops_tile_columns(OpsShape* p, int n, int pairs);
// Splits the launch's problems into work units (see OpsProblem) for `pairs`
// resident CTA pairs; `slots` partial-sum slots are available.  Host only.
void ops_schedule(OpsLaunch& l, int pairs, int slots, int tails);
cudaError_t ops_pairs(int* pairs);  // resident CTA pairs of the GEMM kernel on the current device
cudaError_t ops_status_word(void** p);   // the GEMM's time-out flag on the current device
cudaError_t norm_status_word(void** p);  // the same of the layer norm's ring kernels
cudaError_t launch_ops_gemm(const OpsLaunch& l, int32_t kind, bool f32, cudaStream_t s);

}  // namespace dmuon
