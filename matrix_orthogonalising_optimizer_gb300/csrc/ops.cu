// Host side of the gated feed-forward block and the vocabulary loss: argument
// checks, workspace layout, tensor maps and launches, and the two small
// kernels around the shared tensor-core GEMM (ops_gemm.cu) -- the operand
// pack (fp32 into bf16 parts, rows whose stride TMA cannot take into padded
// ones) and the loss's row pass.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "act.cuh"
#include "attn.h"
#include "checks.h"
#include "dmuon.h"
#include "ops.h"
#include "tc.cuh"

namespace dmuon {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxVocab = int64_t(1) << 22;
// K slabs per chain of MMAs under register sums: 512 deep for logits of bf16
// operands, 256 for fp32 operands (their error against 64-bit products: 1.5e-6
// with 512, against about 9e-7 of fp32 FMAs)
constexpr int kChain = 8, kChainF32 = 4;
// bf16 sums over more slabs than kLongSum (131072 deep) are added up in registers
// too, from chains of kLongChain slabs, so that they drift by less than 2^-13 of
// the sum.  Measured on 140000 terms of one sign: 8.6e-4 of the sum too little in one
// chain (9.8e-8 per 16 terms), 1.4e-4 in chains of 512 slabs, 5.1e-5 in these; a
// sum of kLongSum slabs, left in one chain, can lose 8e-4, a fifth of a bf16 ulp.
constexpr int kLongSum = 2048, kLongChain = 256;
// Up to this many bf16 tokens the logit gradients are kept in two bf16 parts: in one,
// the target's rounding, most of a token's gradient, is off by up to 2^-8, and a few
// tokens do not average that out (3 tokens, 64 x 5169: error of dW 2.8e-3 against
// 1.7e-3 of the result's own rounding).  More tokens do where their roundings differ,
// which the coefficients' common factor sees to (common_factor).  The parts are rows
// of one product for dx, which reads W once, and two part products of dW (3 tokens,
// 4096 x 131072: 687 us with one part, 690 with two, 961 with W read for each).
constexpr int kPartTokens = 32;
constexpr int kMaxLaunches = 4;   // GEMM launches of one call (of one piece)
constexpr int kSlots = 192;       // partial-sum slots: 48 MiB
constexpr int kTails = 192;       // split tiles per launch
constexpr int kStatusWords = 4;   // kernels with bounded waits: GEMM, layer norm, attention
constexpr uint64_t kDefaultBudget = uint64_t(2) << 30;

// ------------------------------------------------------------ workspace

// The coefficients of a call's tokens and where their common factor goes.
struct CoefArgs {
    const float* coef;  // NULL: nothing to do
    const int64_t* targets;
    int64_t n, ignore, vocab;
    float* factor;
};

// The factor, in [1, 2), that is left out of the logit gradients' bf16 values and
// multiplied into the products' sums: the significand of a coefficient that counts.
// With the usual one coefficient for all tokens what is left is a power of two,
// which adds no rounding; left in, its rounding is the same in every token's target,
// most of a token's gradient, so that no number of tokens averages it out (1 / 255
// is off by 2^-8: error of dx and dW 4.1e-3 at 255 tokens, 256 x 5169, untrained; now
// 1.7e-3, that of the results' own rounding).  What is left is the rounding of
// 1 - p: 2.0e-3 in all where the tokens' p differ, 2.2e-3 where all p are near
// 1 / 500.  A significand, not the coefficient, so that dz keeps its range; the
// largest of 4096 tokens, the first that have one, so that no order matters and one
// block does not read millions.
__device__ __forceinline__ void common_factor(const CoefArgs& c) {
    __shared__ uint32_t red[32];
    float factor = 1.0f;  // no normal coefficient
    for (int64_t i0 = threadIdx.x; i0 - threadIdx.x < c.n; i0 += 4096) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = i0 + 1024 * k;
            if (i >= c.n) break;
            const int64_t t = c.targets[i];
            const uint32_t b = __float_as_uint(c.coef[i]) & 0x7fffffffu;
            if (t != c.ignore && t >= 0 && t < c.vocab && b >= 0x00800000u && b < 0x7f800000u) top = max(top, b);
        }
        if (!__syncthreads_or(top != 0)) continue;
        top = __reduce_max_sync(tc::kFullMask, top);
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = top;
        __syncthreads();
        top = __reduce_max_sync(tc::kFullMask, red[threadIdx.x % 32]);
        factor = __uint_as_float(0x3f800000u | (top & 0x7fffffu));
        break;
    }
    if (threadIdx.x == 0) *c.factor = factor;
}

// Zeroes a launch's counters: n ints, a multiple of 64, at 256 bytes.  A kernel
// rather than a memset, so that the GEMM launched after it as a programmatic
// dependent sets up its barriers and tensor memory meanwhile.
__global__ void __launch_bounds__(1024) zero_kernel(int4* p, int n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * 1024 + threadIdx.x; i < n / 4; i += gridDim.x * 1024) p[i] = make_int4(0, 0, 0, 0);
}

// The same, and the last block finds the coefficients' common factor.
__global__ void __launch_bounds__(1024) zero_factor_kernel(int4* p, int n, const __grid_constant__ CoefArgs c) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x + 1 == gridDim.x) {
        common_factor(c);
        return;
    }
    for (int i = blockIdx.x * 1024 + threadIdx.x; i < n / 4; i += (gridDim.x - 1) * 1024) p[i] = make_int4(0, 0, 0, 0);
}

// Counters and partial sums of a call's GEMM launches.
struct Common {
    int32_t* counters = nullptr;  // [kMaxLaunches] unit counters, 64 ints apart, then the tail counts
    float* partials = nullptr;
    static constexpr int64_t kTailInts = int64_t(kTails) * kOpsTailCounts;
    static constexpr int64_t kInts = kMaxLaunches * (64 + kTailInts);
    void lay(Arena& a) {
        counters = a.take<int32_t>(kInts);
        partials = a.take<float>(kSlots * kOpsSlotFloats);
    }
    void bind(OpsLaunch& l, int launch) const {
        l.counter = counters + launch * 64;
        l.tail_count = counters + kMaxLaunches * 64 + launch * kTailInts;
        l.partials = partials;
    }
    // Zeroes the counters that the scheduled launches use (none where every
    // unit is some pair's first and no tile is split), and finds the
    // coefficients' common factor where there are some.
    cudaError_t clear(const OpsLaunch* l, int launches, int pairs, const CoefArgs& coef, cudaStream_t s) const {
        int64_t ints = 0;
        for (int i = 0; i < launches; ++i) {
            bool split = false;
            for (int k = 0; k < l[i].n; ++k) split = split || l[i].p[k].split > 1;
            if (split) ints = kMaxLaunches * 64 + (i + 1) * kTailInts;
            else if (l[i].total_units > pairs) ints = std::max<int64_t>(ints, (i + 1) * 64);
        }
        int4* p = reinterpret_cast<int4*>(counters);
        const int n = static_cast<int>(ints), blocks = static_cast<int>(ceil_div(ints, 4096));
        if (coef.coef) zero_factor_kernel<<<blocks + 1, 1024, 0, s>>>(p, n, coef);
        else if (ints > 0) zero_kernel<<<blocks, 1024, 0, s>>>(p, n);
        return cudaGetLastError();
    }
};

// An operand as the tensor cores read it: bf16 rows of 16-byte stride, `parts`
// of them; either the caller's matrix itself or a packed copy.
struct Operand {
    const void* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0, part = 0;
    int parts = 1;
};

// ------------------------------------------------------------ operand pack

constexpr int kMaxPacks = 6;

struct PackItem {
    const void* src;
    __nv_bfloat16* dst;
    int64_t rows, cols, ld, part, first;  // first: running count of 8-column groups
};

struct PackArgs {
    PackItem item[kMaxPacks];
    int32_t n;
    int32_t f32;
    int64_t groups;
};

// One thread per 8 destination columns: fp32 values split into three bf16
// parts, x = hi + mid + lo, or bf16 values copied.  Memory-bound; only fp32
// operands and row strides that are not a multiple of 16 bytes come here.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g < a.groups;
         g += static_cast<int64_t>(gridDim.x) * 256) {
        int k = 0;
        while (k + 1 < a.n && a.item[k + 1].first <= g) ++k;
        const PackItem& it = a.item[k];
        const int64_t gr = it.ld / 8, r = (g - it.first) / gr, c0 = (g - it.first - r * gr) * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t i = r * it.cols + c0 + j;
            v[j] = c0 + j >= it.cols ? 0.0f
                   : a.f32           ? static_cast<const float*>(it.src)[i]
                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(it.src)[i]);
        }
        __nv_bfloat16* d = it.dst + r * it.ld + c0;
        const int parts = a.f32 ? kF32Parts : 1;
        const bool plain = tc::all_plain(v);
        for (int p = 0; p < parts; ++p) {
            uint32_t w[8];
            tc::bf16_parts(v, w, plain);
            *reinterpret_cast<uint4*>(d + p * it.part) =
                make_uint4(tc::pack_parts(w[0], w[1]), tc::pack_parts(w[2], w[3]), tc::pack_parts(w[4], w[5]),
                           tc::pack_parts(w[6], w[7]));
        }
    }
}

struct Packer {
    PackArgs args = {};
    explicit Packer(bool f32) { args.f32 = f32 ? 1 : 0; }

    // The operand of the row-major contiguous matrix src (rows x cols); a copy
    // in the workspace where the tensor cores cannot read it in place.
    Operand add(Arena& a, const void* src, int64_t rows, int64_t cols) {
        Operand o;
        o.rows = rows;
        o.cols = cols;
        o.ld = up(cols, 8);
        o.parts = args.f32 ? kF32Parts : 1;
        o.part = rows * o.ld;
        if (!args.f32 && cols % 8 == 0) {
            o.p = src;
            return o;
        }
        __nv_bfloat16* d = a.take<__nv_bfloat16>(o.part * o.parts);
        o.p = d;
        PackItem& it = args.item[args.n++];
        it = PackItem{src, d, rows, cols, o.ld, o.part, args.groups};
        args.groups += rows * o.ld / 8;
        return o;
    }
    cudaError_t run(cudaStream_t s) const {
        if (args.groups == 0) return cudaSuccess;
        const int64_t blocks = std::min<int64_t>(ceil_div(args.groups, 256), 4096);
        return launch_dependent(pack_kernel, dim3(static_cast<unsigned>(blocks)), 256, s, args);
    }
};

// A bf16 (parts) buffer written by one product's epilogue and read by others.
Operand scratch(Arena& a, int64_t rows, int64_t cols, int parts, int64_t pad = 8) {
    Operand o;
    o.rows = rows;
    o.cols = cols;
    o.ld = up(cols, pad);
    o.parts = parts;
    o.part = rows * o.ld;
    o.p = a.take<__nv_bfloat16>(o.part * parts);
    return o;
}

OpsMat out_of(const Operand& o) {
    return OpsMat{const_cast<void*>(o.p), o.ld, ELEM_BF16, 1, o.parts > 1 ? o.part : 0};
}

OpsMat user_mat(const void* p, int64_t ld, bool f32) {
    return OpsMat{const_cast<void*>(p), ld, f32 ? ELEM_F32 : ELEM_BF16, ld % (f32 ? 4 : 8) == 0 ? 1 : 0, 0};
}

// ------------------------------------------------------------ products

int encode(CUtensorMap* map, const Operand& o, bool mn, int rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return fail(DMUON_ERR_CUDA, "cuTensorMapEncodeTiled entry point not found");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows),
                                static_cast<cuuint64_t>(o.parts)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld * 2), static_cast<cuuint64_t>(o.part * 2)};
    // K-major: 64 deep x `rows`; MN-major: 64 columns x 64 deep
    const cuuint32_t box[3] = {64, mn ? 64u : static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(DMUON_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
    return DMUON_OK;
}

// D (M x N) = sum over sources of A_s B_s, K deep each.  `dual`: B's two
// sources are two matrices of N rows against one A.
int set_problem(OpsProblem& P, int64_t M, int64_t N, int64_t K, const Operand* a, bool a_mn, const Operand* b,
                bool b_mn, int sources, bool dual, int bn) {
    const int na = dual ? 1 : sources;
    // With fewer than 256 rows in all, the rows of A beyond M are not loaded (64 rows
    // of 4096 x 14336: 118 -> 115 us): what their place in shared memory holds only
    // reaches accumulator rows that are never stored.
    const int rows = a_mn || M > 128 ? 128 : static_cast<int>(up(M, 8));
    P.a_rows[0] = rows;
    P.a_rows[1] = a_mn || M > 128 ? 128 : 0;
    for (int s = 0; s < na; ++s) OPS_TRY(encode(&P.a[s], a[s], a_mn, rows));
    for (int s = 0; s < sources; ++s) OPS_TRY(encode(&P.b[s], b[s], b_mn, bn / 2));
    P.bn = bn;
    P.maps_a = na;
    P.maps_b = sources;
    P.M = static_cast<int32_t>(M);
    P.N = static_cast<int32_t>(N);
    P.slabs = static_cast<int32_t>(ceil_div(K, 64));
    P.a_mn = a_mn;
    P.b_mn = b_mn;
    P.dual = dual;
    P.tiles_m = static_cast<int32_t>(ceil_div(M, 256));
    P.tiles_n = static_cast<int32_t>(ceil_div(N, dual ? bn / 2 : bn));
    // products of the operands' parts above 2^-24 of the whole, the smallest first
    static const int kPairs[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};
    P.nseg = 0;
    for (const auto& pair : kPairs)
        for (int s = 0; s < na && pair[0] < a[0].parts && pair[1] < b[0].parts; ++s)
            P.seg[P.nseg++] = static_cast<uint16_t>(s | pair[0] << 4 | pair[1] << 8);
    return DMUON_OK;
}

OpsShape shape_of(int64_t M, int64_t N, int64_t K, int sources, bool f32, bool dual = false) {
    return OpsShape{M, N, static_cast<int32_t>(ceil_div(K, 64) * sources * (f32 ? 6 : 1)), dual ? 1 : 0, 256};
}

// Columns per tile of a launch's only product.
int tile_columns(OpsShape s, int pairs) {
    ops_tile_columns(&s, 1, pairs);
    return s.bn;
}

bool is_long(const OpsLaunch& l) {
    bool r = false;
    for (int k = 0; k < l.n; ++k) r = r || l.p[k].slabs * l.p[k].nseg > kLongSum;
    return r;
}

// The instance with fp32 arithmetic and register sums also takes long sums of
// bf16 products.
cudaError_t launch(const OpsLaunch& l, int32_t kind, bool f32, cudaStream_t s) {
    return launch_ops_gemm(l, kind, f32 || is_long(l), s);
}

// Schedules a call's launches (`logits`: the first computes logits) and zeroes the
// counters they need.
int schedule(OpsLaunch* l, int launches, const Common& common, bool f32, bool logits, int pairs,
             cudaStream_t s, const char* where, const CoefArgs& coef = {}) {
    for (int i = 0; i < launches; ++i) {
        l[i].chain = f32 ? kChainF32 : logits && i == 0 ? kChain : kLongChain;
        common.bind(l[i], i);
        ops_schedule(l[i], pairs, kSlots, kTails);
    }
    OPS_CUDA(common.clear(l, launches, pairs, coef, s));
    return DMUON_OK;
}

// ------------------------------------------------------------ checks

// The streaming kernels take products of a few rows whose K they can read in
// whole 16-byte pieces.
bool use_stream(int64_t tokens, int64_t most, int64_t k0, int64_t k1, bool f32) {
    const int64_t vec = f32 ? 4 : 8;
    return tokens <= most && k0 % vec == 0 && k1 % vec == 0;
}

OpsStream stream_args(const void* x, const void* w, int64_t tokens, int64_t N, int64_t K) {
    OpsStream a = {};
    a.x = x;
    a.w[0] = w;
    a.ldx = K;
    a.ldw = K;
    a.tokens = static_cast<int32_t>(tokens);
    a.N = static_cast<int32_t>(N);
    a.K = static_cast<int32_t>(K);
    return a;
}

// ------------------------------------------------------------ gated block

struct FfnLayout {
    Common common;
    Packer pack;
    Operand x, wg, wu, wd, dy, h, da, du;
    size_t bytes = 0;

    // forward: h is written (in the caller's saved h where the next product can
    // read it there); backward: h is read
    FfnLayout(char* base, const void* px, const void* pg, const void* pu, const void* pd, const void* pdy,
              const void* ph, int64_t n, int64_t d, int64_t f, bool f32, bool backward)
        : pack(f32) {
        Arena a{base};
        if (!backward && use_stream(n, kStreamTokens, d, f, f32)) {
            h.p = a.take<char>(n * f * (f32 ? 4 : 2));
            if (ph) h.p = ph;
            bytes = a.off;
            return;
        }
        common.lay(a);
        x = pack.add(a, px, n, d);
        wg = pack.add(a, pg, f, d);
        wu = pack.add(a, pu, f, d);
        wd = pack.add(a, pd, d, f);
        const int parts = f32 ? kF32Parts : 1;
        if (backward) {
            dy = pack.add(a, pdy, n, d);
            h = pack.add(a, ph, n, f);
            da = scratch(a, n, f, parts);
            du = scratch(a, n, f, parts);
        } else {
            h = scratch(a, n, f, parts);
            if (ph && !f32 && f % 8 == 0) h.p = ph;
        }
        bytes = a.off;
    }
};

// act(a) and u act'(a) are kept in the tensors' type or in fp32.
int check_saved(int32_t saved, int32_t dtype, const char* where) {
    if (saved != DMUON_FP32 && saved != dtype)
        return fail(DMUON_ERR_UNSUPPORTED_DTYPE, std::string(where) + ": saved_dtype must be dtype or DMUON_FP32");
    return DMUON_OK;
}

bool ffn_sizes_ok(int64_t n, int64_t d, int64_t f) {
    return in_range(n, 0, kMaxTokens) && in_range(d, 1, kMaxWidth) && in_range(f, 1, kMaxWidth);
}

int check_ffn(int64_t n, int64_t d, int64_t f, int32_t dtype, const char* where) {
    if (!ffn_sizes_ok(n, d, f))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": tokens must be in [0, 2^24], dim and hidden in [1, 2^20]");
    return check_dtype(dtype, where);
}

// ------------------------------------------------------------ vocabulary loss

struct LossRowArgs {
    const float2* stats;        // [rows][nblk]
    const float* target_logit;  // [rows]
    const int64_t* targets;
    const float* coef;          // NULL: 1
    const float* factor;        // left out of dz, NULL: 1
    float* loss;
    float* lse;
    const void* e;              // exponentials (16-bit codes or fp32), NULL: losses only
    __nv_bfloat16* dz;          // logit gradients in `parts` bf16 parts
    int64_t ld, part, ignore;
    int64_t vocab;
    int32_t nblk, shift;        // statistics blocks of a row, log2 of their columns
    int32_t groups;             // 8-column groups of a row
    int32_t seg_groups;         // groups per blockIdx.y
    int32_t parts;              // kF32Parts for fp32, 2 or 1 for bf16
};

constexpr int kRowThreads = 256;

// Row pass of the loss.  Each block reduces its row's (max, sum) blocks to the
// maximum M and S = sum_b s_b exp(m_b - M), lse = M + log S, in a fixed order (a block
// without a finite logit has s_b = 0; a row without one gets lse = -inf, a NaN loss
// and a NaN gradient).  The first writes the loss, and each turns its share of the
// row's exponentials e = exp(z - m_b) into logit gradients dz = c e exp(m_b - M) / S,
// the target's as c expm1(-loss), so that p and 1 are not subtracted (what is left is
// the rounding of S, about 2^-23 of 1).  The loss is (M - z_t) + log S: lse itself
// loses log S where |M| is large (all of it for a row of equal masked logits), and
// with it the loss and every p.  Memory-bound: 4 bytes per bf16 logit, in place.
template <bool kF32>
__global__ void __launch_bounds__(kRowThreads) loss_row_kernel(const __grid_constant__ LossRowArgs a) {
    __shared__ float red[kRowThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float2* st = a.stats + row * a.nblk;
    float m = __int_as_float(0xff800000);
    for (int b = tid; b < a.nblk; b += kRowThreads) m = fmaxf(m, st[b].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(tc::kFullMask, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < kRowThreads / 32; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    const float ms = exp_shift(m);
    float s = 0.0f;
    for (int b = tid; b < a.nblk; b += kRowThreads) {
        const float2 v = st[b];
        s += v.y * expf(v.x - ms);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(tc::kFullMask, s, o);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) s += red[w];
    const float ls = logf(s);
    const int64_t t = a.targets[row];
    const bool ignored = t == a.ignore;
    const bool valid = !ignored && t >= 0 && t < a.vocab;
    const float nll = valid ? (m - a.target_logit[row]) + ls : 0.0f;
    if (blockIdx.y == 0 && tid == 0) {
        a.lse[row] = m + ls;
        a.loss[row] = valid || ignored ? nll : __int_as_float(0x7fc00000);
    }
    if (!a.e) return;
    float c = valid ? (a.coef ? a.coef[row] : 1.0f) : 0.0f;
    if (a.factor) c /= *a.factor;
    const float cs = c / s;
    const int tg = valid ? static_cast<int>(t >> 3) : -1, tk = static_cast<int>(t & 7);  // the target's group, place
    const int g0 = blockIdx.y * a.seg_groups, g1 = min(a.groups, g0 + a.seg_groups);
    for (int g = g0 + tid; g < g1; g += kRowThreads) {
        const int c0 = g * 8;
        const int64_t off = row * a.ld + c0;
        float v[8];
        if (!valid) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        } else {
            const float scale = cs * expf(st[c0 >> a.shift].x - ms);
            if (kF32) {
                const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.e) + off);
                const float4 x = p[0], y = p[1];
                v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
                v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.e) + off);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[2 * k] = e16_decode(w[k] & 0xffffu);
                    v[2 * k + 1] = e16_decode(w[k] >> 16);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= scale;
            if (g == tg) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k == tk) v[k] = c * expm1f(-nll);
            }
        }
        __nv_bfloat16* d = a.dz + off;
        if (kF32 || a.parts > 1) {
            const bool plain = tc::all_plain(v);
#pragma unroll
            for (int p = 0; p < (kF32 ? kF32Parts : 2); ++p) {
                uint32_t w[8];
                tc::bf16_parts(v, w, plain);
                *reinterpret_cast<uint4*>(d + p * a.part) =
                    make_uint4(tc::pack_parts(w[0], w[1]), tc::pack_parts(w[2], w[3]), tc::pack_parts(w[4], w[5]),
                               tc::pack_parts(w[6], w[7]));
            }
        } else {
            *reinterpret_cast<uint4*>(d) =
                make_uint4(tc::pack_bf16x2(v[0], v[1]), tc::pack_bf16x2(v[2], v[3]), tc::pack_bf16x2(v[4], v[5]),
                           tc::pack_bf16x2(v[6], v[7]));
        }
    }
}

// dx = bf16(s_r + s_(n+r)): the sums of the two parts' rows.
__global__ void __launch_bounds__(256) add_parts_kernel(const float* s, int64_t ld, int n, int dim,
                                                        __nv_bfloat16* dx) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.y;
    for (int c = blockIdx.x * 256 + threadIdx.x; c < dim; c += gridDim.x * 256)
        dx[static_cast<int64_t>(r) * dim + c] = __float2bfloat16_rn(s[r * ld + c] + s[(n + r) * ld + c]);
}

struct LossLayout {
    Common common;
    Packer pack;
    Operand x, w, dz;
    void* e = nullptr;         // exponentials (bf16: in dz's buffer)
    float2* stats = nullptr;
    float* target_logit = nullptr;
    float* factor = nullptr;   // bf16, one part: left out of dz
    float* dx_sum = nullptr;   // bf16, two parts: fp32 dx of each part
    float* dw_sum = nullptr;   // fp32 sum of dW over pieces (bf16, more than one piece)
    int64_t piece = 0, pieces = 0;  // tokens per piece
    bool stream;               // a few rows: the streaming kernel
    int block = 128, nblk = 0;  // columns per statistics block, blocks
    size_t bytes = 0;

    LossLayout(char* base, const void* px, const void* pw, int64_t n, int64_t d, int64_t v, bool f32, bool grad,
               uint64_t budget)
        : pack(f32) {
        Arena a{base};
        stream = use_stream(n, f32 ? kStreamLossTokensF32 : kStreamLossTokens, d, d, f32);
        if (stream) block = ops_stream_block(n, f32);
        if (grad || !stream) {
            common.lay(a);
            x = pack.add(a, px, n, d);
            w = pack.add(a, pw, v, d);
        }
        nblk = static_cast<int>(ceil_div(v, block));
        const int64_t ld = up(v, 16);  // whole epilogue chunks
        // bytes of one token's logits: statistics, exponentials, gradients
        const int64_t row = 8 * nblk + (grad ? (f32 ? 10 : 2) * ld : 0);
        const int64_t limit = static_cast<int64_t>(std::min<uint64_t>(budget ? budget : kDefaultBudget, 1ull << 46));
        // whole 256-row tiles per piece, at least one; pieces of equal size
        piece = std::max<int64_t>(limit / row / 256 * 256, 256);
        pieces = std::max<int64_t>(ceil_div(n, piece), 1);
        piece = std::min(n, up(ceil_div(n, pieces), 256));
        pieces = n > 0 ? ceil_div(n, piece) : 0;
        stats = a.take<float2>(piece * nblk);
        target_logit = a.take<float>(piece);
        if (grad) {
            dz = scratch(a, piece, v, f32 ? kF32Parts : n <= kPartTokens ? 2 : 1, 16);
            e = f32 ? static_cast<void*>(a.take<float>(piece * ld)) : const_cast<void*>(dz.p);
            if (!f32 && dz.parts == 1) factor = a.take<float>(1);
            if (!f32 && dz.parts > 1) dx_sum = a.take<float>(2 * n * up(d, 4));
            if (!f32 && pieces > 1) dw_sum = a.take<float>(v * up(d, 4));
        }
        bytes = a.off;
    }
};

bool loss_sizes_ok(int64_t n, int64_t d, int64_t v) {
    return in_range(n, 0, kMaxTokens) && in_range(d, 1, kMaxWidth) && in_range(v, 1, kMaxVocab);
}

// Reads and clears the time-out flags in one step, so that none set meanwhile is lost.
struct StatusWords {
    void* p[kStatusWords];
};
__device__ int32_t g_taken;
__global__ void take_status_kernel(StatusWords w) {
    int32_t v = 0;
    for (int i = 0; i < kStatusWords; ++i) v |= atomicExch(static_cast<int32_t*>(w.p[i]), 0);
    g_taken = v;
}

// Rows [r0, r0 + n) of an operand.
Operand rows_of(const Operand& o, int64_t r0, int64_t n) {
    Operand s = o;
    s.p = static_cast<const __nv_bfloat16*>(o.p) + r0 * o.ld;
    s.rows = n;
    return s;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" int dmuon_ops_status(void) {
    const char* where = "dmuon_ops_status";
    static std::mutex one;  // g_taken serves one caller at a time
    std::lock_guard<std::mutex> lock(one);
    StatusWords words = {};
    OPS_CUDA(ops_status_word(&words.p[0]));
    OPS_CUDA(norm_status_word(&words.p[1]));
    OPS_CUDA(attn_fwd_status_word(&words.p[2]));
    OPS_CUDA(attn_bwd_status_word(&words.p[3]));
    // every stream's calls: a copy alone would wait for the legacy stream and those
    // that synchronise with it
    OPS_CUDA(cudaDeviceSynchronize());
    take_status_kernel<<<1, 1>>>(words);
    OPS_CUDA(cudaGetLastError());
    int32_t v = 0;
    OPS_CUDA(cudaMemcpyFromSymbol(&v, g_taken, sizeof(v)));
    return v ? DMUON_ERR_DEVICE_TIMEOUT : DMUON_OK;
}

extern "C" size_t dmuon_gated_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t hidden, int32_t dtype,
                                                  int32_t backward) {
    if (!ffn_sizes_ok(tokens, dim, hidden) || check_dtype(dtype, "dmuon_gated_ffn_workspace_bytes") != DMUON_OK)
        return 0;
    if (tokens == 0) return 0;
    return FfnLayout(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, tokens, dim, hidden,
                     dtype == DMUON_FP32, backward != 0)
        .bytes;
}

extern "C" int dmuon_gated_ffn_forward(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                                       void* y, void* saved_act, void* saved_slope, void* saved_h,
                                       int32_t saved_dtype, int64_t tokens, int64_t dim, int64_t hidden, int32_t dtype,
                                       int32_t activation, void* workspace, size_t workspace_bytes, void* stream) {
    const char* where = "dmuon_gated_ffn_forward";
    OPS_TRY(check_ffn(tokens, dim, hidden, dtype, where));
    if (activation != DMUON_ACT_SILU && activation != DMUON_ACT_GELU)
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": unknown activation");
    if ((saved_act == nullptr) != (saved_slope == nullptr) || (saved_act == nullptr) != (saved_h == nullptr))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": saved_act, saved_slope and saved_h are stored together or not at all");
    if (saved_act) OPS_TRY(check_saved(saved_dtype, dtype, where));
    if (tokens == 0) return DMUON_OK;
    OPS_TRY(check_ptr(x, "x", where));
    OPS_TRY(check_ptr(w_gate, "w_gate", where));
    OPS_TRY(check_ptr(w_up, "w_up", where));
    OPS_TRY(check_ptr(w_down, "w_down", where));
    OPS_TRY(check_ptr(y, "y", where));
    if (saved_act) {
        OPS_TRY(check_ptr(saved_act, "saved_act", where));
        OPS_TRY(check_ptr(saved_slope, "saved_slope", where));
        OPS_TRY(check_ptr(saved_h, "saved_h", where));
    }
    const bool f32 = dtype == DMUON_FP32;
    FfnLayout L(static_cast<char*>(workspace), x, w_gate, w_up, w_down, nullptr, saved_h, tokens, dim, hidden, f32,
                false);
    OPS_TRY(check_workspace(workspace, workspace_bytes, L.bytes, where));
    OPS_TRY(check_device(where));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (use_stream(tokens, kStreamTokens, dim, hidden, f32)) {
        // h in dtype, in the caller's saved_h if there is one
        OpsStream a = stream_args(x, w_gate, tokens, hidden, dim);
        a.w[1] = w_up;
        a.act = activation == DMUON_ACT_GELU ? OPS_GELU : OPS_SILU;
        a.out[0] = user_mat(L.h.p, hidden, f32);
        if (saved_act) {
            a.out[1] = user_mat(saved_act, hidden, saved_dtype == DMUON_FP32);
            a.out[2] = user_mat(saved_slope, hidden, saved_dtype == DMUON_FP32);
        }
        OPS_CUDA(launch_ops_stream(a, OPS_GATE, f32, s));
        a = stream_args(L.h.p, w_down, tokens, dim, hidden);
        a.after = 1;
        a.out[0] = user_mat(y, dim, f32);
        OPS_CUDA(launch_ops_stream(a, OPS_STORE, f32, s));
        return DMUON_OK;
    }
    int pairs = 0;
    OPS_CUDA(ops_pairs(&pairs));
    OpsLaunch l[2] = {};
    l[0].n = l[1].n = 1;
    OpsProblem& P = l[0].p[0];
    const Operand b[2] = {L.wg, L.wu};
    OPS_TRY(set_problem(P, tokens, hidden, dim, &L.x, false, b, false, 2, true,
                        tile_columns(shape_of(tokens, hidden, dim, 1, f32, true), pairs)));
    P.act = activation == DMUON_ACT_GELU ? OPS_GELU : OPS_SILU;
    P.out[0] = out_of(L.h);
    if (saved_act) {
        P.out[1] = user_mat(saved_act, hidden, saved_dtype == DMUON_FP32);
        P.out[2] = user_mat(saved_slope, hidden, saved_dtype == DMUON_FP32);
        if (L.h.p != saved_h) P.out[3] = user_mat(saved_h, hidden, f32);
    }
    OPS_TRY(set_problem(l[1].p[0], tokens, dim, hidden, &L.h, false, &L.wd, false, 1, false,
                        tile_columns(shape_of(tokens, dim, hidden, 1, f32), pairs)));
    l[1].p[0].out[0] = user_mat(y, dim, f32);
    OPS_TRY(schedule(l, 2, L.common, f32, false, pairs, s, where));
    OPS_CUDA(L.pack.run(s));
    OPS_CUDA(launch(l[0], OPS_GATE, f32, s));
    OPS_CUDA(launch(l[1], OPS_STORE, f32, s));
    return DMUON_OK;
}

extern "C" int dmuon_gated_ffn_backward(const void* dy, const void* x, const void* w_gate, const void* w_up,
                                        const void* w_down, const void* saved_act, const void* saved_slope,
                                        const void* saved_h, int32_t saved_dtype, void* dx, void* dw_gate, void* dw_up,
                                        void* dw_down, int64_t tokens, int64_t dim, int64_t hidden, int32_t dtype,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    const char* where = "dmuon_gated_ffn_backward";
    OPS_TRY(check_ffn(tokens, dim, hidden, dtype, where));
    OPS_TRY(check_saved(saved_dtype, dtype, where));
    OPS_TRY(check_ptr(dw_gate, "dw_gate", where));
    OPS_TRY(check_ptr(dw_up, "dw_up", where));
    OPS_TRY(check_ptr(dw_down, "dw_down", where));
    const bool f32 = dtype == DMUON_FP32;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {  // no rows: the weights' gradients are sums over none
        const size_t bytes = static_cast<size_t>(dim) * hidden * (f32 ? 4 : 2);
        OPS_CUDA(cudaMemsetAsync(dw_gate, 0, bytes, s));
        OPS_CUDA(cudaMemsetAsync(dw_up, 0, bytes, s));
        OPS_CUDA(cudaMemsetAsync(dw_down, 0, bytes, s));
        return DMUON_OK;
    }
    OPS_TRY(check_ptr(dy, "dy", where));
    OPS_TRY(check_ptr(x, "x", where));
    OPS_TRY(check_ptr(w_gate, "w_gate", where));
    OPS_TRY(check_ptr(w_up, "w_up", where));
    OPS_TRY(check_ptr(w_down, "w_down", where));
    OPS_TRY(check_ptr(saved_act, "saved_act", where));
    OPS_TRY(check_ptr(saved_slope, "saved_slope", where));
    OPS_TRY(check_ptr(saved_h, "saved_h", where));
    OPS_TRY(check_ptr(dx, "dx", where));
    FfnLayout L(static_cast<char*>(workspace), x, w_gate, w_up, w_down, dy, saved_h, tokens, dim, hidden, f32, true);
    OPS_TRY(check_workspace(workspace, workspace_bytes, L.bytes, where));
    OPS_TRY(check_device(where));
    int pairs = 0;
    OPS_CUDA(ops_pairs(&pairs));
    OpsLaunch l[2] = {};
    // dh = dy Wd; the epilogue turns it into da and du
    l[0].n = 1;
    OpsProblem& P = l[0].p[0];
    OPS_TRY(set_problem(P, tokens, hidden, dim, &L.dy, false, &L.wd, true, 1, false,
                        tile_columns(shape_of(tokens, hidden, dim, 1, f32), pairs)));
    P.in[0] = user_mat(saved_slope, hidden, saved_dtype == DMUON_FP32);
    P.in[1] = user_mat(saved_act, hidden, saved_dtype == DMUON_FP32);
    P.out[0] = out_of(L.da);
    P.out[1] = out_of(L.du);
    // dx and the three weight gradients in one launch, the longest K first
    l[1].n = 4;
    OpsProblem* p = l[1].p;
    const bool dx_first = 2 * hidden >= tokens;
    int k = dx_first ? 1 : 0;
    OpsShape sh[4];
    sh[k] = sh[k + 1] = shape_of(hidden, dim, tokens, 1, f32);
    sh[k + 2] = shape_of(dim, hidden, tokens, 1, f32);
    sh[dx_first ? 0 : 3] = shape_of(tokens, dim, hidden, 2, f32);
    ops_tile_columns(sh, 4, pairs);
    OPS_TRY(set_problem(p[k], hidden, dim, tokens, &L.da, true, &L.x, true, 1, false, sh[k].bn));
    p[k++].out[0] = user_mat(dw_gate, dim, f32);
    OPS_TRY(set_problem(p[k], hidden, dim, tokens, &L.du, true, &L.x, true, 1, false, sh[k].bn));
    p[k++].out[0] = user_mat(dw_up, dim, f32);
    OPS_TRY(set_problem(p[k], dim, hidden, tokens, &L.dy, true, &L.h, true, 1, false, sh[k].bn));
    p[k++].out[0] = user_mat(dw_down, hidden, f32);
    k = dx_first ? 0 : 3;
    const Operand a[2] = {L.da, L.du}, b[2] = {L.wg, L.wu};
    OPS_TRY(set_problem(p[k], tokens, dim, hidden, a, false, b, true, 2, false, sh[k].bn));
    p[k].out[0] = user_mat(dx, dim, f32);
    OPS_TRY(schedule(l, 2, L.common, f32, false, pairs, s, where));
    OPS_CUDA(L.pack.run(s));
    OPS_CUDA(launch(l[0], OPS_DGATE, f32, s));
    OPS_CUDA(launch(l[1], OPS_STORE, f32, s));
    return DMUON_OK;
}

extern "C" size_t dmuon_vocab_loss_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab, int32_t dtype,
                                                   int32_t grad, uint64_t budget) {
    if (!loss_sizes_ok(tokens, dim, vocab) || check_dtype(dtype, "dmuon_vocab_loss_workspace_bytes") != DMUON_OK)
        return 0;
    if (tokens == 0) return 0;
    return LossLayout(nullptr, nullptr, nullptr, tokens, dim, vocab, dtype == DMUON_FP32, grad != 0, budget).bytes;
}

extern "C" int dmuon_vocab_loss(const void* x, const void* weight, const int64_t* targets, const float* coef,
                                int64_t ignore_index, float* loss, float* lse, void* dx, void* dweight, int64_t tokens,
                                int64_t dim, int64_t vocab, int32_t dtype, uint64_t budget, void* workspace,
                                size_t workspace_bytes, void* stream) {
    const char* where = "dmuon_vocab_loss";
    if (!loss_sizes_ok(tokens, dim, vocab))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": tokens must be in [0, 2^24], dim in [1, 2^20], vocab in [1, 2^22]");
    OPS_TRY(check_dtype(dtype, where));
    if (tokens > 0 && (dx == nullptr) != (dweight == nullptr))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": dx and dweight come together or not at all");
    const bool f32 = dtype == DMUON_FP32, grad = dweight != nullptr;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (grad) OPS_TRY(check_ptr(dweight, "dweight", where));
    if (tokens == 0) {
        if (grad) OPS_CUDA(cudaMemsetAsync(dweight, 0, static_cast<size_t>(vocab) * dim * (f32 ? 4 : 2), s));
        return DMUON_OK;
    }
    OPS_TRY(check_ptr(x, "x", where));
    OPS_TRY(check_ptr(weight, "weight", where));
    OPS_TRY(check_ptr(targets, "targets", where, 8));
    OPS_TRY(check_ptr(loss, "loss", where, 4));
    OPS_TRY(check_ptr(lse, "lse", where, 4));
    if (grad) OPS_TRY(check_ptr(dx, "dx", where));
    if (coef) OPS_TRY(check_ptr(coef, "coef", where, 4));
    LossLayout L(static_cast<char*>(workspace), x, weight, tokens, dim, vocab, f32, grad, budget);
    OPS_TRY(check_workspace(workspace, workspace_bytes, L.bytes, where));
    OPS_TRY(check_device(where));
    int pairs = 0;
    OPS_CUDA(ops_pairs(&pairs));
    const int64_t es = f32 ? 4 : 2;
    float* factor = coef ? L.factor : nullptr;  // all coefficients 1: as it is
    for (int64_t i = 0; i < L.pieces; ++i) {
        const int64_t r0 = i * L.piece, n = std::min(L.piece, tokens - r0);
        const Operand xp = rows_of(L.x, r0, n), dz = rows_of(L.dz, 0, n);
        // logits; then, from dz, dx (K = vocab) and dW (K = the piece's tokens)
        // in one launch
        OpsLaunch l[2] = {};
        if (!L.stream) {
            l[0].n = 1;
            OpsProblem& P = l[0].p[0];
            OPS_TRY(set_problem(P, n, vocab, dim, &xp, false, &L.w, false, 1, false, 256));
            P.stats = L.stats;
            P.nblk = L.nblk;
            P.target_logit = L.target_logit;
            P.targets = targets + r0;
            if (grad) P.out[0] = OpsMat{L.e, L.dz.ld, f32 ? ELEM_F32 : ELEM_BF16, 1, 0};
        }
        if (grad) {
            l[1].n = 2;
            const int kx = vocab >= n ? 0 : 1;
            OpsShape sh[2];
            Operand rows = dz;
            if (L.dx_sum) {  // the second part's rows follow the first's
                rows.rows = 2 * n;
                rows.parts = 1;
            }
            sh[kx] = shape_of(rows.rows, dim, vocab, 1, f32);
            sh[1 - kx] = shape_of(vocab, dim, n, f32 ? 1 : dz.parts, f32);
            ops_tile_columns(sh, 2, pairs);
            OPS_TRY(set_problem(l[1].p[kx], rows.rows, dim, vocab, &rows, false, &L.w, true, 1, false, sh[kx].bn));
            l[1].p[kx].out[0] = L.dx_sum ? user_mat(L.dx_sum, up(dim, 4), true)
                                         : user_mat(static_cast<char*>(dx) + r0 * dim * es, dim, f32);
            OpsProblem& W = l[1].p[1 - kx];
            OPS_TRY(set_problem(W, vocab, dim, n, &dz, true, &xp, true, 1, false, sh[1 - kx].bn));
            // the sum over pieces stays in fp32: rounded once, with the last piece
            const OpsMat sum = L.dw_sum ? user_mat(L.dw_sum, up(dim, 4), true) : user_mat(dweight, dim, f32);
            const bool last = i + 1 == L.pieces;
            W.out[0] = last ? user_mat(dweight, dim, f32) : sum;
            if (i > 0) W.in[0] = sum;
            l[1].scale = factor;
        }
        CoefArgs first = {};
        if (factor && i == 0) first = CoefArgs{coef, targets, tokens, ignore_index, vocab, factor};
        OPS_TRY(schedule(l, 2, L.common, f32, true, pairs, s, where, first));
        if (i == 0) OPS_CUDA(L.pack.run(s));
        if (L.stream) {
            OpsStream a = stream_args(static_cast<const char*>(x) + r0 * dim * es, weight, n, vocab, dim);
            a.stats = L.stats;
            a.nblk = L.nblk;
            a.target_logit = L.target_logit;
            a.targets = targets + r0;
            if (grad) a.out[0] = OpsMat{L.e, L.dz.ld, f32 ? ELEM_F32 : ELEM_BF16, 1, 0};
            OPS_CUDA(launch_ops_stream(a, OPS_LOGITS, f32, s));
        } else {
            OPS_CUDA(launch_ops_gemm(l[0], OPS_LOGITS, f32, s));
        }
        LossRowArgs a = {};
        a.stats = L.stats;
        a.target_logit = L.target_logit;
        a.targets = targets + r0;
        a.coef = coef ? coef + r0 : nullptr;
        a.factor = factor;
        a.loss = loss + r0;
        a.lse = lse + r0;
        a.ignore = ignore_index;
        a.vocab = vocab;
        a.nblk = L.nblk;
        while ((1 << a.shift) < L.block) ++a.shift;
        int segs = 1;
        if (grad) {
            a.e = L.e;
            a.dz = static_cast<__nv_bfloat16*>(const_cast<void*>(L.dz.p));
            a.ld = L.dz.ld;
            a.part = L.dz.part;
            a.parts = L.dz.parts;
            a.groups = static_cast<int32_t>(ceil_div(vocab, 8));
            // a few rows: share each row among blocks, so that about 1200 run
            segs = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(a.groups, 1024), 1200 / n)));
            a.seg_groups = static_cast<int32_t>(ceil_div(a.groups, segs));
        }
        const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(segs));
        OPS_CUDA(launch_dependent(f32 ? loss_row_kernel<true> : loss_row_kernel<false>, grid, kRowThreads, s, a));
        if (grad) OPS_CUDA(launch(l[1], factor ? OPS_STORE_SCALED : OPS_STORE, f32, s));
        if (L.dx_sum)
            OPS_CUDA(launch_dependent(add_parts_kernel,
                                      dim3(static_cast<unsigned>(ceil_div(dim, 256)), static_cast<unsigned>(n)), 256, s,
                                      L.dx_sum, up(dim, 4), static_cast<int>(n), static_cast<int>(dim),
                                      static_cast<__nv_bfloat16*>(dx)));
    }
    return DMUON_OK;
}
