// Grouped GEMM of the training operators on the 5th-generation tensor cores
// (sm_103a), with the operators' element-wise parts fused into its epilogue.
//
// One launch holds up to four products D = A B of any sizes, each with A and B
// K-major or MN-major, so every product of a forward and a backward pass reads
// its operands where they lie (no transposed copies):
//   gated block  h = act(x Wg^T) * (x Wu^T)   one pass, dual B tile   OPS_GATE
//                y = h Wd^T                                           OPS_STORE
//                dh = dy Wd -> da, du, h                              OPS_DGATE
//                dx = da Wg + du Wu (two K sources), dW = . ^T .      OPS_STORE
//   vocab loss   z = x W^T -> exp(z - block max), block max and sum   OPS_LOGITS
//                dx = dz W, dW = dz^T x                               OPS_STORE
//
// What bounds it: the tensor cores for more than a few hundred rows, else the
// read of the weights.  A 256 x 256 tile of a CTA pair
// (tcgen05.mma.cta_group::2, CTA rank r holds rows 128 r .. of A and columns
// 128 r .. of B in its own shared memory) takes 32 KB of operands per CTA and
// 64-deep K slab from L2 for 8.4 MFLOP, and six such stages are in flight.
// Two 256-column TMEM accumulators let the eight epilogue warps work on one
// tile while the next one's MMAs run.  Measured at 8192 x 4096 x 14336 and 4096 x
// 4096 x 131072: tensor pipe 92 to 99 % active (DGATE 77 %: 1.4 GB of stored
// activations and gradients beside the operands), the whole training step
// 5.1 to 5.4 ms = 1.61 to 1.71 PFLOP/s, where the power cap sets the clock.
//
// Schedule: units are taken in order from a counter (neighbouring tiles stay
// together in L2).  Tiles that would leave most pairs idle at the end of a
// launch are split along K (ops_schedule): each unit of a split tile stores its
// partial sum, and the warp that arrives last at a tile's counter adds the
// partial sums in K order -- a fixed order, so results do not depend on which
// unit was last -- and runs the epilogue.  No unit waits for another.
//
// Warp roles and the bounded waits are those of the optimizer's GEMM
// (gemm_tc.cu): warp 0 TMA, warp 1 MMA (leader CTA), warps 4..11 epilogue.
#include <type_traits>

#include "act.cuh"
#include "ops.h"
#include "tc.cuh"

namespace dmuon {
namespace {

using namespace tc;

// set by a wait that gave up; read and cleared by dmuon_ops_status
__device__ int32_t g_ops_status = 0;

constexpr int BM = 128, BN = 256;               // per-CTA accumulator
constexpr int STAGES = 6;
constexpr int SLAB_K = 64;                      // bf16 per 128-byte swizzled row
constexpr int UMMA_K = 16;
constexpr int kPair = 2;
constexpr int kThreads = 384;
constexpr int OP_BYTES = 128 * 128;             // one CTA's share of an operand slab
constexpr int MN_BOX_BYTES = SLAB_K * 128;      // one MN-major box: 64 K-rows x 128 B
constexpr uint32_t TMEM_COLS = 512;
constexpr int kTileRing = 4;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kRegsLow = 56, kRegsEpi = 224;    // 56 + 2 x 224 = 3 x 168: the launch's registers
constexpr uint32_t kTileReaders = kPair * kEpiWarps + 2;
constexpr int CH = 16;
constexpr uint16_t kPairMask = 3;
constexpr int kStageLd = CH + 1;                // odd: rows and columns are both free of bank conflicts

struct __align__(1024) Smem {
    uint8_t a[STAGES][OP_BYTES];
    uint8_t b[STAGES][OP_BYTES];
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t tile_full[kTileRing];
    uint64_t tile_empty[kTileRing];
    int32_t tile_slot[kTileRing];
    uint32_t tmem_base;
    float stage[kEpiWarps][32 * kStageLd];  // a 32 x 16 chunk per epilogue warp (rows of unaligned matrices)
};

__device__ __forceinline__ uint32_t make_idesc(bool a_mn, bool b_mn, int bn) {
    // kind::f16: bf16 A and B, fp32 D, M = 256 (the pair), N = bn
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>((kPair * BM) >> 4) << 24);
}

struct Unit {
    int p, tm, tn, kb0, kb1, part, split, slot, tail;
};

__device__ __forceinline__ Unit decode_unit(const OpsLaunch& L, int t) {
    Unit u;
    u.p = 0;
    while (u.p + 1 < L.n && L.p[u.p + 1].unit_begin <= t) ++u.p;
    const OpsProblem& P = L.p[u.p];
    const int local = t - P.unit_begin;
    const int total = P.slabs * P.nseg;
    int tile = local;
    u.split = 1;
    u.part = u.slot = u.tail = 0;
    u.kb0 = 0;
    u.kb1 = total;
    if (local >= P.whole) {
        const int r = local - P.whole, tt = r / P.split;
        tile = P.whole + tt;
        u.split = P.split;
        u.part = r - tt * P.split;
        u.kb0 = static_cast<int>(static_cast<int64_t>(total) * u.part / P.split);
        u.kb1 = static_cast<int>(static_cast<int64_t>(total) * (u.part + 1) / P.split);
        u.slot = P.slot_begin + tt * P.split;
        u.tail = P.tail_begin + tt;
    }
    // panels of 8 column tiles, row tiles inside a panel: the pairs in flight
    // then cover about 10 x 8 tiles, whose rows and columns stay in L2
    constexpr int kPanel = 8;
    const int panel_tiles = P.tiles_m * kPanel;
    const int panel = tile / panel_tiles;
    const int within = tile - panel * panel_tiles;
    const int width = min(kPanel, P.tiles_n - panel * kPanel);
    u.tm = within / width;
    u.tn = panel * kPanel + within % width;
    return u;
}

__device__ __forceinline__ int wait_tile(uint64_t* full, const int32_t* slots, int k, int32_t* status, int total) {
    const int slot = k % kTileRing;
    const uint32_t ph = static_cast<uint32_t>(k / kTileRing) & 1u;
    if (!mbar_wait<true>(&full[slot], ph, status)) return total;
    int32_t t;
    asm volatile("ld.acquire.cluster.shared::cta.b32 %0, [%1];" : "=r"(t) : "r"(saddr(&slots[slot])) : "memory");
    return t;
}

__device__ __forceinline__ void release_tile(uint64_t* empty, int k) {
    mbar_arrive_cluster_relaxed(mapa(saddr(&empty[k % kTileRing]), 0));
}

// ------------------------------------------------------- matrix accesses
// After tcgen05.ld lane i of a warp holds row r0 + i, columns c0 .. c0 + 15.
// Whole chunks of 16-byte-aligned rows are regrouped between lanes so that one
// instruction covers whole 32-byte sectors; other chunks go through the warp's
// slice of shared memory and move as two 16-element row segments per
// instruction (element by element from each lane's own row, an instruction
// touches 32 rows: six times the sectors).  All 32 lanes call these; rows >= M
// and columns >= N are not touched.

template <typename T>
__device__ __forceinline__ void st_staged(T* base, int64_t ld, int r0, int c0, int lane, const float (&v)[CH], int M,
                                          int N, float* stg) {
#pragma unroll
    for (int j = 0; j < CH; ++j) stg[lane * kStageLd + j] = v[j];
    __syncwarp();
    const int c = lane % CH;
    T* p = base + (r0 + static_cast<int64_t>(lane / CH)) * ld + c0 + c;
    const int rows = c0 + c < N ? M - r0 - lane / CH : 0;
    // all loads before the first store (as ld_staged)
    float x[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) x[i] = stg[(2 * i + lane / CH) * kStageLd + c];
#pragma unroll
    for (int i = 0; i < CH; ++i, p += 2 * ld)
        if (2 * i < rows) {
            if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(x[i]);
            else *p = x[i];
        }
    __syncwarp();
}

template <typename T>
__device__ __forceinline__ void ld_staged(const T* base, int64_t ld, int r0, int c0, int lane, float (&v)[CH], int M,
                                          int N, float* stg) {
    const int c = lane % CH;
    const T* p = base + static_cast<int64_t>(r0) * ld + c0 + c;
    // all loads before the first store: the compiler cannot tell the staging
    // slice from the matrix and would wait for each in turn
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int r = 2 * i + lane / CH;
        v[i] = r0 + r < M && c0 + c < N ? static_cast<float>(p[r * ld]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) stg[(2 * i + lane / CH) * kStageLd + c] = v[i];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = stg[lane * kStageLd + j];
    __syncwarp();
}

// A whole chunk of 16-bit elements, two per word, in 16-byte-aligned rows.
__device__ __forceinline__ void st_words(void* base, int64_t ld, int r0, int c0, int lane, const uint32_t (&w)[8],
                                         int M) {
    const bool odd = lane & 1;
    uint32_t d0[4], d1[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t keep = odd ? w[4 + k] : w[k];
        const uint32_t recv = __shfl_xor_sync(kFullMask, odd ? w[k] : w[4 + k], 1);
        d0[k] = odd ? recv : keep;  // row (lane & ~1), half `odd`
        d1[k] = odd ? keep : recv;  // row (lane | 1),  half `odd`
    }
    const int ra = r0 + (lane & ~1);
    uint16_t* p = static_cast<uint16_t*>(base) + static_cast<int64_t>(ra) * ld + c0 + 8 * odd;
    if (ra < M) *reinterpret_cast<uint4*>(p) = make_uint4(d0[0], d0[1], d0[2], d0[3]);
    if (ra + 1 < M) *reinterpret_cast<uint4*>(p + ld) = make_uint4(d1[0], d1[1], d1[2], d1[3]);
}

__device__ __forceinline__ void st_bf16(__nv_bfloat16* base, int64_t ld, bool vec, int r0, int c0, int lane,
                                        const float (&v)[CH], int M, int N, float* stg) {
    if (!vec || c0 + CH > N) {
        st_staged(base, ld, r0, c0, lane, v, M, N, stg);
        return;
    }
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    st_words(base, ld, r0, c0, lane, w, M);
}

__device__ __forceinline__ void st_f32(float* base, int64_t ld, bool vec, int r0, int c0, int lane,
                                       const float (&v)[CH], int M, int N, float* stg) {
    if (!vec || c0 + CH > N) {
        st_staged(base, ld, r0, c0, lane, v, M, N, stg);
        return;
    }
    float w[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) w[j] = v[j];
    quad_transpose(w, lane);
    const int rq = r0 + (lane & ~3);
    float* p = base + static_cast<int64_t>(rq) * ld + c0 + 4 * (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (rq + j < M)
            *reinterpret_cast<float4*>(p + j * ld) = make_float4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// A matrix of the given element type, or of bf16 parts (part > 0).
__device__ __forceinline__ void st_mat(const OpsMat& m, int r0, int c0, int lane, float (&v)[CH], int M, int N,
                                       float* stg) {
    if (m.type == ELEM_F32) {
        st_f32(static_cast<float*>(m.p), m.ld, m.vec, r0, c0, lane, v, M, N, stg);
        return;
    }
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(m.p);
    if (m.part == 0) {
        st_bf16(p, m.ld, m.vec, r0, c0, lane, v, M, N, stg);
        return;
    }
    const bool plain = all_plain(v);
#pragma unroll 1
    for (int k = 0; k < kF32Parts; ++k, p += m.part) {
        uint32_t h[CH];
        bf16_parts(v, h, plain);
        if (m.vec && c0 + CH <= N) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = pack_parts(h[2 * j], h[2 * j + 1]);
            st_words(p, m.ld, r0, c0, lane, w, M);
        } else {
            float x[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) x[j] = __uint_as_float(h[j]);
            st_staged(p, m.ld, r0, c0, lane, x, M, N, stg);
        }
    }
}

// A load in two halves, so that several can be in flight: ld_issue's words are
// the lane's 16-byte pieces (or, for a staged chunk, its finished values), which
// ld_finish regroups.
__device__ __forceinline__ void ld_issue(const OpsMat& m, int r0, int c0, int lane, float (&x)[CH], int M, int N,
                                         float* stg) {
    if (!m.vec || c0 + CH > N) {
        if (m.type == ELEM_BF16)
            ld_staged(static_cast<const __nv_bfloat16*>(m.p), m.ld, r0, c0, lane, x, M, N, stg);
        else
            ld_staged(static_cast<const float*>(m.p), m.ld, r0, c0, lane, x, M, N, stg);
        return;
    }
    // bf16: two rows of a lane pair, 8 elements each; fp32: four rows of a quad, 4 each
    const bool bf = m.type == ELEM_BF16;
    const int rq = r0 + (bf ? lane & ~1 : lane & ~3);
    const int es = bf ? 2 : 4;
    const char* p = static_cast<const char*>(m.p) + (static_cast<int64_t>(rq) * m.ld + c0) * es +
                    16 * (bf ? lane & 1 : lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if ((j < 2 || !bf) && rq + j < M) q = *reinterpret_cast<const float4*>(p + j * m.ld * es);
        x[4 * j] = q.x;
        x[4 * j + 1] = q.y;
        x[4 * j + 2] = q.z;
        x[4 * j + 3] = q.w;
    }
}

__device__ __forceinline__ void ld_finish(const OpsMat& m, int c0, int lane, float (&x)[CH], int N) {
    if (!m.vec || c0 + CH > N) return;
    if (m.type != ELEM_BF16) {
        quad_transpose(x, lane);
        return;
    }
    const bool odd = lane & 1;
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t d0 = __float_as_uint(x[k]), d1 = __float_as_uint(x[4 + k]);
        const uint32_t recv = __shfl_xor_sync(kFullMask, odd ? d0 : d1, 1);
        w[k] = odd ? recv : d0;
        w[4 + k] = odd ? d1 : recv;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 f = unpack_bf16x2(w[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}

// ------------------------------------------------------- accumulator source
// A warp's share of an accumulator is bn / 2 columns of 32 rows: columns (bn / 2)
// half .. of the tile, or for the dual tile columns (bn / 4) half .. of each of its
// two matrices.  It is worked off in chunks of 16 columns; chunk ci of eight (dual:
// ci / 4 is the matrix) starts at this accumulator column.  With bn = 128 the
// upper chunks (of each matrix) do not exist.

template <int kKind>
__device__ __forceinline__ int chunk_col(int bn, int half, int ci) {
    if (kKind == OPS_GATE) return (ci >> 2) * (bn / 2) + half * (bn / 4) + (ci & 3) * CH;
    return half * (bn / 2) + ci * CH;
}

template <int kKind>
__device__ __forceinline__ bool chunk_in(int bn, int ci) {
    return bn == BN || (kKind == OPS_GATE ? (ci & 3) < 2 : ci < 4);
}

// First output column of a warp's share, and its chunks (per matrix).
template <int kKind>
__device__ __forceinline__ int first_col(int bn, int tn, int half) {
    return kKind == OPS_GATE ? tn * (bn / 2) + half * (bn / 4) : tn * bn + half * (bn / 2);
}

// Sums left in TMEM (one chain of MMAs over the tile's whole K range).
template <int kKind>
struct TmemSrc {
    uint32_t taddr;
    int bn, half;
    __device__ __forceinline__ void load(int ci, float (&v)[CH]) {
        __syncwarp();
        tmem_ld16(taddr + static_cast<uint32_t>(chunk_col<kKind>(bn, half, ci)), v);
    }
    __device__ __forceinline__ void load_pair(int ci, float (&a)[CH], float (&b)[CH]) {
        load(ci, a);
        load(ci + 4, b);
    }
};

// Sums in registers, added up there from several shorter chains of MMAs or, for
// a split tile, from all units' stored partial sums.  Chunks are taken in order:
// each load hands out the first 16 values and moves the others down, so that
// the chunk loop stays a loop (unrolled eight times it tripled the code).
struct RegSrc {
    float (&r)[BN / 2];
    __device__ __forceinline__ void load(int, float (&v)[CH]) {
#pragma unroll
        for (int j = 0; j < CH; ++j) v[j] = r[j];
#pragma unroll
        for (int j = 0; j < BN / 2 - CH; ++j) r[j] = r[j + CH];
    }
    __device__ __forceinline__ void load_pair(int, float (&a)[CH], float (&b)[CH]) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            a[j] = r[j];
            b[j] = r[BN / 4 + j];
        }
#pragma unroll
        for (int j = 0; j < BN / 4 - CH; ++j) {
            r[j] = r[j + CH];
            r[BN / 4 + j] = r[BN / 4 + j + CH];
        }
    }
};

// ------------------------------------------------------- epilogues
// u: the unit; half: this warp's column half; r0: its first row.
//
// The loops over chunks, outputs and parts stay loops: an epilogue runs once or
// a few times per launch, so its instructions come from L2, and the first form,
// inlined per output and unrolled, spent 6 to 11 us per fp32 chunk on
// instruction fetches.

template <bool kScaled, typename Src>
__device__ __forceinline__ void epi_store(const OpsProblem& P, const float* factor, Src acc, const Unit& u, int half,
                                          int r0, int lane, float* stg) {
    const float scale = kScaled ? *factor : 1.0f;
#pragma unroll 1
    for (int kc = 0; kc < P.bn / 32; ++kc) {
        const int c0 = first_col<OPS_STORE>(P.bn, u.tn, half) + kc * CH;
        if (c0 >= P.N) break;
        float v[CH];
        acc.load(kc, v);
        if constexpr (kScaled) {
#pragma unroll
            for (int j = 0; j < CH; ++j) v[j] *= scale;
        }
        if (P.in[0].p) {
            float add[CH];
            ld_issue(P.in[0], r0, c0, lane, add, P.M, P.N, stg);
            ld_finish(P.in[0], c0, lane, add, P.N);
#pragma unroll
            for (int j = 0; j < CH; ++j) v[j] += add[j];
        }
        st_mat(P.out[0], r0, c0, lane, v, P.M, P.N, stg);
    }
}

template <bool kF32, typename Src>
__device__ __forceinline__ void epi_gate(const OpsProblem& P, Src acc, const Unit& u, int half, int r0, int lane,
                                         float* stg) {
#pragma unroll 1
    for (int kc = 0; kc < P.bn / 64; ++kc) {
        const int c0 = first_col<OPS_GATE>(P.bn, u.tn, half) + kc * CH;
        if (c0 >= P.N) break;
        float f[CH], s[CH], h[CH];
        acc.load_pair(kc, f, h);
        // one branch per chunk: the activations' instructions are fetched apart
        const auto activate = [&](auto act, auto save) {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const float a = f[j], w = h[j], g = act_gate<kF32>(decltype(act)::value, a);
                f[j] = a * g;
                h[j] = f[j] * w;
                if (decltype(save)::value) s[j] = w * act_slope<kF32>(decltype(act)::value, a, g);
            }
        };
        using Silu = std::integral_constant<int, OPS_SILU>;
        using Gelu = std::integral_constant<int, OPS_GELU>;
        if (P.act == OPS_SILU) {
            if (P.out[1].p) activate(Silu{}, std::true_type{});
            else activate(Silu{}, std::false_type{});
        } else {
            if (P.out[1].p) activate(Gelu{}, std::true_type{});
            else activate(Gelu{}, std::false_type{});
        }
#pragma unroll 1
        for (int o = 0; o < 4; ++o) {
            if (!P.out[o].p) continue;
            float v[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) v[j] = o == 1 ? f[j] : o == 2 ? s[j] : h[j];
            st_mat(P.out[o], r0, c0, lane, v, P.M, P.N, stg);
        }
    }
}

template <bool kF32, typename Src>
__device__ __forceinline__ void epi_dgate(const OpsProblem& P, Src acc, const Unit& u, int half, int r0, int lane,
                                          float* stg) {
    const int cb = first_col<OPS_DGATE>(P.bn, u.tn, half), chunks = P.bn / 32;
    // da = dh u act'(a), du = dh act(a); the next chunk's loads are issued before
    // this one's stores
    float ns[CH], nf[CH];
    ld_issue(P.in[0], r0, cb, lane, ns, P.M, P.N, stg);
    ld_issue(P.in[1], r0, cb, lane, nf, P.M, P.N, stg);
#pragma unroll 1
    for (int kc = 0; kc < chunks; ++kc) {
        const int c0 = cb + kc * CH;
        if (c0 >= P.N) break;
        float s[CH], f[CH], v[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            s[j] = ns[j];
            f[j] = nf[j];
        }
        ld_finish(P.in[0], c0, lane, s, P.N);
        ld_finish(P.in[1], c0, lane, f, P.N);
        if (kc + 1 < chunks && c0 + CH < P.N) {
            ld_issue(P.in[0], r0, c0 + CH, lane, ns, P.M, P.N, stg);
            ld_issue(P.in[1], r0, c0 + CH, lane, nf, P.M, P.N, stg);
        }
        acc.load(kc, v);
#pragma unroll 1
        for (int o = 0; o < 2; ++o) {
            float x[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) x[j] = (o ? f[j] : s[j]) * v[j];
            st_mat(P.out[o], r0, c0, lane, x, P.M, P.N, stg);
        }
    }
}

// exp(z - m).  The difference is taken before it is scaled: in z log2(e) - m log2(e),
// one FMA, the rounding of m log2(e) stays as an error of the exponent, and at
// |m| of 10^10 (masked logits) the maximum's own exponential became infinite.
// Two at a time: the subtraction and the scaling then cost what the FMA did.
template <bool kF32>
__device__ __forceinline__ void exp_pair(float& a, float& b, float m) {
    if constexpr (kF32) {
        a = expf(a - m);
        b = expf(b - m);
    } else {
        const float2 t = mul2(add2(make_float2(a, b), both(-m)), both(kLog2e));
        a = ex2(t.x);
        b = ex2(t.y);
    }
}

template <bool kF32>
__device__ __forceinline__ void epi_logits(const OpsProblem& P, const Unit& u, int half, int r0, int lane,
                                           float (&z)[BN / 2], float* stg) {
    const int cb = u.tn * BN + half * (BN / 2);
    const int r = r0 + lane;
    const float ninf = __int_as_float(0xff800000);
    if (cb + BN / 2 > P.N) {  // columns past the vocabulary: exp gives 0
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) z[j] = cb + j < P.N ? z[j] : ninf;
    }
    float mx[8];  // several chains: two warps per scheduler do not hide one
#pragma unroll
    for (int j = 0; j < 8; ++j) mx[j] = z[j];
#pragma unroll
    for (int j = 8; j < BN / 2; ++j) mx[j % 8] = fmaxf(mx[j % 8], z[j]);
    const float m = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                          fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
    const int64_t t = r < P.M ? P.targets[r] - cb : -1;
    if (t >= 0 && t < BN / 2 && cb + t < P.N) {
        float zt = 0.0f;
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) zt = t == j ? z[j] : zt;
        P.target_logit[r] = zt;
    }
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float ms = exp_shift(m);
    if (P.out[0].p) {
        RegSrc src{z};
#pragma unroll 1
        for (int kc = 0; kc < 8; ++kc) {
            if (cb + kc * CH >= P.N) break;
            float v[CH];
            src.load(kc, v);
#pragma unroll
            for (int j = 0; j < CH; j += 2) {
                exp_pair<kF32>(v[j], v[j + 1], ms);
                sum[j % 4] += v[j];
                sum[j % 4 + 1] += v[j + 1];
            }
            // rows are padded to whole chunks, so every chunk is stored whole
            if constexpr (kF32) {
                st_f32(static_cast<float*>(P.out[0].p), P.out[0].ld, true, r0, cb + kc * CH, lane, v, P.M,
                       static_cast<int>(P.out[0].ld), stg);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = e16_encode(v[2 * k]) | e16_encode(v[2 * k + 1]) << 16;
                st_words(P.out[0].p, P.out[0].ld, r0, cb + kc * CH, lane, w, P.M);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < BN / 2; j += 2) {
            exp_pair<kF32>(z[j], z[j + 1], ms);
            sum[j % 4] += z[j];
            sum[j % 4 + 1] += z[j + 1];
        }
    }
    if (r < P.M) P.stats[static_cast<int64_t>(r) * P.nblk + 2 * u.tn + half] =
        make_float2(m, (sum[0] + sum[1]) + (sum[2] + sum[3]));
}

template <int kKind, bool kF32>
__global__ void __launch_bounds__(kThreads, 1) ops_gemm_kernel(const __grid_constant__ OpsLaunch L) {
    // Sums that must keep fp32 accuracy (fp32 matrices, logits) are added up in
    // registers from chains of L.chain slabs: the tensor cores truncate each
    // addition to the accumulator, and over a 4096-deep chain that bias reached
    // 2.6e-6 of a logit, five times the error of fp32 FMAs.  Sums that a bf16
    // store rounds anyway stay in TMEM.
    constexpr bool kRegs = kF32 || kKind == OPS_LOGITS;
    extern __shared__ uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(kFullMask, static_cast<int>(threadIdx.x) / 32, 0);  // uniform to the compiler
    const int lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.acc_full[b], 1);
            mbar_init(&S.acc_empty[b], kPair * kEpiWarps);
        }
        for (int i = 0; i < kTileRing; ++i) {
            mbar_init(&S.tile_full[i], 1);
            mbar_init(&S.tile_empty[i], kTileReaders);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tmem = S.tmem_base;
    const int rank = static_cast<int>(cluster_rank());
    const int total = L.total_units;
    if (warp == 2 && lane < 4 * L.n) {
        // the used tensor maps into the descriptor cache before their first use
        const OpsProblem& P = L.p[lane / 4];
        const bool of_b = lane & 2, second = lane & 1;
        if (!second || (of_b ? P.maps_b : P.maps_a) > 1)
            asm volatile("prefetch.tensormap [%0];" ::"l"(
                             reinterpret_cast<uint64_t>(of_b ? &P.b[second] : &P.a[second]))
                         : "memory");
    }
    // programmatic dependent launch: global memory only after the previous
    // kernel has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            // (the whole warp runs the loop, one elected lane issues)
            const uint32_t e = elect_one();
            const uint32_t sa = saddr(S.a[0]), sb = saddr(S.b[0]);
            uint32_t stage = 0, phase = 0, n_issued = 0;
            bool ok = true;
            const uint32_t full0 = mapa(saddr(&S.full[0]), 0);
            // the first unit is the pair's own index; a launch with more units
            // than pairs hands out the others from the counter
            const int pairs = static_cast<int>(gridDim.x) / kPair;
            int t_next = static_cast<int>(blockIdx.x) / kPair;  // lane 0's counts
            const bool more = total > pairs;
            for (int k = 0; ok; ++k) {
                int t;
                if (rank == 0) {
                    const int slot = k % kTileRing;
                    const uint32_t ph = static_cast<uint32_t>(k / kTileRing) & 1u;
                    if (!__all_sync(kFullMask, mbar_wait<true>(&S.tile_empty[slot], ph ^ 1u, &g_ops_status))) {
                        ok = false;
                        break;
                    }
                    t = min(__shfl_sync(kFullMask, t_next, 0), total);
                    if (lane == 0) {
                        if (t < total) t_next = more ? pairs + atomicAdd(L.counter, 1) : total;
#pragma unroll
                        for (int c = 0; c < kPair; ++c)
                            send_u32(mapa(saddr(&S.tile_slot[slot]), c), t, mapa(saddr(&S.tile_full[slot]), c));
                    }
                    __syncwarp();
                } else {
                    // every unit in turn, the first too: slot 0's barrier must be past
                    // its first phase before unit kTileRing is looked for there, where
                    // the parity of the second reads as complete until then
                    t = wait_tile(S.tile_full, S.tile_slot, k, &g_ops_status, total);
                    t = __shfl_sync(kFullMask, t, 0);
                    if (lane == 0) release_tile(S.tile_empty, k);
                    __syncwarp();
                }
                if (t >= total) {
                    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
                    break;
                }
                const Unit u = decode_unit(L, t);
                const OpsProblem& P = L.p[u.p];
                const int slabs = P.slabs;
                const bool a_mn = P.a_mn != 0, b_mn = P.b_mn != 0;
                const int a_row = (2 * u.tm + rank) * BM;
                const int half_n = P.bn / 2;  // this CTA's columns of B
                const int b_col = P.dual ? u.tn * half_n : u.tn * P.bn + rank * half_n;
                const uint32_t tx = 128 * (P.a_rows[0] + P.a_rows[1] + P.bn);
                const uint32_t e_a = P.a_rows[rank] > 0 ? e : 0u, e_b2 = half_n > 64 ? e : 0u;
                const uint32_t e_tx = rank == 0 ? e : 0u;
                int seg = u.kb0 / slabs, within = (u.kb0 - seg * slabs) * SLAB_K;
                const int seg_end = slabs * SLAB_K;
                const CUtensorMap *ma = nullptr, *mb = nullptr;
                int pa = 0, pb = 0;
                bool fresh = true;
                for (int kb = u.kb0; kb < u.kb1; ++kb) {
                    if (fresh) {
                        const uint32_t sg = P.seg[seg];
                        const int src = sg & 15;
                        ma = &P.a[src];
                        mb = &P.b[P.dual ? rank : src];
                        pa = (sg >> 4) & 15;
                        pb = sg >> 8;
                        fresh = false;
                    }
                    if (!__all_sync(kFullMask, mbar_wait<false>(&S.empty[stage], phase ^ 1, &g_ops_status))) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx_if(e_tx, &S.full[stage], tx);
                    ++n_issued;
                    const uint32_t fb = full0 + stage * static_cast<uint32_t>(sizeof(uint64_t));
                    const uint32_t da = sa + stage * OP_BYTES, db = sb + stage * OP_BYTES;
                    if (!a_mn) {
                        tma_load_3d_pair(e_a, da, ma, fb, within, a_row, pa);
                    } else {
                        tma_load_3d_pair(e, da, ma, fb, a_row, within, pa);
                        tma_load_3d_pair(e, da + MN_BOX_BYTES, ma, fb, a_row + 64, within, pa);
                    }
                    if (!b_mn) {
                        tma_load_3d_pair(e, db, mb, fb, within, b_col, pb);
                    } else {
                        tma_load_3d_pair(e, db, mb, fb, b_col, within, pb);
                        tma_load_3d_pair(e_b2, db + MN_BOX_BYTES, mb, fb, b_col + 64, within, pb);
                    }
                    within += SLAB_K;
                    if (within == seg_end) {
                        within = 0;
                        ++seg;
                        fresh = true;
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) {
                // let copies already issued land before the CTA can exit
                if (rank == 0)
                    for (uint32_t j = 1; j <= STAGES && j <= n_issued; ++j) {
                        const uint32_t q = n_issued - j;
                        mbar_wait<false>(&S.full[q % STAGES], (q / STAGES) & 1u, &g_ops_status);
                    }
            } else {
                // the MMA's releases of the last ring round: no commit is still
                // in flight towards this CTA when the pair leaves
                for (int i = 0; i < STAGES && ok; ++i) {
                    ok = __all_sync(kFullMask, mbar_wait<true>(&S.empty[stage], phase ^ 1, &g_ops_status));
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------ MMA issuer (leader)
            const uint32_t e = elect_one();
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            const uint32_t empty0 = saddr(&S.empty[0]), acc0 = saddr(&S.acc_full[0]);
            const uint64_t a_k = smem_desc(saddr(S.a[0]), 0, 1024), a_m = smem_desc(saddr(S.a[0]), MN_BOX_BYTES, 1024);
            const uint64_t b_k = smem_desc(saddr(S.b[0]), 0, 1024), b_m = smem_desc(saddr(S.b[0]), MN_BOX_BYTES, 1024);
            constexpr uint64_t step_k = (UMMA_K * 2) >> 4, step_mn = (UMMA_K * 128) >> 4;
            int it = 0;
            for (int k = 0; ok; ++k) {
                const int t = __shfl_sync(
                    kFullMask, wait_tile(S.tile_full, S.tile_slot, k, &g_ops_status, total), 0);
                if (lane == 0) release_tile(S.tile_empty, k);
                __syncwarp();
                if (t >= total) break;
                const Unit u = decode_unit(L, t);
                const bool a_mn = L.p[u.p].a_mn != 0, b_mn = L.p[u.p].b_mn != 0;
                const uint32_t idesc = make_idesc(a_mn, b_mn, L.p[u.p].bn);
                const uint64_t a0 = a_mn ? a_m : a_k, b0 = b_mn ? b_m : b_k;
                const uint64_t a_step = a_mn ? step_mn : step_k, b_step = b_mn ? step_mn : step_k;
                // one accumulator per chain of MMAs: the unit's whole K range, or
                // (register sums) L.chain slabs of it
                for (int c0 = u.kb0; ok && c0 < u.kb1; ++it) {
                    const int c1 = kRegs && c0 + L.chain < u.kb1 ? c0 + L.chain : u.kb1;
                    const int buf = it & 1;
                    const uint32_t use = static_cast<uint32_t>(it >> 1);
                    if (!__all_sync(kFullMask, mbar_wait<true>(&S.acc_empty[buf], (use & 1) ^ 1, &g_ops_status))) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(buf * BN);
                    for (int kb = c0; kb < c1; ++kb) {
                        if (!__all_sync(kFullMask, mbar_wait<false>(&S.full[stage], phase, &g_ops_status))) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint64_t ad = a0 + static_cast<uint64_t>(stage) * (OP_BYTES >> 4);
                        const uint64_t bd = b0 + static_cast<uint64_t>(stage) * (OP_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < SLAB_K / UMMA_K; ++kk)
                            umma_bf16_pair(e, d, ad + kk * a_step, bd + kk * b_step, idesc, (kb != c0 || kk) ? 1u : 0u);
                        umma_commit_pair(e, empty0 + stage * static_cast<uint32_t>(sizeof(uint64_t)), kPairMask);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    // also on failure: covers every MMA issued so far
                    umma_commit_pair(e, acc0 + buf * static_cast<uint32_t>(sizeof(uint64_t)), kPairMask);
                    c0 = c1;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // ------------------------------------------------ epilogue
        const int q = warp & 3;                   // TMEM lane quarter this warp may access
        const int half = (warp - kEpiWarp0) / 4;  // column half
        float* stg = S.stage[warp - kEpiWarp0];
        int it = 0;
        float r[kRegs ? BN / 2 : 1];
        for (int k = 0;; ++k) {
            const int t = wait_tile(S.tile_full, S.tile_slot, k, &g_ops_status, total);
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa(saddr(&S.tile_empty[k % kTileRing]), 0));
            if (t >= total) break;
            const Unit u = decode_unit(L, t);
            const OpsProblem& P = L.p[u.p];
            const int r0 = (2 * u.tm + rank) * BM + q * 32;
            // false: this warp's rows or columns lie outside the matrix
            const int bn = kKind == OPS_LOGITS ? BN : P.bn;
            const int c_first = first_col<kKind>(bn, u.tn, half);
            bool active = r0 < P.M && c_first < P.N;
            uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
            const int buf = it & 1;
            if (kKind == OPS_DGATE && u.part == 0 && r0 + lane < P.M) {
                // this warp's share of the stored act and slope into L2, a
                // mainloop ahead of their use
#pragma unroll 1
                for (int o = 0; o < 2; ++o) {
                    const int es = P.in[o].type == ELEM_BF16 ? 2 : 4;
                    const char* row = static_cast<const char*>(P.in[o].p) + (r0 + lane) * P.in[o].ld * es;
                    for (int c = c_first; c < min(c_first + bn / 2, P.N); c += 128 / es)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(row + c * es)));
                }
            }
            if constexpr (kRegs) {
                // add the chains up; each accumulator goes back to the MMAs
                // before anything is done with the sum
#pragma unroll
                for (int j = 0; j < BN / 2; ++j) r[j] = 0.0f;
                for (int c0 = u.kb0; c0 < u.kb1; c0 += L.chain, ++it) {
                    const bool ready = mbar_wait<true>(&S.acc_full[it & 1], (it >> 1) & 1, &g_ops_status);
                    fence_after();
                    active = active && ready;
                    if (active) {
                        const uint32_t base = taddr + static_cast<uint32_t>((it & 1) * BN);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if (!chunk_in<kKind>(bn, 2 * b)) continue;
                            float v[32];
                            __syncwarp();
                            tmem_ld32(base + static_cast<uint32_t>(chunk_col<kKind>(bn, half, 2 * b)), v);
#pragma unroll
                            for (int j = 0; j < 32; ++j) r[b * 32 + j] += v[j];
                        }
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(mapa(saddr(&S.acc_empty[it & 1]), 0));
                }
            } else {
                const bool ready = mbar_wait<true>(&S.acc_full[buf], (it >> 1) & 1, &g_ops_status);
                fence_after();
                active = active && ready;
                taddr += static_cast<uint32_t>(buf * BN);
                ++it;
            }
            const auto finish = [&](auto acc) {
                if constexpr (kKind == OPS_STORE || kKind == OPS_STORE_SCALED)
                    epi_store<kKind == OPS_STORE_SCALED>(P, L.scale, acc, u, half, r0, lane, stg);
                else if constexpr (kKind == OPS_GATE) epi_gate<kF32>(P, acc, u, half, r0, lane, stg);
                else if constexpr (kKind == OPS_DGATE) epi_dgate<kF32>(P, acc, u, half, r0, lane, stg);
                else epi_logits<kF32>(P, u, half, r0, lane, acc.r, stg);
            };
            if (active && u.split == 1) {
                if constexpr (kRegs) finish(RegSrc{r});
                else finish(TmemSrc<kKind>{taddr, bn, half});
            } else if (active) {
                // store this unit's partial sum [column][row]; the last unit of
                // the tile adds them all up, in K order
                float* slot = L.partials + static_cast<int64_t>(u.slot) * kOpsSlotFloats +
                              static_cast<int64_t>(rank) * BN * BM + q * 32;
                const auto inside = [&](int ci, int tcol) {
                    return chunk_in<kKind>(bn, ci) &&
                           (kKind == OPS_GATE ? u.tn * (bn / 2) + tcol % (bn / 2) : u.tn * bn + tcol) < P.N;
                };
                constexpr int kUnroll = kRegs ? 8 : 1;
#pragma unroll kUnroll
                for (int ci = 0; ci < 8; ++ci) {
                    const int tcol = chunk_col<kKind>(bn, half, ci);
                    if (!inside(ci, tcol)) continue;
                    float v[CH];
                    if constexpr (kRegs) {
#pragma unroll
                        for (int j = 0; j < CH; ++j) v[j] = r[ci * CH + j];
                    } else {
                        TmemSrc<kKind>{taddr, bn, half}.load(ci, v);
                    }
                    float* p = slot + static_cast<int64_t>(u.part) * kOpsSlotFloats + static_cast<int64_t>(tcol) * BM +
                               lane;
#pragma unroll
                    for (int j = 0; j < CH; ++j) __stcg(p + j * BM, v[j]);
                }
                __threadfence();
                __syncwarp();
                int before = 0;
                if (lane == 0)
                    before = atomicAdd(&L.tail_count[u.tail * kOpsTailCounts + rank * kEpiWarps + (warp - kEpiWarp0)],
                                       1);
                before = __shfl_sync(kFullMask, before, 0);
                if (before == u.split - 1) {
                    __threadfence();
                    float sum[BN / 2];
#pragma unroll
                    for (int j = 0; j < BN / 2; ++j) sum[j] = 0.0f;
#pragma unroll 1
                    for (int i = 0; i < u.split; ++i) {
                        const float* p = slot + i * kOpsSlotFloats + lane;
#pragma unroll
                        for (int ci = 0; ci < 8; ++ci) {
                            const int tcol = chunk_col<kKind>(bn, half, ci);
                            if (inside(ci, tcol)) {
#pragma unroll
                                for (int j = 0; j < CH; ++j) sum[ci * CH + j] += __ldcg(p + (tcol + j) * BM);
                            }
                        }
                    }
                    finish(RegSrc{sum});
                }
            }
            if constexpr (!kRegs) {
                // every tcgen05.ld of the accumulator has completed (wait::ld):
                // the release is relaxed, so it does not wait for this warp's
                // stores
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(mapa(saddr(&S.acc_empty[buf]), 0));
            }
        }
    }

    fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

using Kernel = void (*)(OpsLaunch);

Kernel kernel_of(int32_t kind, bool f32) {
    switch (kind) {
        case OPS_STORE: return f32 ? ops_gemm_kernel<OPS_STORE, true> : ops_gemm_kernel<OPS_STORE, false>;
        case OPS_GATE: return f32 ? ops_gemm_kernel<OPS_GATE, true> : ops_gemm_kernel<OPS_GATE, false>;
        case OPS_STORE_SCALED:
            return f32 ? ops_gemm_kernel<OPS_STORE_SCALED, true> : ops_gemm_kernel<OPS_STORE_SCALED, false>;
        case OPS_DGATE: return f32 ? ops_gemm_kernel<OPS_DGATE, true> : ops_gemm_kernel<OPS_DGATE, false>;
        default: return f32 ? ops_gemm_kernel<OPS_LOGITS, true> : ops_gemm_kernel<OPS_LOGITS, false>;
    }
}

constexpr size_t kSmemBytes = sizeof(Smem) + 1024;

}  // namespace

cudaError_t ops_pairs(int* pairs) {
    static PerDevice cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // shared-memory attribute of every instance and the resident pairs, once
    // per device with that device current
    return cache.get(dev, pairs, [&](int* out) {
        cudaError_t r = cudaSuccess;
        for (int kind = 0; kind < kOpsKinds && r == cudaSuccess; ++kind)
            for (int f = 0; f < 2 && r == cudaSuccess; ++f)
                r = cudaFuncSetAttribute(kernel_of(kind, f != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
        if (r != cudaSuccess) return r;
        int sms = 0;
        r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (r != cudaSuccess) return r;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kPair;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(sms / kPair * kPair);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        r = cudaOccupancyMaxActiveClusters(&n, kernel_of(OPS_STORE, false), &cfg);
        if (r != cudaSuccess) return r;
        *out = n > 0 ? n : sms / kPair;
        return cudaSuccess;
    });
}

// Work units.  Whole tiles are split into S ranges of K where that shortens the
// launch.  The estimate, in 64-deep slabs of a 256 x 256 tile (about 0.3 us each), is
// measured on tiles of a few hundred tokens: a unit costs its slabs (0.65 of them
// with 128-column tiles) and kUnitCost, the epilogue kEpiCost per 256 columns; a
// unit of a split tile kStoreCost more (its partial sum's way to L2 and the
// arrival), and the tile's last unit kPartCost for each part it adds up.
//  - One product: T equal tiles on P pairs leave P - T mod P pairs idle in the
//    last round, so the tiles of that round are the ones split.
//  - Several products: the estimate is the larger of the work per pair and the
//    longest unit (which the caller places first); the product with the longest
//    unit is split further while that lowers it.
namespace {

constexpr double kUnitCost = 4.0, kEpiCost = 8.0, kStoreCost = 14.0, kPartCost = 12.0;
constexpr int kMinSlabs = 8, kMaxSplit = 32;

double slab_cost(int bn) { return bn == 256 ? 1.0 : 0.65; }

// The longest chain of a tile in s ranges of K, and its work.
double unit_cost(const OpsShape& p, int s) {
    return slab_cost(p.bn) * p.total / s + kUnitCost + kEpiCost * p.bn / 256 +
           (s > 1 ? kStoreCost + kPartCost * s : 0.0);
}
double tile_work(const OpsShape& p, int s) {
    return slab_cost(p.bn) * p.total + s * kUnitCost + kEpiCost * p.bn / 256 +
           (s > 1 ? s * kStoreCost + kPartCost * s : 0.0);
}

int64_t tiles_of(const OpsShape& p) {
    const int n = p.dual ? p.bn / 2 : p.bn;
    return (p.M + 255) / 256 * ((p.N + n - 1) / n);
}

// Ranges per split tile of each product and the tiles to split; the launch's estimate.
double plan_splits(const OpsShape* p, int n, int pairs, int* split, int64_t* rem) {
    for (int i = 0; i < n; ++i) {
        split[i] = 1;
        rem[i] = tiles_of(p[i]);
    }
    if (n == 1) {
        const int64_t tiles = rem[0];
        rem[0] %= pairs;
        double best = unit_cost(p[0], 1);
        for (int s = 2; s <= kMaxSplit && rem[0] > 0 && p[0].total / s >= kMinSlabs; ++s) {
            const int64_t rounds = (rem[0] * s + pairs - 1) / pairs;
            const double c = (rounds - 1) * (slab_cost(p[0].bn) * p[0].total / s + kUnitCost + kStoreCost) +
                             unit_cost(p[0], s);
            if (c < best) {
                best = c;
                split[0] = s;
            }
        }
        return static_cast<double>(tiles / pairs) * unit_cost(p[0], 1) + (rem[0] ? best : 0.0);
    }
    const auto estimate = [&](int* longest) {
        double work = 0.0, most = 0.0;
        for (int i = 0; i < n; ++i) {
            work += tile_work(p[i], split[i]) * static_cast<double>(tiles_of(p[i]));
            const double c = unit_cost(p[i], split[i]);
            if (c > most) {
                most = c;
                *longest = i;
            }
        }
        return work / pairs > most ? work / pairs : most;
    };
    int longest = 0;
    double best = estimate(&longest);
    for (;;) {
        const int k = longest, was = split[k];
        int s = was + 1, now = 0;
        double c = best;
        for (; s <= kMaxSplit && p[k].total / s >= kMinSlabs; ++s) {
            split[k] = s;
            c = estimate(&now);
            if (c < best) break;
        }
        if (!(c < best)) {
            split[k] = was;
            return best;
        }
        best = c;
        longest = now;
    }
}

}  // namespace

// Each product's columns per tile: every combination of 128 and 256 is estimated
// (at most 16).
void ops_tile_columns(OpsShape* p, int n, int pairs) {
    int split[kOpsMaxProblems], choice = 0;
    int64_t rem[kOpsMaxProblems];
    double best = 0.0;
    for (int c = 0; c < 1 << n; ++c) {
        for (int i = 0; i < n; ++i) p[i].bn = c >> i & 1 ? 128 : 256;
        const double e = plan_splits(p, n, pairs, split, rem);
        if (c == 0 || e < best) {
            best = e;
            choice = c;
        }
    }
    for (int i = 0; i < n; ++i) p[i].bn = choice >> i & 1 ? 128 : 256;
}

void ops_schedule(OpsLaunch& l, int pairs, int slots, int tails) {
    OpsShape shape[kOpsMaxProblems];
    int split[kOpsMaxProblems];
    int64_t rem[kOpsMaxProblems];
    for (int i = 0; i < l.n; ++i) {
        const OpsProblem& p = l.p[i];
        shape[i] = OpsShape{p.M, p.N, p.slabs * p.nseg, p.dual, p.bn};
    }
    if (l.n > 0) plan_splits(shape, l.n, pairs, split, rem);
    int unit = 0, tail = 0, slot = 0;
    for (int i = 0; i < l.n; ++i) {
        OpsProblem& p = l.p[i];
        const int tiles = p.tiles_m * p.tiles_n;
        int64_t r = rem[i];
        int s = split[i];
        while (s > 1 && r * s > slots - slot) --s;
        if (s <= 1 || r > tails - tail) {
            r = 0;
            s = 1;
        }
        p.whole = tiles - static_cast<int>(r);
        p.split = s;
        p.unit_begin = unit;
        p.tail_begin = tail;
        p.slot_begin = slot;
        unit += p.whole + static_cast<int>(r) * s;
        tail += static_cast<int>(r);
        slot += static_cast<int>(r) * s;
    }
    l.total_units = unit;
}

cudaError_t ops_status_word(void** p) { return cudaGetSymbolAddress(p, g_ops_status); }

cudaError_t launch_ops_gemm(const OpsLaunch& l, int32_t kind, bool f32, cudaStream_t s) {
    if (l.total_units <= 0) return cudaSuccess;
    int pairs = 0;
    const cudaError_t e = ops_pairs(&pairs);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPair;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((l.total_units < pairs ? l.total_units : pairs) * kPair);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel_of(kind, f32), l);
}

}  // namespace dmuon
