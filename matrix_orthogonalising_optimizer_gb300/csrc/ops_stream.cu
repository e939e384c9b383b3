// Products of a few rows with a weight matrix: generated tokens through the
// gated block, a handful of positions against the vocabulary.
//
// Bound by the read of the weights (2 bytes per weight, 2 FLOP per weight and
// row), so the kernel is built around loads in flight: a weight goes from HBM
// straight to the registers that feed the tensor cores, without shared memory,
// and is read once for all rows.  A block holds 16 MT weight rows (for the gated
// block 8 MT of each projection, so a gate and its up value meet in one
// thread); its eight warps take 32-column pieces of K in turn -- 512 contiguous
// bytes per row and round -- and add up their sums in shared memory.  When there
// are few weight rows, K is also shared by a cluster of up to 8 blocks, whose
// leader adds their sums through distributed shared memory; the order is fixed.
//
// mma.sync.m16n8k16 with K permuted: a thread's 16-byte load holds 8 consecutive
// k of its row, of which elements (0,1), (2,3) serve one MMA and (4,5), (6,7)
// the next as the fragment's two column pairs.  The sum over k does not depend
// on which k sits in which slot as long as weights and x agree, and both are
// loaded alike.  The tcgen05 kernel needs the weights in shared memory and waits
// for whole tiles: at one row of 4096 x 14336 it took 125 us, this one 56 (352 MB
// at 6.3 TB/s, 94 % of the copy rate).
#include <cuda_bf16.h>

#include "act.cuh"
#include "ops.h"
#include "tc.cuh"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Per instance, by n8 tiles of x rows (1: up to 8 rows, 2: 16, 3: 24, 4: 32):
// 16-row weight tiles of a warp, K pieces loaded at a time, resident blocks per
// SM, whether x is loaded a piece ahead, and the blocks per SM below which K is
// shared by a cluster.  Measured at 4096 x 14336 (block) and 4096 x 131072 (loss):
// one row 56 and 156 us, 16, 24 and 32 rows of the block 60, 64 and 74; deeper
// unrolling, more residents or wider clusters each lost 4 to 50 %.  Above 16 rows
// the x rows come from L2 as often as the weights (9.6 TB/s together), and their
// latency was the bound before they were loaded ahead (24 rows 87, 32 rows 88 us);
// up to 16 rows the registers are better spent on weights in flight (16 rows 60
// us, 61 with x ahead).
__host__ __device__ constexpr int kTiles(int nt) { return nt == 1 ? 1 : 2; }
__host__ __device__ constexpr int kUnroll(int nt) { return nt > 2 ? 2 : nt + 1; }
__host__ __device__ constexpr int kResident(int nt) { return nt == 1 ? 4 : 2; }
__host__ __device__ constexpr bool kAhead(int nt) { return nt > 2; }
constexpr int kSpread(int nt) { return nt == 1 ? 2 : 1; }

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(reinterpret_cast<uint64_t>(p)));
    return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void st1(const OpsMat& m, int64_t r, int64_t c, float v) {
    if (m.type == ELEM_BF16) static_cast<__nv_bfloat16*>(m.p)[r * m.ld + c] = __float2bfloat16_rn(v);
    else static_cast<float*>(m.p)[r * m.ld + c] = v;
}

// The end of a block: the warps' sums part[k][token * R + row] (every thread has
// passed a barrier after writing them), the cluster's, and the element-wise part.
// Rows tok0 .. tok0 + T - 1 of x, output columns n0 ..; for the gated block a
// gate's up value is UP rows further on.
template <int kKind, bool kF32, int R, int T, int UP, int kParts>
__device__ __forceinline__ void finish(const OpsStream& P, float (&part)[kParts][R * T], float (&sum)[R * T], int tile,
                                       int n0, int tok0, uint32_t rank, uint32_t cluster) {
    for (int i = threadIdx.x; i < R * T; i += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) s += part[k][i];
        sum[i] = s;
    }
    if (cluster > 1) {
        tc::cluster_sync();
        if (rank == 0) {
            for (int i = threadIdx.x; i < R * T; i += kThreads) {
                float s = sum[i];
                for (uint32_t k = 1; k < cluster; ++k) {
                    float v;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(v)
                                 : "r"(tc::mapa(tc::saddr(&sum[i]), k))
                                 : "memory");
                    s += v;
                }
                part[0][i] = s;
            }
        }
        tc::cluster_sync();  // the leader has read the others' shared memory
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    const float* v = cluster > 1 ? part[0] : sum;
    if constexpr (kKind == OPS_STORE) {
        for (int i = threadIdx.x; i < R * T; i += kThreads) {
            const int tok = tok0 + i / R, n = n0 + i % R;
            if (tok < P.tokens && n < P.N) st1(P.out[0], tok, n, v[i]);
        }
    } else if constexpr (kKind == OPS_GATE) {
        for (int i = threadIdx.x; i < R * T / 2; i += kThreads) {
            const int tok = tok0 + i / (R / 2), j = i % (R / 2), n = n0 + j;
            const int at = i / (R / 2) * R + 2 * UP * (j / UP) + j % UP;
            if (tok >= P.tokens || n >= P.N) continue;
            const float a = v[at], u = v[at + UP];
            const float gate = act_gate<kF32>(P.act, a), f = a * gate;
            if (P.out[1].p) {
                st1(P.out[1], tok, n, f);
                st1(P.out[2], tok, n, u * act_slope<kF32>(P.act, a, gate));
                if (P.out[3].p) st1(P.out[3], tok, n, f * u);
            }
            st1(P.out[0], tok, n, f * u);
        }
    } else {
        // R lanes per token: maximum and sum of exponentials of the block's columns
        const float ninf = __int_as_float(0xff800000);
        for (int i = threadIdx.x; i < R * T; i += kThreads) {
            const int tok = tok0 + i / R, n = n0 + i % R;
            const float z = n < P.N ? v[i] : ninf;
            float m = z;
#pragma unroll
            for (int o = R / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(tc::kFullMask, m, o));
            const float ms = exp_shift(m), e = kF32 ? expf(z - ms) : ex2((z - ms) * kLog2e);
            float s = e;
#pragma unroll
            for (int o = R / 2; o; o >>= 1) s += __shfl_xor_sync(tc::kFullMask, s, o);
            if (tok >= P.tokens || n >= P.N) continue;
            if (P.targets[tok] == n) P.target_logit[tok] = z;
            if (P.out[0].p) {
                const int64_t at = tok * P.out[0].ld + n;
                if constexpr (kF32) static_cast<float*>(P.out[0].p)[at] = e;
                else static_cast<uint16_t*>(P.out[0].p)[at] = static_cast<uint16_t>(e16_encode(e));
            }
            if (i % R == 0) P.stats[static_cast<int64_t>(tok) * P.nblk + tile] = make_float2(m, s);
        }
    }
}

template <int kKind, int NT, int MT>
__global__ void __launch_bounds__(kThreads, kResident(NT)) ops_stream_kernel(const __grid_constant__ OpsStream P) {
    constexpr int R = 16 * MT, T = 8 * NT;     // weight rows, x rows of the block's result
    constexpr int U = kUnroll(NT);         // K pieces loaded at a time
    // the warps' sums [token][row]; large results in two rounds of four warps
    constexpr int kParts = R * T > 1024 ? kWarps / 2 : kWarps;
    __shared__ float part[kParts][R * T];
    __shared__ float sum[R * T];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    uint32_t rank, cluster;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cluster));
    const int tile = blockIdx.x / cluster;
    const int n0 = tile * (kKind == OPS_GATE ? R / 2 : R);  // first output column

    // this thread's weight rows: g and g + 8 of every 16-row tile (rows past the
    // matrix read its last row and are dropped at the end)
    const __nv_bfloat16* wp[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = kKind == OPS_GATE ? n0 + 8 * m + g : n0 + 16 * m + 8 * h + g;
            wp[m][h] = static_cast<const __nv_bfloat16*>(P.w[kKind == OPS_GATE ? h : 0]) +
                       static_cast<int64_t>(min(n, P.N - 1)) * P.ldw + 8 * t;
        }
    const __nv_bfloat16* xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        xp[n] = static_cast<const __nv_bfloat16*>(P.x) +
                static_cast<int64_t>(min(8 * n + g, P.tokens - 1)) * P.ldx + 8 * t;

    // K pieces of 32: the cluster's blocks take contiguous shares, a block's
    // warps every eighth piece of its share
    const int pieces = (P.K + 31) / 32;
    const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * rank / cluster);
    const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (rank + 1) / cluster);
    float c[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[m][n][i] = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // pieces of 32 k; pieces past p1 are zero
    uint4 w[U][MT][2], x[kAhead(NT) ? 2 : U][NT];
    const auto load_w = [&](int p, int u) {
        const int k = p * 32;
        const bool in = p < p1 && k + 8 * t < P.K;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[u][m][h] = in ? ld_stream(wp[m][h] + k) : zero;
    };
    const auto load_x = [&](int p, int i) {
        const int k = p * 32;
        const bool in = p < p1 && k + 8 * t < P.K;
#pragma unroll
        for (int n = 0; n < NT; ++n) x[i][n] = in ? *reinterpret_cast<const uint4*>(xp[n] + k) : zero;
    };
    const auto multiply = [&](int u, int i) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma(c[m][n], w[u][m][0].x, w[u][m][1].x, w[u][m][0].y, w[u][m][1].y, x[i][n].x, x[i][n].y);
                mma(c[m][n], w[u][m][0].z, w[u][m][1].z, w[u][m][0].w, w[u][m][1].w, x[i][n].z, x[i][n].w);
            }
    };
    const auto load_round = [&](int p) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_w(p + u * kWarps, u);
    };
    // programmatic dependent launch: after the library's own kernel the weights
    // may be read before that kernel has finished (it waited for everything
    // before it, and writes no weights); x and all outputs wait
    if (P.after) load_round(p0 + warp);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!P.after) load_round(p0 + warp);
    if constexpr (kAhead(NT)) {
        // each piece of the weights is replaced by the one U ahead as soon as it
        // is used, each piece of x by the next but one
        load_x(p0 + warp, 0);
        for (int p = p0 + warp; p < p1; p += U * kWarps) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                load_x(p + (u + 1) * kWarps, (u + 1) & 1);
                multiply(u, u & 1);
                load_w(p + (u + U) * kWarps, u);
            }
        }
    } else {
        for (int p = p0 + warp; p < p1; p += U * kWarps) {
#pragma unroll
            for (int u = 0; u < U; ++u) load_x(p + u * kWarps, u);
#pragma unroll
            for (int u = 0; u < U; ++u) multiply(u, u);
            if (p + U * kWarps < p1) load_round(p + U * kWarps);
        }
    }
#pragma unroll
    for (int round = 0; round < kWarps / kParts; ++round) {
        if (warp / kParts == round) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& p = part[warp % kParts][(8 * n + 2 * t + (i & 1)) * R + 16 * m + 8 * (i >> 1) + g];
                        p = round ? p + c[m][n][i] : c[m][n][i];
                    }
        }
        __syncthreads();
    }
    finish<kKind, false, R, T, 8, kParts>(P, part, sum, tile, n0, 0, rank, cluster);
}

// fp32: the same stream with FFMA (the tensor cores would need the weights in
// bf16 parts: a packed copy costs four times their read).  A warp holds R = 8
// weight rows (gated block: 4 of each projection) and T = 8 rows of x; a lane
// loads four consecutive k of each, and the 64 sums are reduced over the lanes
// at the end by halving.  More rows of x take further blocks that find the
// weights in L2.
constexpr int kF32Rows = 8;

template <int kKind>
__global__ void __launch_bounds__(kThreads, 2) ops_stream_f32_kernel(const __grid_constant__ OpsStream P) {
    constexpr int R = kF32Rows, T = 8, UP = R / 2;
    __shared__ float part[kWarps][R * T];
    __shared__ float sum[R * T];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint32_t rank, cluster;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cluster));
    const int groups = (P.tokens + T - 1) / T;
    const int tile = blockIdx.x / cluster / groups, tok0 = blockIdx.x / cluster % groups * T;
    const int n0 = tile * (kKind == OPS_GATE ? R / 2 : R);
    const float* wp[R];
    const float* xp[T];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = kKind == OPS_GATE ? n0 + r % UP : n0 + r;
        wp[r] = static_cast<const float*>(P.w[kKind == OPS_GATE ? r / UP : 0]) +
                static_cast<int64_t>(min(n, P.N - 1)) * P.ldw + 4 * lane;
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
        xp[t] = static_cast<const float*>(P.x) + static_cast<int64_t>(min(tok0 + t, P.tokens - 1)) * P.ldx + 4 * lane;
    const int pieces = (P.K + 127) / 128;
    const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * rank / cluster);
    const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (rank + 1) / cluster);
    float acc[T * R];
#pragma unroll
    for (int i = 0; i < T * R; ++i) acc[i] = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 w[R];
    const auto load_w = [&](int p) {
        const bool in = p < p1 && p * 128 + 4 * lane < P.K;
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = in ? ld_stream(wp[r] + p * 128) : zero;
    };
    if (P.after) load_w(p0 + warp);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!P.after) load_w(p0 + warp);
    for (int p = p0 + warp; p < p1; p += kWarps) {
        const bool in = p * 128 + 4 * lane < P.K;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (in) x = *reinterpret_cast<const float4*>(xp[t] + p * 128);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float& s = acc[t * R + r];
                s = fmaf(__uint_as_float(w[r].x), x.x, s);
                s = fmaf(__uint_as_float(w[r].y), x.y, s);
                s = fmaf(__uint_as_float(w[r].z), x.z, s);
                s = fmaf(__uint_as_float(w[r].w), x.w, s);
            }
        }
        load_w(p + kWarps);
    }
    // reduce-scatter over the lanes: each step halves the sums a lane holds
#pragma unroll
    for (int o = 16, n = T * R / 2; o; o >>= 1, n >>= 1) {
        const bool hi = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = hi ? acc[i] : acc[i + n];
            const float keep = hi ? acc[i + n] : acc[i];
            acc[i] = keep + __shfl_xor_sync(tc::kFullMask, send, o);
        }
    }
    const int at = (lane >> 4 & 1) * 32 + (lane >> 3 & 1) * 16 + (lane >> 2 & 1) * 8 + (lane >> 1 & 1) * 4 +
                   (lane & 1) * 2;
    part[warp][at] = acc[0];
    part[warp][at + 1] = acc[1];
    __syncthreads();
    finish<kKind, true, R, T, UP, kWarps>(P, part, sum, tile, n0, tok0, rank, cluster);
}

using Kernel = void (*)(OpsStream);

template <int kKind>
Kernel pick(int tokens, bool f32) {
    if (f32) return ops_stream_f32_kernel<kKind>;
    if constexpr (kKind != OPS_LOGITS) {  // at most kStreamLossTokens rows
        if (tokens > 24) return ops_stream_kernel<kKind, 4, kTiles(4)>;
        if (tokens > 16) return ops_stream_kernel<kKind, 3, kTiles(3)>;
        if (tokens > 8) return ops_stream_kernel<kKind, 2, kTiles(2)>;
    }
    return ops_stream_kernel<kKind, 1, kTiles(1)>;
}

}  // namespace

int ops_stream_block(int64_t tokens, bool f32) {
    if (f32) return kF32Rows;
    return 16 * kTiles(tokens <= 8 ? 1 : tokens <= 16 ? 2 : 4);
}

cudaError_t launch_ops_stream(const OpsStream& a, int32_t kind, bool f32, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static PerDevice count;
    e = count.get(dev, &sms,
                  [&](int* out) { return cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev); });
    if (e != cudaSuccess) return e;
    const int rows = ops_stream_block(a.tokens, f32) / (kind == OPS_GATE ? 2 : 1);
    const int tiles = (a.N + rows - 1) / rows * (f32 ? (a.tokens + 7) / 8 : 1);
    // a block keeps at least two rounds of its eight warps
    const int spread = f32 ? 2 : kSpread(a.tokens <= 8 ? 1 : 2), piece = f32 ? 128 : 32;
    int cluster = 1;
    while (cluster < 8 && tiles * cluster < spread * sms && a.K / (cluster * 2) >= 2 * piece * kWarps) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(tiles * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const Kernel k = kind == OPS_GATE     ? pick<OPS_GATE>(a.tokens, f32)
                     : kind == OPS_LOGITS ? pick<OPS_LOGITS>(a.tokens, f32)
                                          : pick<OPS_STORE>(a.tokens, f32);
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace dmuon
