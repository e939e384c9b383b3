// Layer norm, forward and backward, with the reduction of the weight's and the
// bias's gradient over the rows.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), n = (x - mu) r
//   y  = n w + b
//   g  = dy w;  dx = r (g - mean(g) - n mean(g n));  dw = sum dy n, db = sum dy
//
// HBM-bound: forward 4 bytes per bf16 element (read x, write y), backward 6
// (read x and dy, write dx), twice that in fp32.  Each row is read once and
// held in registers by the threads of its group (WPR warps, VPT 16-byte vectors
// per thread), so the variance is the mean of squared deviations from the
// finished mean -- no difference of large sums.  All arithmetic is fp32, one
// rounding per stored value.
//
// Aligned rows, unless they are few and short (ring kernels): persistent groups; bulk asynchronous copies
// bring each group's next rows into a shared-memory ring while it works on the
// current one, so the loads in flight do not cost registers, and the arithmetic
// runs on packed pairs (fma.rn.f32x2).  Few rows, or rows that do not start on
// 16 bytes (register kernels): a row is spread over as many threads as hold it
// and the next row is loaded into registers ahead.
//
// In the backward pass a thread meets the same columns in every row and keeps
// their dw and db sums in registers; a block's groups add theirs up in shared
// memory, each block writes one partial row, and a second kernel adds the
// partial rows in a fixed order, so the result does not depend on scheduling.
// Rows wider than a group holds (16384 bf16 or 8192 fp32 columns) take three plain
// passes (wide kernels).
//
// Measured at 16384 x 4096 in bf16: forward 49 us (268 MB at 5.5 TB/s, 82 % of the
// copy rate; launch and first rows are about 5 us of it), backward 73 us with the
// reduction (403 MB at 5.5 TB/s).  Before the rings and the packed arithmetic:
// 52 and 122 us, 14 and 40 instructions per element.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "dmuon.h"
#include "ops.h"
#include "tc.cuh"

namespace {

// set by a wait that gave up; read and cleared by dmuon_ops_status
__device__ int32_t g_norm_status = 0;

constexpr unsigned kFull = 0xffffffffu;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kBwdThreads = 512;
constexpr int kMaxPartials = 1024;  // partial rows of the backward pass
__host__ __device__ constexpr int bwd_groups(int wpr) { return kBwdThreads / (32 * wpr); }

struct NormArgs {
    const void* x;
    const void* dy;
    const void* w;
    const void* b;
    void* out;          // y or dx
    float* mean;
    float* rstd;
    float* partial;     // backward: [blocks][2][cols]
    int64_t rows;
    int32_t cols;
    int32_t aligned;    // rows start on 16-byte boundaries
    float eps;
    int32_t stages;     // ring kernels: rows in a group's ring
};

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ float to_f(T v) {
    return static_cast<float>(v);
}

template <typename T>
__device__ __forceinline__ T from_f(float v) {
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
    else return v;
}

// 16 bytes from column c of a row; columns >= cols read as zero.
template <typename T>
__device__ __forceinline__ uint4 ld_raw(const T* row, int c, int cols, bool aligned) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (c >= cols) return q;
    if (aligned) return *reinterpret_cast<const uint4*>(row + c);
    T t[kVec<T>];
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) t[j] = c + j < cols ? row[c + j] : from_f<T>(0.0f);
    if constexpr (sizeof(T) == 4) {
        q = make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]), __float_as_uint(t[3]));
    } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(t);
        q = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    return q;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[kVec<T>]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ void st_vec(T* row, int c, int cols, bool aligned, const float (&v)[kVec<T>]) {
    if (c >= cols) return;
    if (aligned) {
        uint4 q;
        if constexpr (sizeof(T) == 4) {
            q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else {
            __nv_bfloat162 h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            q = *reinterpret_cast<const uint4*>(h);
        }
        *reinterpret_cast<uint4*>(row + c) = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
        if (c + j < cols) row[c + j] = from_f<T>(v[j]);
}

template <int N>
__device__ __forceinline__ void warp_sum(float (&s)[N]) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(kFull, s[k], o);
}

// Sum over the WPR warps of a row group, in a fixed order.  `red` alternates
// between two buffers from call to call, so one barrier per reduction is enough:
// a buffer is written again only after the barrier of the reduction in between.
// Every thread reads all warps' sums, 16 bytes at a time.
template <int WPR, int N>
struct alignas(16) GroupRed {
    float v[N][WPR < 4 ? 4 : WPR];
};

template <int WPR, int N>
__device__ __forceinline__ void group_sum(float (&s)[N], GroupRed<WPR, N>& red, int bar) {
    warp_sum(s);
    if constexpr (WPR > 1) {
        const int w = (threadIdx.x / 32) % WPR;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) red.v[k][w] = s[k];
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(WPR * 32) : "memory");
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (WPR == 2) {
                s[k] = red.v[k][0] + red.v[k][1];
            } else {
                s[k] = 0.0f;
#pragma unroll
                for (int i = 0; i < WPR; i += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(&red.v[k][i]);
                    s[k] += (q.x + q.y) + (q.z + q.w);
                }
            }
        }
    }
}

template <typename T, int VPT, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32) norm_fwd_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>, TPR = WPR * 32, G = WPR == 1 ? 4 : 1;
    __shared__ GroupRed<WPR, 1> red[2];
    const int g = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    const bool al = a.aligned != 0;
    uint4 w[VPT], b[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = (k * TPR + tr) * V;
        w[k] = a.w ? ld_raw(static_cast<const T*>(a.w), c, a.cols, al) : make_uint4(0, 0, 0, 0);
        b[k] = a.b ? ld_raw(static_cast<const T*>(a.b), c, a.cols, al) : make_uint4(0, 0, 0, 0);
    }
    const float inv = 1.0f / static_cast<float>(a.cols);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
    int64_t row = static_cast<int64_t>(blockIdx.x) * G + g;
    uint4 next[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        if (row < a.rows)
            next[k] = ld_raw(static_cast<const T*>(a.x) + row * a.cols, (k * TPR + tr) * V, a.cols, al);
    for (; row < a.rows; row += stride) {
        float x[VPT][V];
#pragma unroll
        for (int k = 0; k < VPT; ++k) unpack<T>(next[k], x[k]);
        if (row + stride < a.rows) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                next[k] = ld_raw(static_cast<const T*>(a.x) + (row + stride) * a.cols, (k * TPR + tr) * V, a.cols, al);
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] += x[k][j];
        group_sum<WPR>(s, red[0], 1 + g);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[k][j] -= mean;
                if (c + j < a.cols) s[0] = fmaf(x[k][j], x[k][j], s[0]);
            }
        }
        group_sum<WPR>(s, red[1], 1 + g);
        const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
        if (tr == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float wv[V], bv[V];
            unpack<T>(w[k], wv);
            unpack<T>(b[k], bv);
#pragma unroll
            for (int j = 0; j < V; ++j) x[k][j] = fmaf(x[k][j] * rstd, a.w ? wv[j] : 1.0f, bv[j]);
            st_vec(static_cast<T*>(a.out) + row * a.cols, (k * TPR + tr) * V, a.cols, al, x[k]);
        }
    }
}

template <typename T, int VPT, int WPR>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>, TPR = WPR * 32, G = kBwdThreads / TPR;
    __shared__ GroupRed<WPR, 2> red[G][2];
    extern __shared__ float sums[];  // [2][TPR * VPT * V], groups > 1 only
    const int g = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    const bool al = a.aligned != 0;
    uint4 w[VPT];
    float dw[VPT][V], db[VPT][V];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        w[k] = a.w ? ld_raw(static_cast<const T*>(a.w), (k * TPR + tr) * V, a.cols, al) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] = db[k][j] = 0.0f;
    }
    const float inv = 1.0f / static_cast<float>(a.cols);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
    int64_t row = static_cast<int64_t>(blockIdx.x) * G + g;
    uint4 nx[VPT], nd[VPT];
    float nm = 0.0f, nr = 0.0f;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V;
            nx[k] = ld_raw(static_cast<const T*>(a.x) + r * a.cols, c, a.cols, al);
            nd[k] = ld_raw(static_cast<const T*>(a.dy) + r * a.cols, c, a.cols, al);
        }
        nm = a.mean[r];
        nr = a.rstd[r];
    };
    if (row < a.rows) fetch(row);
    int flip = 0;
    for (; row < a.rows; row += stride, flip ^= 1) {
        uint4 cx[VPT], cd[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            cx[k] = nx[k];
            cd[k] = nd[k];
        }
        const float mean = nm, rstd = nr;
        if (row + stride < a.rows) fetch(row + stride);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V;
            float x[V], d[V], wv[V];
            unpack<T>(cx[k], x);
            unpack<T>(cd[k], d);
            unpack<T>(w[k], wv);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = (x[j] - mean) * rstd;
                const float gr = a.w ? d[j] * wv[j] : d[j];
                // beyond the row d is zero, x - mean is not
                s[0] += gr;
                s[1] = c + j < a.cols ? fmaf(gr, n, s[1]) : s[1];
                dw[k][j] = c + j < a.cols ? fmaf(d[j], n, dw[k][j]) : 0.0f;
                db[k][j] += d[j];
            }
        }
        group_sum<WPR>(s, red[g][flip], 1 + g);
        const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float x[V], d[V], wv[V];
            unpack<T>(cx[k], x);
            unpack<T>(cd[k], d);
            unpack<T>(w[k], wv);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = (x[j] - mean) * rstd;
                const float gr = a.w ? d[j] * wv[j] : d[j];
                x[j] = rstd * (gr - m1 - n * m2);
            }
            st_vec(static_cast<T*>(a.out) + row * a.cols, (k * TPR + tr) * V, a.cols, al, x);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!a.partial) return;
    float* p = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if constexpr (G > 1) {
        // the groups' sums, one group after the other
        for (int i = 0; i < G; ++i) {
            if (g == i) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int c = j * (TPR * VPT) + k * TPR + tr;  // conflict-free order
                        sums[c] = i ? sums[c] + dw[k][j] : dw[k][j];
                        sums[TPR * VPT * V + c] = i ? sums[TPR * VPT * V + c] + db[k][j] : db[k][j];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.cols; c += kBwdThreads) {
            const int i = (c % V) * (TPR * VPT) + c / V;
            p[c] = sums[i];
            p[a.cols + c] = sums[TPR * VPT * V + i];
        }
    } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (k * TPR + tr) * V + j;
                if (c < a.cols) {
                    p[c] = dw[k][j];
                    p[a.cols + c] = db[k][j];
                }
            }
    }
}

// ------------------------------------------------ ring kernels

using dmuon::tc::add2;
using dmuon::tc::both;
using dmuon::tc::fma2;
using dmuon::tc::mbar_expect_tx;
using dmuon::tc::mbar_init;
using dmuon::tc::mbar_wait;
using dmuon::tc::mul2;
using dmuon::tc::saddr;

constexpr int kMaxStages = 3;
constexpr size_t kRingBytes = 196608;  // most ring memory of a block

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     saddr(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(saddr(bar))
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void unpack2(const uint4& q, float2 (&v)[kVec<T> / 2]) {
    float t[kVec<T>];
    unpack<T>(q, t);
#pragma unroll
    for (int k = 0; k < kVec<T> / 2; ++k) v[k] = make_float2(t[2 * k], t[2 * k + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 pack2(const float2 (&v)[kVec<T> / 2]) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                          __float_as_uint(v[1].y));
    } else {
        return make_uint4(dmuon::tc::pack_bf16x2(v[0].x, v[0].y), dmuon::tc::pack_bf16x2(v[1].x, v[1].y),
                          dmuon::tc::pack_bf16x2(v[2].x, v[2].y), dmuon::tc::pack_bf16x2(v[3].x, v[3].y));
    }
}

// A group's ring of rows in shared memory, `arrays` rows per stage.  Thread 0 of
// the group issues; a stage is refilled once the whole group has passed a
// barrier after reading it.
struct Ring {
    uint8_t* rows;
    uint64_t* full;
    uint32_t bytes;  // of one row
    int arrays;
    bool dead;       // a wait gave up: the results are lost (status), the loop goes on without copies
    __device__ __forceinline__ uint8_t* at(int stage, int k) const { return rows + (stage * arrays + k) * bytes; }
    __device__ __forceinline__ void issue(int stage, const void* a, const void* b) {
        if (dead) return;
        mbar_expect_tx(&full[stage], bytes * arrays);
        bulk_load(at(stage, 0), a, bytes, &full[stage]);
        if (arrays > 1) bulk_load(at(stage, 1), b, bytes, &full[stage]);
    }
    // `issuer`: the thread that issues the copies.  Where its wait gives up, it waits
    // once more (with the same limit) for each stage's copy still under way, so that
    // none lands after the block has left.
    __device__ __forceinline__ void wait(int stage, uint32_t phase, int stages, bool issuer) {
        if (dead || mbar_wait<false>(&full[stage], phase, &g_norm_status)) return;
        dead = true;
        for (int s = 0; issuer && s < stages; ++s)
            mbar_wait<false>(&full[s], s < stage ? phase ^ 1 : phase, &g_norm_status);
    }
};

__device__ __forceinline__ Ring make_ring(uint8_t* smem, uint32_t bytes, int arrays, int stages, int groups, int g,
                                          int tr) {
    // barriers first, then the groups' rows
    Ring r;
    r.full = reinterpret_cast<uint64_t*>(smem) + g * kMaxStages;
    r.rows = smem + (groups * kMaxStages * 8 + 15) / 16 * 16 + static_cast<size_t>(g) * stages * arrays * bytes;
    r.bytes = bytes;
    r.arrays = arrays;
    r.dead = false;
    if (tr == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&r.full[s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    return r;
}

__host__ __device__ constexpr int ring_bwd_threads(int wpr) { return wpr > 8 ? wpr * 32 : 256; }
__host__ __device__ constexpr int ring_groups(int wpr) { return wpr >= 4 ? 1 : 4 / wpr; }

template <typename T, int VPT, int WPR>
__global__ void
__launch_bounds__(ring_groups(WPR) * WPR * 32, 512 / (ring_groups(WPR) * WPR * 32)) norm_fwd_ring_kernel(
    const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>, TPR = WPR * 32, G = ring_groups(WPR);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ GroupRed<WPR, 1> red[G][2];
    const int g = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    Ring ring = make_ring(smem, a.cols * static_cast<uint32_t>(sizeof(T)), 1, a.stages, G, g, tr);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * G + g;
    const T* x0 = static_cast<const T*>(a.x);
    if (tr == 0)
        for (int s = 0; s < a.stages; ++s)
            if (first + s * stride < a.rows) ring.issue(s, x0 + (first + s * stride) * a.cols, nullptr);
    uint4 w[VPT], b[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = (k * TPR + tr) * V;
        w[k] = a.w ? ld_raw(static_cast<const T*>(a.w), c, a.cols, true) : make_uint4(0, 0, 0, 0);
        b[k] = a.b ? ld_raw(static_cast<const T*>(a.b), c, a.cols, true) : make_uint4(0, 0, 0, 0);
    }
    const float inv = 1.0f / static_cast<float>(a.cols);
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t row = first; row < a.rows; row += stride) {
        ring.wait(stage, phase, a.stages, tr == 0);
        float2 x[VPT][V / 2];
        float2 s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (c < a.cols) q = *reinterpret_cast<const uint4*>(ring.at(stage, 0) + c * sizeof(T));
            unpack2<T>(q, x[k]);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) s2 = add2(s2, x[k][j]);
        }
        float s[1] = {s2.x + s2.y};
        group_sum<WPR>(s, red[g][0], 1 + g);
        // the whole group has its part of the row in registers (WPR = 1: the
        // warp's shuffles ordered its reads): refill the stage
        if (tr == 0 && row + a.stages * stride < a.rows)
            ring.issue(stage, x0 + (row + a.stages * stride) * a.cols, nullptr);
        const float mean = s[0] * inv;
        s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const bool in = (k * TPR + tr) * V < a.cols;  // a vector lies inside the row or past it
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                x[k][j] = add2(x[k][j], both(in ? -mean : 0.0f));
                s2 = fma2(x[k][j], x[k][j], s2);
            }
        }
        s[0] = s2.x + s2.y;
        group_sum<WPR>(s, red[g][1], 1 + g);
        const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
        if (tr == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V;
            float2 wv[V / 2], bv[V / 2];
            unpack2<T>(w[k], wv);
            unpack2<T>(b[k], bv);
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
                x[k][j] = fma2(mul2(x[k][j], both(rstd)), a.w ? wv[j] : both(1.0f), bv[j]);
            if (c < a.cols)
                *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * a.cols + c) = pack2<T>(x[k]);
        }
        if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
}

template <typename T, int VPT, int WPR>
__global__ void __launch_bounds__(ring_bwd_threads(WPR), 512 / ring_bwd_threads(WPR)) norm_bwd_ring_kernel(
    const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>, TPR = WPR * 32, G = ring_bwd_threads(WPR) / TPR;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ GroupRed<WPR, 2> red[G][2];
    const int g = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    Ring ring = make_ring(smem, a.cols * static_cast<uint32_t>(sizeof(T)), 2, a.stages, G, g, tr);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * G + g;
    const T *x0 = static_cast<const T*>(a.x), *d0 = static_cast<const T*>(a.dy);
    if (tr == 0)
        for (int s = 0; s < a.stages; ++s) {
            const int64_t r = first + s * stride;
            if (r < a.rows) ring.issue(s, x0 + r * a.cols, d0 + r * a.cols);
        }
    // kAgain: four vectors' column sums leave no registers for n and g, which are
    // computed once more from the row in shared memory for dx; the row's stage is
    // then refilled one row later
    constexpr bool kAgain = VPT == 4;
    constexpr int kKeep = kAgain ? 1 : VPT;
    uint4 w[VPT];
    float2 dw[VPT][V / 2], db[VPT][V / 2];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        w[k] = a.w ? ld_raw(static_cast<const T*>(a.w), (k * TPR + tr) * V, a.cols, true) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) dw[k][j] = db[k][j] = both(0.0f);
    }
    // n, g (and dy, for the sums) of vector k of the row in the given stage
    const auto vec = [&](int stage, int k, float mean, float rstd, float2 (&n)[V / 2], float2 (&gr)[V / 2],
                         float2 (&d)[V / 2]) {
        const int c = (k * TPR + tr) * V;
        uint4 qx = make_uint4(0, 0, 0, 0), qd = qx;
        if (c < a.cols) {
            qx = *reinterpret_cast<const uint4*>(ring.at(stage, 0) + c * sizeof(T));
            qd = *reinterpret_cast<const uint4*>(ring.at(stage, 1) + c * sizeof(T));
        }
        // past the row n is zero too: -mean rstd could be infinite, and its product
        // with g = 0 NaN
        const float2 shift = both(c < a.cols ? -mean : 0.0f);
        float2 wv[V / 2];
        unpack2<T>(qx, n);
        unpack2<T>(qd, d);
        unpack2<T>(w[k], wv);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            n[j] = mul2(add2(n[j], shift), both(rstd));
            gr[j] = a.w ? mul2(d[j], wv[j]) : d[j];
        }
    };
    const auto refill = [&](int stage, int64_t r) {
        if (tr == 0 && r < a.rows) ring.issue(stage, x0 + r * a.cols, d0 + r * a.cols);
    };
    const float inv = 1.0f / static_cast<float>(a.cols);
    int stage = 0, flip = 0;
    uint32_t phase = 0;
    float nm = first < a.rows ? a.mean[first] : 0.0f, nr = first < a.rows ? a.rstd[first] : 0.0f;
    for (int64_t row = first; row < a.rows; row += stride, flip ^= 1) {
        const float mean = nm, rstd = nr;
        if (row + stride < a.rows) {
            nm = a.mean[row + stride];
            nr = a.rstd[row + stride];
        }
        ring.wait(stage, phase, a.stages, tr == 0);
        float2 n[kKeep][V / 2], gr[kKeep][V / 2], s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int q = kAgain ? 0 : k;
            float2 d[V / 2];
            vec(stage, k, mean, rstd, n[q], gr[q], d);
            // a vector past the row is never stored, and its d = n = 0 adds nothing
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                s1 = add2(s1, gr[q][j]);
                s2 = fma2(gr[q][j], n[q][j], s2);
                dw[k][j] = fma2(d[j], n[q][j], dw[k][j]);
                db[k][j] = add2(db[k][j], d[j]);
            }
        }
        float s[2] = {s1.x + s1.y, s2.x + s2.y};
        group_sum<WPR>(s, red[g][flip], 1 + g);
        // past the barrier the group has read this row (kAgain: is done with the
        // row before)
        if (!kAgain) refill(stage, row + a.stages * stride);
        else if (row != first) refill(stage ? stage - 1 : a.stages - 1, row + (a.stages - 1) * stride);
        const float2 m1 = both(-s[0] * inv), m2 = both(-s[1] * inv);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V, q = kAgain ? 0 : k;
            if (kAgain) {
                float2 d[V / 2];
                vec(stage, k, mean, rstd, n[q], gr[q], d);
            }
            float2 o[V / 2];
#pragma unroll
            for (int j = 0; j < V / 2; ++j) o[j] = mul2(fma2(n[q][j], m2, add2(gr[q][j], m1)), both(rstd));
            if (c < a.cols) *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * a.cols + c) = pack2<T>(o);
        }
        if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!a.partial) return;
    float* p = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if constexpr (G > 1) {
        // the groups' sums, one group after the other, in the ring's memory
        // (every copy has been waited for)
        float* sums = reinterpret_cast<float*>(smem);
        constexpr int kCols = TPR * VPT * V;
        __syncthreads();
        for (int i = 0; i < G; ++i) {
            if (g == i) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        const int c = 2 * j * (TPR * VPT) + k * TPR + tr;  // conflict-free order
                        const float2 u = dw[k][j], v = db[k][j];
                        sums[c] = i ? sums[c] + u.x : u.x;
                        sums[c + TPR * VPT] = i ? sums[c + TPR * VPT] + u.y : u.y;
                        sums[kCols + c] = i ? sums[kCols + c] + v.x : v.x;
                        sums[kCols + c + TPR * VPT] = i ? sums[kCols + c + TPR * VPT] + v.y : v.y;
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.cols; c += G * TPR) {
            const int i = (c % V) * (TPR * VPT) + c / V;
            p[c] = sums[i];
            p[a.cols + c] = sums[kCols + i];
        }
    } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + tr) * V;
            if (c < a.cols)
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    *reinterpret_cast<float2*>(p + c + 2 * j) = dw[k][j];
                    *reinterpret_cast<float2*>(p + a.cols + c + 2 * j) = db[k][j];
                }
        }
    }
}

// dw and db: column sums of the partial rows [n][2][cols], 32 columns per block,
// 32 slices of the rows, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* partial, int n, int cols, T* dw, T* db) {
    __shared__ float red[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // column of the 2 x cols pair
    float s = 0.0f;
    if (i < 2 * static_cast<int64_t>(cols)) {
        const float* p = partial + i;
#pragma unroll 4
        for (int r = slice; r < n; r += 32) s += p[static_cast<int64_t>(r) * 2 * cols];
    }
    red[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && i < 2 * static_cast<int64_t>(cols)) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; ++k) s += red[k][lane];
        T* out = i < cols ? dw : db;
        if (out) out[i < cols ? i : i - cols] = from_f<T>(s);
    }
}

// ------------------------------------------------ rows wider than a group

__device__ __forceinline__ float block_sum(float s, float* red) {
    float v[1] = {s};
    warp_sum(v);
    __syncthreads();  // the previous sum has been read
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v[0];
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) s += red[i];
    return s;
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float red[32];
    const float inv = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        T* y = static_cast<T*>(a.out) + row * a.cols;
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) s += to_f(x[c]);
        const float mean = block_sum(s, red) * inv;
        s = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float d = to_f(x[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, red) * inv + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float n = (to_f(x[c]) - mean) * rstd;
            y[c] = from_f<T>(fmaf(n, a.w ? to_f(static_cast<const T*>(a.w)[c]) : 1.0f,
                                  a.b ? to_f(static_cast<const T*>(a.b)[c]) : 0.0f));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float red[32];
    const float inv = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        const T* dy = static_cast<const T*>(a.dy) + row * a.cols;
        T* dx = static_cast<T*>(a.out) + row * a.cols;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float g = to_f(dy[c]) * (a.w ? to_f(static_cast<const T*>(a.w)[c]) : 1.0f);
            s1 += g;
            s2 = fmaf(g, (to_f(x[c]) - mean) * rstd, s2);
        }
        const float m1 = block_sum(s1, red) * inv, m2 = block_sum(s2, red) * inv;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float g = to_f(dy[c]) * (a.w ? to_f(static_cast<const T*>(a.w)[c]) : 1.0f);
            dx[c] = from_f<T>(rstd * (g - m1 - (to_f(x[c]) - mean) * rstd * m2));
        }
    }
}

// Partial row blockIdx.y of dw and db: its share of the rows, one column per thread.
template <typename T>
__global__ void __launch_bounds__(256) norm_cols_wide_kernel(const __grid_constant__ NormArgs a, int64_t per) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
    const int64_t r0 = blockIdx.y * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float d = to_f(static_cast<const T*>(a.dy)[r * a.cols + c]);
        dw = fmaf(d, (to_f(static_cast<const T*>(a.x)[r * a.cols + c]) - a.mean[r]) * a.rstd[r], dw);
        db += d;
    }
    float* p = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    p[c] = dw;
    p[a.cols + c] = db;
}

// ------------------------------------------------ host

int fail(int code, const std::string& msg) {
    dmuon::set_last_error(msg);
    return code;
}

// Row group of `vecs` 16-byte vectors: warps per row and vectors per thread.
struct Shape {
    int vpt = 0, wpr = 0;  // 0: wide kernels
};

// Smallest group with at most `vpt` vectors per thread; rows wider than 16 warps
// take more vectors.
Shape choose(int64_t vecs, int vpt) {
    for (int w = 1; w <= 16; w *= 2)
        if (static_cast<int64_t>(vpt) * w * 32 >= vecs) return {vpt, w};
    for (int v = 2 * vpt; v <= 4; v *= 2)
        if (static_cast<int64_t>(v) * 512 >= vecs) return {v, 16};
    return {};
}

// Ring kernels: rows that start on 16 bytes, enough of them to give every SM a
// block; backward over rows that take a block each, any number.  Below that the
// register kernels' wider groups finish a row sooner.  Measured in bf16, 152 SMs,
// register -> ring kernels:
//   forward     768 columns (4 rows per block): 320 rows 2.3 -> 2.6 us, 640 rows
//               2.8 -> 2.8, 1300 rows 3.6 -> 3.1;  4096 columns (1 row): 80 rows
//               2.5 -> 2.6, 160 rows 2.9 -> 2.7, 1300 rows 8.4 -> 6.0
//   backward    768 columns (4 rows): 320 rows 4.9 -> 5.2, 640 rows 6.7 -> 5.6;
//               4096 columns (1 row): 8 rows 7.9 -> 5.8, 320 rows 20.1 -> 10.9;
//               12288 columns: 8 rows 25.3 -> 13.3, 1300 rows 150 -> 39
bool use_ring(int64_t vecs, const NormArgs& a, bool bwd, int sms) {
    const int wpr = choose(vecs, bwd ? 2 : 4).wpr;
    const int groups = bwd ? ring_bwd_threads(wpr) / (32 * wpr) : ring_groups(wpr);
    return a.aligned && ((bwd && groups == 1) || a.rows >= static_cast<int64_t>(groups) * sms);
}

size_t ring_bytes(int groups, int arrays, int stages, int64_t cols, int es) {
    return (static_cast<size_t>(groups) * kMaxStages * 8 + 15) / 16 * 16 +
           static_cast<size_t>(groups) * stages * arrays * cols * es;
}

// Rows per ring: up to kMaxStages, as many as kRingBytes holds.  At least two do
// (the widest group's row is 32 KB per array), which the backward kernel needs
// where it refills a stage one row late.
int ring_stages(int groups, int arrays, int64_t cols, int es) {
    const size_t row = static_cast<size_t>(groups) * arrays * cols * es;
    return static_cast<int>(std::min<size_t>(kMaxStages, kRingBytes / row));
}

// Launches a ring kernel on as many blocks as fit the device, at most `rows`
// groups of them; *grid receives the block count.
template <typename K>
cudaError_t run_ring(K kernel, dmuon::PerDevice& cfg, const NormArgs& a, int threads, int groups, size_t smem,
                     int max_grid, int* grid, cudaStream_t s) {
    int dev = 0, unused = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cfg.get(dev, &unused, [&](int*) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kRingBytes) + 1024);
        });
    int per_sm = 0, sms = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    *grid = static_cast<int>(std::min<int64_t>({(a.rows + groups - 1) / groups,
                                                static_cast<int64_t>(std::max(per_sm, 1)) * sms, max_grid}));
    kernel<<<*grid, threads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int VPT, int WPR>
cudaError_t run_fwd_ring(const NormArgs& a, int max_grid, int* grid, cudaStream_t s) {
    static dmuon::PerDevice cfg;
    constexpr int groups = ring_groups(WPR), es = sizeof(T);
    NormArgs r = a;
    r.stages = ring_stages(groups, 1, a.cols, es);
    return run_ring(norm_fwd_ring_kernel<T, VPT, WPR>, cfg, r, groups * WPR * 32, groups,
                    ring_bytes(groups, 1, r.stages, a.cols, es), max_grid, grid, s);
}

template <typename T, int VPT, int WPR>
cudaError_t run_bwd_ring(const NormArgs& a, int max_grid, int* grid, cudaStream_t s) {
    static dmuon::PerDevice cfg;
    constexpr int G = ring_bwd_threads(WPR) / (32 * WPR), es = sizeof(T);
    NormArgs r = a;
    r.stages = ring_stages(G, 2, a.cols, es);
    // the groups' column sums reuse the ring
    const size_t sums = G > 1 ? static_cast<size_t>(2) * WPR * 32 * VPT * kVec<T> * 4 : 0;
    return run_ring(norm_bwd_ring_kernel<T, VPT, WPR>, cfg, r, ring_bwd_threads(WPR), G,
                    std::max(sums, ring_bytes(G, 2, r.stages, a.cols, es)), max_grid, grid, s);
}

template <typename T, int VPT, int WPR>
cudaError_t run_registers(const NormArgs& a, bool bwd, int max_grid, int* grid, cudaStream_t s) {
    if (bwd) {
        constexpr int G = bwd_groups(WPR);
        // the groups' column sums: at most 32 KB
        constexpr size_t smem = G > 1 ? static_cast<size_t>(2) * WPR * 32 * VPT * kVec<T> * 4 : 0;
        *grid = static_cast<int>(std::min<int64_t>((a.rows + G - 1) / G, max_grid));
        norm_bwd_kernel<T, VPT, WPR><<<*grid, kBwdThreads, smem, s>>>(a);
    } else {
        constexpr int threads = WPR == 1 ? 128 : WPR * 32, groups = WPR == 1 ? 4 : 1;
        *grid = static_cast<int>(std::min<int64_t>((a.rows + groups - 1) / groups, max_grid));
        norm_fwd_kernel<T, VPT, WPR><<<*grid, threads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

// Forward ring: four vectors per thread, so a 4096-column bf16 row belongs to
// four warps (one vector per thread and sixteen warps: 65 us instead of 50 for
// 16384 x 4096, the two block-wide reductions bound it).  Backward: two vectors
// per thread, whose column sums take 32 registers (one vector: 93 us instead of
// 73), four only in rows wider than 16 warps, which then read the row in shared
// memory twice instead of keeping n and g (1300 x 12288: 47.5 us with spills, 39
// now).
template <typename T>
cudaError_t run_shape(int64_t vecs, const NormArgs& a, bool bwd, bool ring, int max_grid, int* grid, cudaStream_t s) {
    if (ring && !bwd) {
        switch (choose(vecs, 4).wpr) {
            case 1: return vecs <= 32 ? run_fwd_ring<T, 1, 1>(a, max_grid, grid, s)
                                      : run_fwd_ring<T, 4, 1>(a, max_grid, grid, s);
            case 2: return run_fwd_ring<T, 4, 2>(a, max_grid, grid, s);
            case 4: return run_fwd_ring<T, 4, 4>(a, max_grid, grid, s);
            case 8: return run_fwd_ring<T, 4, 8>(a, max_grid, grid, s);
            default: return run_fwd_ring<T, 4, 16>(a, max_grid, grid, s);
        }
    }
    if (ring) {
        const Shape sh = choose(vecs, 2);
        if (sh.vpt == 4) return run_bwd_ring<T, 4, 16>(a, max_grid, grid, s);
        switch (sh.wpr) {
            case 1: return run_bwd_ring<T, 2, 1>(a, max_grid, grid, s);
            case 2: return run_bwd_ring<T, 2, 2>(a, max_grid, grid, s);
            case 4: return run_bwd_ring<T, 2, 4>(a, max_grid, grid, s);
            case 8: return run_bwd_ring<T, 2, 8>(a, max_grid, grid, s);
            default: return run_bwd_ring<T, 2, 16>(a, max_grid, grid, s);
        }
    }
    const Shape sh = choose(vecs, 1);
    if (sh.vpt == 2) return run_registers<T, 2, 16>(a, bwd, max_grid, grid, s);
    if (sh.vpt == 4) return run_registers<T, 4, 16>(a, bwd, max_grid, grid, s);
    switch (sh.wpr) {
        case 1: return run_registers<T, 1, 1>(a, bwd, max_grid, grid, s);
        case 2: return run_registers<T, 1, 2>(a, bwd, max_grid, grid, s);
        case 4: return run_registers<T, 1, 4>(a, bwd, max_grid, grid, s);
        case 8: return run_registers<T, 1, 8>(a, bwd, max_grid, grid, s);
        default: return run_registers<T, 1, 16>(a, bwd, max_grid, grid, s);
    }
}

int check(int64_t rows, int64_t cols, int32_t dtype, const char* where) {
    if (rows < 0 || rows > kMaxRows || cols < 1 || cols > DMUON_MAX_DIM)
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": rows must be in [0, 2^30], cols in [1, 2^20]");
    if (dtype != DMUON_BF16 && dtype != DMUON_FP32)
        return fail(DMUON_ERR_UNSUPPORTED_DTYPE, std::string(where) + ": dtype must be DMUON_BF16 or DMUON_FP32");
    return DMUON_OK;
}

int check_ptr(const void* p, const char* name, const char* where, bool required, size_t align = 16) {
    if (!p) return required ? fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": " + name + " is NULL") : DMUON_OK;
    if (reinterpret_cast<uintptr_t>(p) % align)
        return fail(DMUON_ERR_ALIGN,
                    std::string(where) + ": " + name + " is not " + std::to_string(align) + "-byte aligned");
    return DMUON_OK;
}

int device_sms(int* sms, const char* where) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? DMUON_OK : fail(DMUON_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

int cuda_result(cudaError_t e, const char* where) {
    return e == cudaSuccess ? DMUON_OK : fail(DMUON_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

// Partial rows of the backward pass: the blocks of a persistent grid, at most
// kMaxPartials and no more than rows (a block with no row would write zeros).
int64_t partial_rows(int64_t rows) { return std::min<int64_t>(rows, kMaxPartials); }

}  // namespace

namespace dmuon {

cudaError_t norm_status_word(void** p) { return cudaGetSymbolAddress(p, g_norm_status); }

}  // namespace dmuon

extern "C" int dmuon_layer_norm_forward(const void* x, const void* weight, const void* bias, void* y, float* mean,
                                        float* rstd, int64_t rows, int64_t cols, int32_t dtype, float eps,
                                        void* stream) {
    const char* where = "dmuon_layer_norm_forward";
    int r = check(rows, cols, dtype, where);
    if (r != DMUON_OK) return r;
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": eps must be finite and >= 0");
    if (rows == 0) return DMUON_OK;
    if ((r = check_ptr(x, "x", where, true)) || (r = check_ptr(y, "y", where, true)) ||
        (r = check_ptr(weight, "weight", where, false)) || (r = check_ptr(bias, "bias", where, false)) ||
        (r = check_ptr(mean, "mean", where, false, 4)) || (r = check_ptr(rstd, "rstd", where, false, 4)))
        return r;
    int sms = 0;
    if ((r = device_sms(&sms, where))) return r;
    const bool bf = dtype == DMUON_BF16;
    const int vec = bf ? 8 : 4;
    NormArgs a = {};
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.out = y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.aligned = cols % vec == 0;
    a.eps = eps;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t vecs = (cols + vec - 1) / vec;
    if (choose(vecs, 1).wpr == 0) {
        const int grid = static_cast<int>(std::min<int64_t>(rows, 2 * sms));
        if (bf) norm_fwd_wide_kernel<__nv_bfloat16><<<grid, 1024, 0, s>>>(a);
        else norm_fwd_wide_kernel<float><<<grid, 1024, 0, s>>>(a);
        return cuda_result(cudaGetLastError(), where);
    }
    const bool ring = use_ring(vecs, a, false, sms);
    const int most = ring ? 64 * sms : 4 * sms;
    int grid = 0;
    return cuda_result(bf ? run_shape<__nv_bfloat16>(vecs, a, false, ring, most, &grid, s)
                          : run_shape<float>(vecs, a, false, ring, most, &grid, s),
                       where);
}

extern "C" size_t dmuon_layer_norm_workspace_bytes(int64_t rows, int64_t cols, int32_t dtype) {
    if (check(rows, cols, dtype, "dmuon_layer_norm_workspace_bytes") != DMUON_OK) return 0;
    return static_cast<size_t>(partial_rows(rows)) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" int dmuon_layer_norm_backward(const void* dy, const void* x, const void* weight, const float* mean,
                                         const float* rstd, void* dx, void* dweight, void* dbias, int64_t rows,
                                         int64_t cols, int32_t dtype, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    const char* where = "dmuon_layer_norm_backward";
    int r = check(rows, cols, dtype, where);
    if (r != DMUON_OK) return r;
    if ((r = check_ptr(dweight, "dweight", where, false)) || (r = check_ptr(dbias, "dbias", where, false)) ||
        (r = check_ptr(weight, "weight", where, false)))
        return r;
    const bool sums = dweight || dbias;
    if (rows > 0) {
        if ((r = check_ptr(dy, "dy", where, true)) || (r = check_ptr(x, "x", where, true)) ||
            (r = check_ptr(mean, "mean", where, true, 4)) || (r = check_ptr(rstd, "rstd", where, true, 4)) ||
            (r = check_ptr(dx, "dx", where, true)))
            return r;
        const size_t need = sums ? dmuon_layer_norm_workspace_bytes(rows, cols, dtype) : 0;
        if (need && !workspace) return fail(DMUON_ERR_NO_WORKSPACE, std::string(where) + ": workspace is NULL");
        if (need && reinterpret_cast<uintptr_t>(workspace) % 256)
            return fail(DMUON_ERR_ALIGN, std::string(where) + ": workspace is not 256-byte aligned");
        if (workspace_bytes < need)
            return fail(DMUON_ERR_WORKSPACE_TOO_SMALL, std::string(where) + ": workspace of " +
                                                           std::to_string(workspace_bytes) + " bytes, " +
                                                           std::to_string(need) + " needed");
    }
    int sms = 0;
    if ((r = device_sms(&sms, where))) return r;
    const bool bf = dtype == DMUON_BF16;
    const int vec = bf ? 8 : 4;
    NormArgs a = {};
    a.x = x;
    a.dy = dy;
    a.w = weight;
    a.out = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.aligned = cols % vec == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int partials = 0;
    if (rows > 0) {
        const int64_t vecs = (cols + vec - 1) / vec;
        cudaError_t e;
        if (choose(vecs, 1).wpr == 0) {
            const int grid = static_cast<int>(std::min<int64_t>(rows, 2 * sms));
            if (bf) norm_bwd_wide_kernel<__nv_bfloat16><<<grid, 1024, 0, s>>>(a);
            else norm_bwd_wide_kernel<float><<<grid, 1024, 0, s>>>(a);
            e = cudaGetLastError();
            if (e == cudaSuccess && sums) {
                const int64_t want = std::min<int64_t>(partial_rows(rows), 64);
                const int64_t per = (rows + want - 1) / want;
                partials = static_cast<int>((rows + per - 1) / per);
                const dim3 g2(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(partials));
                if (bf) norm_cols_wide_kernel<__nv_bfloat16><<<g2, 256, 0, s>>>(a, per);
                else norm_cols_wide_kernel<float><<<g2, 256, 0, s>>>(a, per);
                e = cudaGetLastError();
            }
        } else {
            const int most = static_cast<int>(std::min<int64_t>(4 * sms, partial_rows(rows)));
            const bool ring = use_ring(vecs, a, true, sms);
            e = bf ? run_shape<__nv_bfloat16>(vecs, a, true, ring, most, &partials, s)
                   : run_shape<float>(vecs, a, true, ring, most, &partials, s);
        }
        if (e != cudaSuccess) return cuda_result(e, where);
    }
    if (!sums) return DMUON_OK;
    const int grid = static_cast<int>((2 * cols + 31) / 32);
    const dim3 blocks(static_cast<unsigned>(grid));
    const cudaError_t e = bf ? dmuon::launch_dependent(norm_reduce_kernel<__nv_bfloat16>, blocks, 1024, s, a.partial,
                                                       partials, a.cols, static_cast<__nv_bfloat16*>(dweight),
                                                       static_cast<__nv_bfloat16*>(dbias))
                             : dmuon::launch_dependent(norm_reduce_kernel<float>, blocks, 1024, s, a.partial, partials,
                                                       a.cols, static_cast<float*>(dweight),
                                                       static_cast<float*>(dbias));
    return cuda_result(e, where);
}
