// Attention forward on the tensor cores (bf16, rows of 16-byte stride).
//
//   s = q k^T, p = exp(scale s - m), o = sum_j p v / sum_j p
//
// A CTA takes 256 queries of one head (two tiles of 128) and runs over their keys, 128
// at a time.  Per tile and key tile the tensor cores form s (128 x 128, in TMEM), a
// warpgroup turns it into p in bf16 in the same TMEM columns -- a thread has a
// whole row, so maximum and sum need no exchange --, and the tensor cores add p v to the
// tile's output in TMEM.  The two tiles alternate: while the warpgroup of one works, the
// tensor cores run the other's products.  The output is not rescaled whenever the
// row's maximum grows but only when it has grown by 2^8 since the last time (p then
// reaches 2^8 at most, exact in fp32 sums and as precise in bf16); s of the tile is
// complete only after the product before it, so the warpgroup may do that itself.
//
// Heads of up to 64 leave TMEM for a third buffer of s, which the two tiles take in turn,
// so that s is formed a unit ahead; larger ones hand p over in two halves instead, the
// first of which the tensor cores take while the second is made.
//
// Warp 0 loads (a ring of K and V tiles), warp 1 issues the MMAs, warps 4 .. work on the
// softmax, one warpgroup per tile.  A CTA that has come to its end takes over the next block
// that has not started, without another set-up.
//
// Bound: the tensor cores, 4 * 128 * 128 * dim operations per pair of tiles -- at dim =
// 128 1024 cycles, against 512 of exponentials (32 a cycle and SM) and about 670 of all the
// softmax's pipes.  Measured: 16384 tokens, 32/8 heads of 128, causal: 1.22 ms, 1.80 PFLOP/s,
// 92 % of cuBLAS's burst rate (1.33 ms = 1.65 in a loop, under the power cap).  Heads of 64: the
// chain of waits of a tile (s, TMEM load, maximum, exponentials, store, arrival) with two warpgroups:
// 12 heads, 8192 tokens: 104 us, 1.0 PFLOP/s, about 1250 cycles a pair of tiles where the MMAs and
// the exponentials take 512 each and all of the softmax's pipes 670; tensor cores and exponentials are
// 48 % busy, issue slots 46 %, and 13 % of the time SMs have run out of tiles.  Short sequences: start and end of a
// tile, about 3 us (23 ragged ones of 356 tokens, 12 heads of 64: 32 us).
#include <cstddef>

#include "attn_tc.cuh"
#include "internal.h"
#include "ops.h"

namespace dmuon {
namespace attn {
namespace {

__device__ int32_t g_status = 0;

constexpr int kSoftWarp0 = 4;

template <int DP, int NT>
struct Cfg {
    static constexpr int kThreads = 128 + 128 * NT;
    static constexpr int kBuffers = NT == 1 ? 1 : DP == 64 ? 3 : 2;  // of s, in TMEM
    static constexpr bool kHalves = kBuffers == 2;                   // p is handed over in two halves
    static constexpr int kStages = NT == 2 ? (DP == 128 ? 5 : 8) : (DP == 128 ? 2 : 4);
    static constexpr uint32_t kCols = NT == 2 ? 512 : 256;
    // shares of 168 x 3 or 128 x 2 (NT = 1: ptxas spills 40 bytes at DP = 64 and 48 at 128)
    static constexpr int kRegsLow = 56, kRegsSoft = NT == 2 ? 224 : 200;
};

// What a CTA does next.
enum Kind : int32_t { TILE, CLEAR, NONE };

struct Item {
    int32_t kind, head;
    int32_t begin, len, tile;  // of the sequence, as AttnTile; CLEAR: tile is the share
};

template <int DP, int NT>
struct __align__(1024) Smem {
    using C = Cfg<DP, NT>;
    uint8_t q[NT][kTile<DP>];
    uint8_t kv[C::kStages][kTile<DP>];
    uint64_t q_full;
    uint64_t full[C::kStages];
    uint64_t empty[C::kStages];
    uint64_t s_full[C::kBuffers];
    uint64_t p_half[C::kBuffers];
    uint64_t p_ready[C::kBuffers];
    uint64_t pv_done[NT][2];  // products of the even and the odd key tiles
    uint64_t o_full[NT];
    uint64_t drained;
    uint4 claim;                // answer to the request for another block's index
    uint64_t claimed;
    Item item[2];               // at hand, and the next
    uint32_t tmem;
    int32_t bad;                // a wait gave up
};

// The products of a CTA, in the order in which the tensor cores run them: unit u is key
// tile j of query tile i, alternating between the query tiles while both have keys
// left.  Its s lies in buffer u % kBuffers.
struct Units {
    int n[2], lo, more;  // key tiles of each query tile, the fewer, the query tile with more
    __device__ __forceinline__ int count() const { return n[0] + n[1]; }
    __device__ __forceinline__ int of(int i, int j) const { return j < lo ? 2 * j + i : lo + j; }
    __device__ __forceinline__ void at(int u, int& i, int& j) const {
        const bool both = u < 2 * lo;
        i = both ? u & 1 : more;
        j = both ? u >> 1 : u - lo;
    }
};

// Place of K_j and V_j in the ring's order, `steps` tiles each: as the tensor cores
// first need them (with three buffers s runs a tile further ahead).
template <int kBuffers>
__device__ __forceinline__ int place(bool v, int j, int steps) {
    if (kBuffers < 3) return 2 * j + (v ? 1 : 0);
    if (!v) return j == 0 ? 0 : 2 * j - 1;
    return j + 1 < steps ? 2 * j + 2 : 2 * j + 1;
}

// Growth of a row's maximum, in powers of two, that is left in p.
constexpr float kLazy = 8.0f;

// The item of a block index.  False: its slot holds no tile.
template <int NT>
__device__ __forceinline__ bool find_item(const AttnArgs& a, unsigned block, Item& item) {
    const unsigned slot = block / static_cast<unsigned>(a.heads);
    const int head = static_cast<int>(block - slot * a.heads);
    item = Item{CLEAR, 0, 0, 0, static_cast<int>(block - static_cast<unsigned>(a.slots) * a.heads)};
    if (static_cast<int>(slot) >= a.slots) return true;
    AttnTile t;
    if (!attn_find(a, static_cast<int>(slot), NT * kRows, t)) return false;
    item = Item{TILE, head, static_cast<int32_t>(t.begin), t.len, t.tile};
    return true;
}

// The next item, by one warp, from the blocks that have not started.
template <int DP, int NT>
__device__ __forceinline__ Item next_item(const AttnArgs& a, Smem<DP, NT>& S, uint32_t& asked, int lane) {
    Item item;
    uint32_t block = 0;
    while (claim_block(&S.claim, &S.claimed, asked, block, &S.bad, lane))
        if (find_item<NT>(a, block, item)) return item;
    return Item{NONE, 0, 0, 0, 0};
}

// One barrier a lane and turn, in the order of Smem.
template <int DP, int NT>
__device__ __forceinline__ void init_barriers(Smem<DP, NT>& S, int lane, bool again) {
    using C = Cfg<DP, NT>;
    using M = Smem<DP, NT>;
    constexpr int n = static_cast<int>((offsetof(M, drained) - offsetof(M, q_full)) / 8) + 1;
    for (int k = lane; k < n; k += 32) {
        uint64_t* bar = &S.q_full + k;
        if (again) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(saddr(bar)) : "memory");
        mbar_init(bar, bar >= S.p_half && bar < S.p_ready + C::kBuffers ? 4 : 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// A tile's output, by the helper warps (kSoft false) or those of the softmax.
template <int DP, int NT, bool kSoft>
__device__ __forceinline__ void run_tile(const AttnArgs& a, Smem<DP, NT>& S, const CUtensorMap* mq, const CUtensorMap* mk,
                                         const CUtensorMap* mv, const AttnTile& t, int head, int warp, int lane,
                                         uint32_t tmem) {
    using C = Cfg<DP, NT>;
    constexpr int NS = C::kStages, NB = C::kBuffers;
    // the tiles with most keys first
    const int row0 = (a.causal ? (t.len - 1) / (NT * kRows) - t.tile : t.tile) * NT * kRows;
    const int token0 = static_cast<int>(t.begin);
    Units units;
    units.n[1] = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int first = row0 + i * kRows;
        const int keys = a.causal ? min(t.len, first + kRows) : t.len;
        units.n[i] = first < t.len ? (keys + kRows - 1) / kRows : 0;  // 0: no rows
    }
    units.lo = min(units.n[0], units.n[1]);
    units.more = units.n[1] > units.n[0] ? 1 : 0;
    const int steps = max(units.n[0], units.n[1]);

    const uint32_t t_s = tmem, t_o = tmem + NB * kRows;

    if constexpr (!kSoft) {
        if (warp == 0) {
            // ------------------------------------------------ loads
            const uint32_t e = elect_one();
            mbar_expect_tx_if(e, &S.q_full, (units.n[1] > 0 ? 2 : 1) * kTile<DP>);
            for (int i = 0; i < NT; ++i)
                if (units.n[i] > 0)
                    load_tile<DP>(e, saddr(S.q[i]), mq, saddr(&S.q_full), head, token0 + row0 + i * kRows);
            int stage = 0;
            uint32_t phase = 0;
            int i = 0;
            for (; i < 2 * steps; ++i) {
                if (!__all_sync(kFullMask, mbar_wait<false>(&S.empty[stage], phase ^ 1, &S.bad))) break;
                bool v = (i & 1) != 0;
                int tile = i / 2;
                if (NB == 3 && i > 0) {  // K0 K1 V0 K2 V1 .. V_last
                    v = i % 2 == 0 || i + 1 == 2 * steps;
                    tile = i + 1 == 2 * steps ? steps - 1 : v ? i / 2 - 1 : (i + 1) / 2;
                }
                mbar_expect_tx_if(e, &S.full[stage], kTile<DP>);
                load_tile<DP>(e, saddr(S.kv[stage]), v ? mv : mk, saddr(&S.full[stage]), head / a.group,
                              token0 + tile * kRows);
                if (++stage == NS) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            await_copies(&S.q_full, S.full, i, NS, &S.bad);
        } else if (warp == 1) {
            // ------------------------------------------------ MMAs
            const uint32_t e = elect_one();
            const uint32_t q0 = saddr(S.q[0]), kv0 = saddr(S.kv[0]);
            const int total = units.count();
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool r = __all_sync(kFullMask, mbar_wait<false>(bar, parity, &S.bad));
                fence_after();
                return r;
            };
            // s of unit u into its buffer, which the product NB units before has left
            const auto form_s = [&](int u) {
                int i, j;
                units.at(u, i, j);
                const int at = place<NB>(false, j, steps), slot = at % NS;
                if (!wait(&S.full[slot], (at / NS) & 1)) return false;
                product_cols<DP>(e, t_s + u % NB * kRows, desc_k(q0 + i * kTile<DP>), desc_k(kv0 + slot * kTile<DP>));
                umma_commit(e, saddr(&S.s_full[u % NB]));
                if (i == 1 || j >= units.lo) umma_commit(e, saddr(&S.empty[slot]));  // K_j's last use
                return true;
            };
            bool ok = wait(&S.q_full, 0);
            for (int u = 0; u < NB && u < total && ok; ++u) ok = form_s(u);
            for (int u = 0; u < total && ok; ++u) {
                int i, j;
                units.at(u, i, j);
                const int at = place<NB>(true, j, steps), slot = at % NS, b = u % NB;
                const uint32_t parity = (u / NB) & 1;
                const uint64_t v = desc_mn(kv0 + slot * kTile<DP>);
                ok = wait(&S.full[slot], (at / NS) & 1) && wait(C::kHalves ? &S.p_half[b] : &S.p_ready[b], parity);
                if (!ok) break;
                product_rows<DP>(e, t_o + i * DP, t_s + b * kRows, v, 0, C::kHalves ? 4 : 8, j > 0);
                if (C::kHalves) {
                    ok = wait(&S.p_ready[b], parity);
                    if (!ok) break;
                    product_rows<DP>(e, t_o + i * DP, t_s + b * kRows + 32, v, 4, 4, true);
                }
                umma_commit(e, saddr(j + 1 == (i ? units.n[1] : units.n[0]) ? &S.o_full[i] : &S.pv_done[i][j & 1]));
                if (i == 1 || j >= units.lo) umma_commit(e, saddr(&S.empty[slot]));
                if (u + NB < total) ok = form_s(u + NB);
            }
            // also after a wait that gave up: no MMA or commit is under way when the CTA leaves
            umma_commit(e, saddr(&S.drained));
            mbar_wait<false>(&S.drained, 0, &S.bad);
        }
    } else {
        // ------------------------------------------------ softmax
        const int tile = (warp - kSoftWarp0) / 4, quarter = warp % 4, thread = threadIdx.x % 128;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t to = t_o + tile * DP + lanes;
        const int row = row0 + tile * kRows + thread;
        const int count = tile ? units.n[1] : units.n[0];
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool r = __all_sync(kFullMask, mbar_wait<false>(bar, parity, &S.bad));
            fence_after();
            return r;
        };
        const float c = a.scale_log2;
        // rows behind the sequence belong to the next one: they have no say in when the
        // others are rescaled, which shows in the last bits
        const float lazy = row < t.len ? kLazy : __int_as_float(0x7f800000);
        float top = __int_as_float(0xff800000), base = 0.0f, sum = 0.0f;
        bool ok = true;
        for (int j = 0; j < count; ++j) {
            const int u = units.of(tile, j), b = u % NB;
            const uint32_t ts = t_s + b * kRows + lanes;
            ok = wait(&S.s_full[b], (u / NB) & 1);
            if (!ok) break;
            float s[kRows];
            tmem_ld128(ts, s);
            const int keys = min(kRows, t.len - j * kRows);
            if (keys < kRows || (a.causal && j + 1 == count)) {
                const int seen = a.causal ? min(row + 1 - j * kRows, keys) : keys;
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    if (k >= seen) s[k] = __int_as_float(0xff800000);
            }
            float m[4] = {top, top, top, top};
#pragma unroll
            for (int k = 0; k < kRows; k += 8)
#pragma unroll
                for (int x = 0; x < 4; ++x) m[x] = fmaxf(m[x], fmaxf(s[k + 2 * x], s[k + 2 * x + 1]));
            const float grown = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            if (j == 0) {
                top = grown;
                base = exp_shift(top) * c;
            } else if (__any_sync(kFullMask, (grown - top) * c > lazy)) {
                // (a row without a finite logit so far has added nothing)
                const float fresh = exp_shift(grown) * c;
                const float f = top == __int_as_float(0xff800000) ? 0.0f : ex2(base - fresh);
                top = grown;
                base = fresh;
                sum *= f;
                // s of this unit was formed after the product of tile j - 3 at the earliest, so
                // the parity means no other phase
                ok = wait(&S.pv_done[tile][(j - 1) & 1], ((j - 1) >> 1) & 1);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < DP; k += 32) {
                    float o[32];
                    uint32_t w[32];
                    tmem_ld32(to + k, o);
#pragma unroll
                    for (int x = 0; x < 32; ++x) w[x] = __float_as_uint(o[x] * f);
                    tmem_st32(to + k, w);
                }
            }
            if (keys < kRows) {
                // the values of keys behind the sequence
                const int at = place<NB>(true, j, steps);
                ok = wait(&S.full[at % NS], (at / NS) & 1);
                if (!ok) break;
                clear_rows<DP>(S.kv[at % NS], keys, thread, 128);
            }
            const float2 c2 = both(c), b2 = both(-base);
            float2 part[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float2 x = fma2(make_float2(s[64 * h + 2 * k], s[64 * h + 2 * k + 1]), c2, b2);
                    const float2 p = make_float2(ex2(x.x), ex2(x.y));
                    part[k % 4] = add2(part[k % 4], p);
                    w[k] = pack_bf16x2(p.x, p.y);
                }
                tmem_st32(ts + 32 * h, w);
                if (h == 1 || C::kHalves) {
                    tmem_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(h == 0 ? &S.p_half[b] : &S.p_ready[b]);
                }
            }
            const float2 all = add2(add2(part[0], part[1]), add2(part[2], part[3]));
            sum += all.x + all.y;
        }
        if (ok && count > 0 && wait(&S.o_full[tile], 0)) {
            const int64_t token = t.begin + row, first = token - lane;
            store_rows<DP / 64>(S.q[tile] + quarter * 4096, to, 1.0f / sum,
                                static_cast<__nv_bfloat16*>(a.out) + (first * a.heads + head) * a.dim,
                                static_cast<int64_t>(a.heads) * a.dim, t.len - (row - lane), a.dim, lane);
            // from what was subtracted, so that lse and p belong together
            if (row < t.len) a.lse[head * a.tokens + token] = (base + log2f(sum)) * 0.6931471805599453f;
        }
    }
}

// All items of a CTA.
template <int DP, int NT, bool kSoft>
__device__ __forceinline__ void work(const AttnArgs& a, Smem<DP, NT>& S, const CUtensorMap* mq, const CUtensorMap* mk,
                                     const CUtensorMap* mv, int warp, int lane, uint32_t tmem) {
    uint32_t asked = 0;
    for (int n = 0;; ++n) {
        const Item& now = S.item[n & 1];
        // from one lane: uniform, as MMAs and copies take their operands
        const int kind = __shfl_sync(kFullMask, now.kind, 0), head = __shfl_sync(kFullMask, now.head, 0);
        AttnTile t;
        t.begin = __shfl_sync(kFullMask, now.begin, 0);
        t.len = __shfl_sync(kFullMask, now.len, 0);
        t.tile = __shfl_sync(kFullMask, now.tile, 0);
        if (kind == NONE) return;
        if (kind == TILE) {
            run_tile<DP, NT, kSoft>(a, S, mq, mk, mv, t, head, warp, lane, tmem);
        } else if (kSoft) {
            attn_clear(a, static_cast<__nv_bfloat16*>(a.out), a.lse, a.heads, t.tile, threadIdx.x - 32 * kSoftWarp0,
                       128 * NT);
        }
        if (!kSoft && warp == 0) {
            // after this item's last loads are issued
            const Item item = next_item<DP, NT>(a, S, asked, lane);
            if (lane == 0) S.item[(n + 1) & 1] = item;
        }
        // shared memory, TMEM and barriers pass to the next item
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        fence_before();
        __syncthreads();
        if (__shfl_sync(kFullMask, S.bad, 0) != 0) return;
        if (!kSoft && warp == 2) init_barriers(S, lane, true);
        __syncthreads();
        fence_after();
    }
}

template <int DP, int NT>
__global__ void __launch_bounds__(Cfg<DP, NT>::kThreads, NT == 1 ? 2 : 1)
    forward_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using C = Cfg<DP, NT>;
    extern __shared__ uint8_t raw[];
    Smem<DP, NT>& S = *reinterpret_cast<Smem<DP, NT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(kFullMask, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    if (warp == 1) {
        tmem_alloc<C::kCols>(&S.tmem);
    } else if (warp == 2) {
        init_barriers(S, lane, false);
    } else if (warp == 0) {
        if (lane == 0) {
            mbar_init(&S.claimed, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            S.bad = 0;
        }
        // meanwhile, and only after the kernels before have finished
        asm volatile("griddepcontrol.wait;" ::: "memory");
        Item item;
        // (a block without a tile ends here: its successor is another block of the grid)
        if (!find_item<NT>(a, blockIdx.x, item)) item.kind = NONE;
        if (lane == 0) S.item[0] = item;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, S.tmem, 0);
    if (warp < kSoftWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsLow));
        work<DP, NT, false>(a, S, &mq, &mk, &mv, warp, lane, tmem);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
        work<DP, NT, true>(a, S, &mq, &mk, &mv, warp, lane, tmem);
    }
    fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && S.bad) atomicExch(&g_status, 1);
    if (warp == 1) {
        __syncwarp();
        fence_after();
        tmem_free<C::kCols>(tmem);
    }
}

template <int DP, int NT>
constexpr size_t smem_bytes() {
    return sizeof(Smem<DP, NT>) + 1024;
}

template <int DP, int NT>
cudaError_t attribute() {
    return cudaFuncSetAttribute(forward_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem_bytes<DP, NT>()));
}

cudaError_t prepare() {
    static PerDevice cache;
    int dev = 0, ok = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cache.get(dev, &ok, [](int* out) {
        *out = 1;
        cudaError_t r = attribute<64, 1>();
        if (r == cudaSuccess) r = attribute<64, 2>();
        if (r == cudaSuccess) r = attribute<128, 1>();
        if (r == cudaSuccess) r = attribute<128, 2>();
        return r;
    });
}

template <int DP, int NT>
cudaError_t launch(AttnArgs a, const AttnMaps& m, cudaStream_t s) {
    a.slots = static_cast<int32_t>(attn_slots(a.tokens, a.sequences, NT * kRows));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.slots) * a.heads + a.fill);
    cfg.blockDim = dim3(Cfg<DP, NT>::kThreads);
    cfg.dynamicSmemBytes = smem_bytes<DP, NT>();
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, forward_kernel<DP, NT>, a, m.q, m.k, m.v);
}

}  // namespace
}  // namespace attn

cudaError_t attn_fwd_status_word(void** p) { return cudaGetSymbolAddress(p, attn::g_status); }

cudaError_t attn_tc_forward(const AttnArgs& a, const AttnMaps& m, cudaStream_t s) {
    const cudaError_t e = attn::prepare();
    if (e != cudaSuccess) return e;
    // One query tile per CTA, two CTAs per SM, where sequences are short: one CTA's start and
    // end fall under the other's work.  Long ones: two tiles that share the keys.  Measured,
    // two tiles -> one (8192 tokens, 32/8 heads of 128 | 12 of 64), sequences of about
    //   100 tokens 100 -> 76 us | 37 -> 29;  356: | 35 -> 37;  512: 82 -> 80;  1024: | 41 -> 41;
    //   1640: 123 -> 127;  2048: 137 -> 146;  8192: 332 -> 358 | 104 -> 117
    const bool one = a.tokens / a.sequences <= (a.dim <= 64 ? 256 : 1024);
    if (a.dim <= 64) return one ? attn::launch<64, 1>(a, m, s) : attn::launch<64, 2>(a, m, s);
    return one ? attn::launch<128, 1>(a, m, s) : attn::launch<128, 2>(a, m, s);
}

}  // namespace dmuon
