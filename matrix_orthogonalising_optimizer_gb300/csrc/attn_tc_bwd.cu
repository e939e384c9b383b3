// Attention backward on the tensor cores (bf16, rows of 16-byte stride).
//
//   p = exp(scale s - lse), dp = do v^T, ds = p (dp - delta)
//   dv = p^T do, dk = scale ds^T q          (a CTA per 128 keys, over the queries)
//   dq = scale ds k                         (a CTA per 128 queries, over the keys)
//
// s and dp are formed twice, once for each side: seven products of 128 x 128 x dim
// where five would do.  In return every gradient is summed by one CTA in TMEM in a
// fixed order -- no atomics, no fp32 partial sums through L2 --, and p and ds never
// pass through shared memory: the side of the keys works on s^T = k q^T, whose rows
// are what dv and dk need as the left operand in TMEM, the side of the queries on s.
// Both kinds of tile are blocks of one launch, so that one fills the other's last wave, and
// a CTA that has come to its end takes over the next block that has not started, without
// another set-up.
//
// Keys: TMEM holds s^T and dp^T (p^T and ds^T take their place, bf16), dv and dk.  The
// tensor cores run dv_i, s_{i+1}, dk_i, dp_{i+1}: the exponentials of tile i + 1 fall
// under dk_i and dp_{i+1}, and ds_i under dv_i and s_{i+1}.  The query heads that share
// the key head follow one another.  (Heads of up to 64: as the queries.)
// Queries: s, dp, ds, Q and dq; s and dp are taken into registers first, so that
// s_{i+1} and dp_{i+1} run while ds_i is made, then dq_i.
// Sequences of one tile, in batches of short ones: a CTA makes all three gradients (short_side).
//
// Bound: the tensor cores.  Per pair of 128-token tiles 7 * 512 cycles at dim = 128;
// measured about 2300 a step of the keys (2048 of MMAs) and 1850 of the queries (1536), and 3
// to 6 us a tile besides.  8192 tokens, 32/8 heads of 128, causal: 1.07 ms with delta,
// 1.28 PFLOP/s of the five products, 1.80 of the seven; five documents packed into 8192
// tokens 0.39 ms; 12 heads of 64 0.31 ms (element-wise work and hand-overs).
//
// delta = do . o is taken from o as it was rounded to bf16 (short_side: from p dp): errors of dq and
// dk of 2.8e-3 of their norm, where the roundings of ds and of the results alone make 2.4e-3; the
// exact delta would take two products more.  A row that sees one key only has ds = 0 exactly.
//
// Warp 0 loads and looks for the next item, warp 1 issues the MMAs, warp 2 fetches lse and
// delta of the query tiles (side of the keys), warps 4 to 11 do the element-wise work, half of
// the columns each warpgroup.
#include <cstddef>

#include "attn_tc.cuh"
#include "internal.h"
#include "ops.h"

namespace dmuon {
namespace attn {
namespace {

__device__ int32_t g_status = 0;

constexpr int kThreads = 384;
constexpr int kEltWarp0 = 4, kEltWarps = 8;
constexpr uint32_t kCols = 512;
// 88 + 2 x 208 = 3 x 168: the launch's registers (with 56 the issuing warp spills: 3 % slower)
constexpr int kRegsLow = 88, kRegsElt = 208;

template <int DP>
constexpr int kStages = DP == 128 ? 5 : 8;

// What a CTA does next: a tile's gradients, or rows and partial sums to clear.
enum Kind : int32_t { KEYS, WHOLE, QUERIES, CLEAR, CLEAR_PART, NONE };

struct Item {
    int32_t kind, head, part;
    int32_t begin, len, tile;  // of the sequence, as AttnTile; CLEAR: tile is the share
};

template <int DP>
struct __align__(1024) Smem {
    uint8_t own[2][kTile<DP>];  // keys: K, V | queries: dO; the second is a slot of the ring, Q its first tile
    uint8_t ring[kStages<DP>][kTile<DP>];
    float stat[2][2][kRows];    // keys: -lse log2(e) and -delta of two query tiles
    uint64_t own_full;
    uint64_t full[kStages<DP> + 1];
    uint64_t empty[kStages<DP> + 1];
    uint64_t s_full;            // s, or s and dp
    uint64_t g_full;            // dp
    uint64_t taken;             // s and dp are in registers
    uint64_t p_ready;
    uint64_t ds_ready;          // ds, or p and ds
    uint64_t used;              // they have been read
    uint64_t q_ready;
    uint64_t stat_full[2];
    uint64_t stat_empty[2];
    uint64_t done;
    uint4 claim;                // answer to the request for another block's index
    uint64_t claimed;
    Item item[2];               // at hand, and the next
    uint32_t tmem;
    int32_t bad;                // a wait gave up
};

template <int kSlots>
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kSlots) {
            stage = 0;
            phase ^= 1;
        }
    }
};

template <int DP>
__device__ __forceinline__ bool wait_warp(Smem<DP>& S, uint64_t* bar, uint32_t parity) {
    const bool r = __all_sync(kFullMask, mbar_wait<false>(bar, parity, &S.bad));
    fence_after();
    return r;
}

// One arrival per warp, after its TMEM stores and its writes to shared memory.
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
    tmem_st_wait();
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// One arrival per warp, after its TMEM loads.
__device__ __forceinline__ void release_warp(uint64_t* bar, int lane) {
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Loads tiles 0 .. count - 1 through a ring of kSlots at `slots`: what(i, map, head, token)
// says which.
template <int DP, int kSlots, typename F>
__device__ __forceinline__ void produce(Smem<DP>& S, uint32_t e, const uint8_t* slots, int count, F what) {
    Ring<kSlots> r;
    int i = 0;
    for (; i < count; ++i) {
        if (!__all_sync(kFullMask, mbar_wait<false>(&S.empty[r.stage], r.phase ^ 1, &S.bad))) break;
        const CUtensorMap* map;
        int head, token;
        what(i, map, head, token);
        mbar_expect_tx_if(e, &S.full[r.stage], kTile<DP>);
        load_tile<DP>(e, saddr(slots) + r.stage * kTile<DP>, map, saddr(&S.full[r.stage]), head, token);
        r.next();
    }
    await_copies(&S.own_full, S.full, i, kSlots, &S.bad);
}

// 64 columns, packed, into TMEM columns t .. t + 31.
__device__ __forceinline__ void store_cols64(uint32_t t, const float (&v)[64]) {
    uint32_t w[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    tmem_st32(t, w);
}

// ---------------------------------------------------------------- side of the keys

// The steps [begin, end) that a part of a key tile takes: query tiles of all its heads,
// from the first that sees any of the keys on.
__device__ __forceinline__ int part_begin(const AttnArgs& a, const AttnTile& t, int part) {
    const int queries = a.causal ? t.len - t.tile * kRows : t.len;
    return attn_part((queries + kRows - 1) / kRows * a.group, part, a.parts);  // one tile: heads
}

// The rows of no sequence, by the element-wise warps: share f of a.fill.
template <typename T>
__device__ __forceinline__ void clear_rows_of(const AttnArgs& a, T* x, int heads, int f) {
    attn_clear(a, x, nullptr, heads, f, threadIdx.x - 32 * kEltWarp0, 32 * kEltWarps);
}

// A part without steps: its sums are zero.
__device__ __forceinline__ void clear_part(const AttnArgs& a, const AttnTile& t, int kv, int part) {
    const int rows = min(kRows, t.len - t.tile * kRows);
    const int64_t first = ((t.begin + t.tile * kRows) * a.kv_heads + kv) * a.dim;
    for (int i = threadIdx.x - 32 * kEltWarp0; i < rows * a.dim; i += 32 * kEltWarps) {
        const int64_t at = first + static_cast<int64_t>(i / a.dim) * a.kv_heads * a.dim + i % a.dim;
        attn_partial(a, 0, part)[at] = 0.0f;
        attn_partial(a, 1, part)[at] = 0.0f;
    }
}

// TMEM columns.  Heads of up to 64 leave room for p and ds beside s and dp, which then
// make way for the next tile as soon as they are in registers.
template <int DP>
struct KeysCols {
    static constexpr bool kApart = DP == 64;
    static constexpr uint32_t kS = 0, kG = kRows;
    static constexpr uint32_t kP = kApart ? 256 : kS, kDs = kApart ? 320 : kG;
    static constexpr uint32_t kDv = kApart ? 384 : 256, kDk = kDv + DP;
    static constexpr uint32_t kHalf = kApart ? 32 : 64;  // between the halves of p and ds
};

// The sums of a key tile: one warpgroup stores dv, the other dk, or their partial sums.
template <int DP>
__device__ __forceinline__ void store_keys(const AttnArgs& a, Smem<DP>& S, const AttnTile& t, int kv, int part, int half,
                                           int quarter, uint32_t dk, uint32_t dv, uint32_t lanes, int lane) {
    const int row = t.tile * kRows + 32 * quarter;
    const int64_t at = ((t.begin + row) * a.kv_heads + kv) * a.dim, ld = static_cast<int64_t>(a.kv_heads) * a.dim;
    uint8_t* stage = S.own[half] + quarter * 4096;
    const uint32_t from = (half ? dk : dv) + lanes;
    if (a.parts > 1)
        store_rows_f32<DP / 64>(stage, from, attn_partial(a, 1 - half, part) + at, ld, t.len - row, a.dim, lane);
    else
        store_rows<DP / 64>(stage, from, half ? a.scale : 1.0f, static_cast<__nv_bfloat16*>(half ? a.dk : a.dv) + at, ld,
                            t.len - row, a.dim, lane);
}

template <int DP, bool kElt>
__device__ __forceinline__ void keys_side(const AttnArgs& a, Smem<DP>& S, const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv, const CUtensorMap* mo, const AttnTile& t, int kv,
                                          int part, int warp, int lane, uint32_t tmem) {
    using C = KeysCols<DP>;
    constexpr int NS = kStages<DP>;
    const int token0 = static_cast<int>(t.begin), row0 = t.tile * kRows;
    const int first = a.causal ? row0 : 0;                             // the first query that sees any of the keys
    const int per_head = (t.len - first + kRows - 1) / kRows;
    const int begin = part_begin(a, t, part), steps = part_begin(a, t, part + 1) - begin;
    const auto where = [&](int i, int& head, int& row) {
        const int h = (begin + i) / per_head;
        head = kv * a.group + h;
        row = first + (begin + i - h * per_head) * kRows;
    };
    if (!kElt && warp == 0) {
        const uint32_t e = elect_one();
        mbar_expect_tx_if(e, &S.own_full, 2 * kTile<DP>);
        load_tile<DP>(e, saddr(S.own[0]), mk, saddr(&S.own_full), kv, token0 + row0);
        load_tile<DP>(e, saddr(S.own[1]), mv, saddr(&S.own_full), kv, token0 + row0);
        produce<DP, NS>(S, e, S.ring[0], 2 * steps, [&](int i, const CUtensorMap*& map, int& head, int& token) {
            where(i / 2, head, token);
            token += token0;
            map = i & 1 ? mo : mq;
        });
    } else if (!kElt && warp == 1) {
        const uint32_t e = elect_one();
        const uint32_t own = saddr(S.own[0]), ring = saddr(S.ring[0]);
        const uint64_t dk_k = desc_k(own), dk_v = desc_k(own + kTile<DP>);
        Ring<NS> r;
        int sq = 0, so = 0;  // ring slots of the tile at hand
        // s, and dp, of the next tile of the ring
        const auto form = [&](uint32_t cols, uint64_t key, uint64_t* full, int& slot) {
            slot = r.stage;
            if (!wait_warp(S, &S.full[slot], r.phase)) return false;
            product_cols<DP>(e, tmem + cols, key, desc_k(ring + slot * kTile<DP>));
            if (full) umma_commit(e, saddr(full));
            r.next();
            return true;
        };
        const auto add = [&](uint32_t cols, uint32_t p, int slot, bool more) {
            product_rows<DP>(e, tmem + cols, tmem + p, desc_mn(ring + slot * kTile<DP>), 0, 4, more);
            product_rows<DP>(e, tmem + cols, tmem + p + C::kHalf, desc_mn(ring + slot * kTile<DP>), 4, 4, true);
        };
        bool ok = wait_warp(S, &S.own_full, 0) && form(C::kS, dk_k, C::kApart ? nullptr : &S.s_full, sq) &&
                  form(C::kG, dk_v, C::kApart ? &S.s_full : &S.g_full, so);
        for (int i = 0; i < steps && ok; ++i) {
            const bool more = i + 1 < steps;
            int sq1 = 0, so1 = 0;
            if constexpr (C::kApart) {
                if (more)
                    ok = wait_warp(S, &S.taken, i & 1) && form(C::kS, dk_k, nullptr, sq1) &&
                         form(C::kG, dk_v, &S.s_full, so1);
                ok = ok && wait_warp(S, &S.ds_ready, i & 1);
                if (!ok) break;
                add(C::kDv, C::kP, so, i > 0);
                umma_commit(e, saddr(&S.empty[so]));
                add(C::kDk, C::kDs, sq, i > 0);
                umma_commit(e, saddr(&S.empty[sq]));
                umma_commit(e, saddr(&S.used));
            } else {
                ok = wait_warp(S, &S.p_ready, i & 1);
                if (!ok) break;
                add(C::kDv, C::kP, so, i > 0);
                umma_commit(e, saddr(&S.empty[so]));
                ok = (!more || form(C::kS, dk_k, &S.s_full, sq1)) && wait_warp(S, &S.ds_ready, i & 1);
                if (!ok) break;
                add(C::kDk, C::kDs, sq, i > 0);
                umma_commit(e, saddr(&S.empty[sq]));
                if (more) ok = form(C::kG, dk_v, &S.g_full, so1);
            }
            sq = sq1;
            so = so1;
        }
        // also after a wait that gave up: no MMA or commit is under way when the CTA leaves
        umma_commit(e, saddr(&S.done));
        mbar_wait<false>(&S.done, 0, &S.bad);
    } else if (!kElt && warp == 2) {
        for (int i = 0; i < steps; ++i) {
            const int st = i & 1;
            if (!wait_warp(S, &S.stat_empty[st], ((i >> 1) & 1) ^ 1)) break;
            int head, row;
            where(i, head, row);
            const int64_t at = head * a.tokens + token0 + row;
#pragma unroll
            for (int k = lane; k < kRows; k += 32) {
                const bool in = row + k < t.len;
                S.stat[st][0][k] = in ? a.lse[at + k] * -kLog2e : 0.0f;
                S.stat[st][1][k] = in ? -a.delta[at + k] : 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.stat_full[st]);
        }
    } else if (kElt) {
        const int half = (warp - kEltWarp0) / 4, thread = threadIdx.x - 32 * kEltWarp0, r = thread % kRows;
        const uint32_t lanes = (static_cast<uint32_t>(warp % 4 * 32) << 16) + tmem;
        const uint32_t ts = C::kS + 64 * half + lanes, tg = C::kG + 64 * half + lanes;
        const uint32_t tp = C::kP + C::kHalf * half + lanes, td = C::kDs + C::kHalf * half + lanes;
        const float2 c2 = both(a.scale_log2);
        bool ok = true;
        for (int i = 0; i < steps && ok; ++i) {
            const int st = i & 1;
            int head, row;
            where(i, head, row);
            const int queries = min(kRows, t.len - row);
            // columns of this half that see key r: [lo, hi)
            const bool masked = queries < kRows || (a.causal && row == row0);
            const int lo = (a.causal ? row0 + r - row : 0) - 64 * half, hi = queries - 64 * half;
            // the same for ds: 0 exactly for a query that sees one key only (the sequence's first one)
            const int lo_ds = row == 0 && (a.causal || t.len == 1) ? max(lo, 1 - 64 * half) : lo;
            ok = wait_warp(S, &S.stat_full[st], (i >> 1) & 1) && wait_warp(S, &S.s_full, i & 1);
            if (!ok) break;
            float p[64], g[C::kApart ? 64 : 32];
            tmem_ld64(ts, p);
            if constexpr (C::kApart) {
                tmem_ld64(tg, g);
                release_warp(&S.taken, lane);
            }
            const float4* nl = reinterpret_cast<const float4*>(&S.stat[st][0][64 * half]);
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
                const float4 l = nl[k / 4];
                const float2 x = fma2(make_float2(p[k], p[k + 1]), c2, make_float2(l.x, l.y));
                const float2 y = fma2(make_float2(p[k + 2], p[k + 3]), c2, make_float2(l.z, l.w));
                p[k] = ex2(x.x);
                p[k + 1] = ex2(x.y);
                p[k + 2] = ex2(y.x);
                p[k + 3] = ex2(y.y);
            }
            if (masked) {
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (k < lo || k >= hi) p[k] = 0.0f;
            }
            if constexpr (C::kApart) {
                // the products of the tile before have read p and ds
                if (i > 0) ok = wait_warp(S, &S.used, (i - 1) & 1);
                if (!ok) break;
            }
            store_cols64(tp, p);
            if (queries < kRows) {
                // query rows behind the sequence, of dO before dv reads it, of Q before dk does
                const int o = 2 * i + 1;
                ok = wait_warp(S, &S.full[o % NS], (o / NS) & 1);
                if (!ok) break;
                clear_rows<DP>(S.ring[o % NS], queries, thread, 256);
                clear_rows<DP>(S.ring[2 * i % NS], queries, thread, 256);
            }
            if constexpr (!C::kApart) {
                arrive_warp(&S.p_ready, lane);
                ok = wait_warp(S, &S.g_full, i & 1);
                if (!ok) break;
            }
            const float4* nd = reinterpret_cast<const float4*>(&S.stat[st][1][64 * half]);
#pragma unroll
            for (int h = 0; h < 64; h += 32) {
                if constexpr (!C::kApart) tmem_ld32(tg + h, reinterpret_cast<float(&)[32]>(g));
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const int n = h + k, m = C::kApart ? n : k;
                    const float4 d = nd[n / 4];
                    const float2 x = mul2(make_float2(p[n], p[n + 1]),
                                          add2(make_float2(g[m], g[m + 1]), make_float2(d.x, d.y)));
                    const float2 y = mul2(make_float2(p[n + 2], p[n + 3]),
                                          add2(make_float2(g[m + 2], g[m + 3]), make_float2(d.z, d.w)));
                    p[n] = x.x;
                    p[n + 1] = x.y;
                    p[n + 2] = y.x;
                    p[n + 3] = y.y;
                }
            }
            if (masked) {
                // not 0 times what the columns behind the sequence hold
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (k < lo_ds || k >= hi) p[k] = 0.0f;
            }
            store_cols64(td, p);
            arrive_warp(&S.ds_ready, lane);
            if (lane == 0) mbar_arrive(&S.stat_empty[st]);
        }
        if (ok && wait_warp(S, &S.done, 0))
            store_keys<DP>(a, S, t, kv, part, half, warp % 4, C::kDk, C::kDv, lanes, lane);
    }
}

// ---------------------------------------------------------------- side of the queries

// TMEM columns: s, dp, ds, Q (the left operand of s, so that its place in shared memory
// becomes one more slot of the ring), dq.
constexpr uint32_t kQs = 0, kQg = 128, kQds = 256, kQq = 320, kQdq = 384;

template <int DP, bool kElt>
__device__ __forceinline__ void queries_side(const AttnArgs& a, Smem<DP>& S, const CUtensorMap* mq,
                                             const CUtensorMap* mk, const CUtensorMap* mv, const CUtensorMap* mo,
                                             const AttnTile& t, int head, int warp, int lane, uint32_t tmem) {
    constexpr int NS = kStages<DP> + 1;  // slots from own[1] on; Q passes through the first
    // the tiles with most keys first
    const int token0 = static_cast<int>(t.begin);
    const int row0 = (a.causal ? (t.len - 1) / kRows - t.tile : t.tile) * kRows;
    const int keys_all = a.causal ? min(t.len, row0 + kRows) : t.len;
    const int steps = (keys_all + kRows - 1) / kRows;
    uint8_t* slots = S.own[1];
    if (!kElt && warp == 0) {
        const uint32_t e = elect_one();
        mbar_expect_tx_if(e, &S.own_full, kTile<DP>);
        load_tile<DP>(e, saddr(S.own[0]), mo, saddr(&S.own_full), head, token0 + row0);
        produce<DP, NS>(S, e, slots, 1 + 2 * steps, [&](int i, const CUtensorMap*& map, int& h, int& token) {
            const bool q = i == 0;
            map = q ? mq : i & 1 ? mk : mv;
            h = q ? head : head / a.group;
            token = q ? token0 + row0 : token0 + (i - 1) / 2 * kRows;
        });
    } else if (!kElt && warp == 1) {
        const uint32_t e = elect_one();
        const uint32_t base = saddr(slots);
        const uint64_t d_o = desc_k(saddr(S.own[0]));
        Ring<NS> r;
        r.next();
        int sk = 0;
        // s and dp of the ring's next two tiles
        const auto form = [&](int& slot) {
            slot = r.stage;
            if (!wait_warp(S, &S.full[slot], r.phase)) return false;
            product_cols_ts<DP>(e, tmem + kQs, tmem + kQq, desc_k(base + slot * kTile<DP>));
            r.next();
            if (!wait_warp(S, &S.full[r.stage], r.phase)) return false;
            product_cols<DP>(e, tmem + kQg, d_o, desc_k(base + r.stage * kTile<DP>));
            umma_commit(e, saddr(&S.s_full));
            umma_commit(e, saddr(&S.empty[r.stage]));
            r.next();
            return true;
        };
        bool ok = wait_warp(S, &S.q_ready, 0);
        if (ok && lane == 0) mbar_arrive(&S.empty[0]);
        __syncwarp();
        ok = ok && wait_warp(S, &S.own_full, 0) && form(sk);
        for (int i = 0; i < steps && ok; ++i) {
            int sk1 = 0;
            if (i + 1 < steps) ok = wait_warp(S, &S.taken, i & 1) && form(sk1);
            ok = ok && wait_warp(S, &S.ds_ready, i & 1);
            if (!ok) break;
            product_rows<DP>(e, tmem + kQdq, tmem + kQds, desc_mn(base + sk * kTile<DP>), 0, 8, i > 0);
            umma_commit(e, saddr(&S.empty[sk]));
            umma_commit(e, saddr(&S.used));
            sk = sk1;
        }
        umma_commit(e, saddr(&S.done));
        mbar_wait<false>(&S.done, 0, &S.bad);
    } else if (kElt) {
        const int half = (warp - kEltWarp0) / 4, thread = threadIdx.x - 32 * kEltWarp0, r = thread % kRows;
        const uint32_t lanes = (static_cast<uint32_t>(warp % 4 * 32) << 16) + tmem;
        const int row = row0 + r;
        const bool in = row < t.len;
        const int64_t token = t.begin + row;
        const float2 c2 = both(a.scale_log2);
        const float2 nl = both(in ? a.lse[head * a.tokens + token] * -kLog2e : 0.0f);
        const float2 nd = both(in ? -a.delta[head * a.tokens + token] : 0.0f);
        bool ok = wait_warp(S, &S.full[0], 0);
        if (ok) {
            // Q into TMEM, half of each row's 16-byte pieces per warpgroup (DP / 4 words)
            uint32_t w[32];
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const int piece = DP / 16 * half + k;
                const uint4 x = *reinterpret_cast<const uint4*>(slots + piece / 8 * kBox + r * 128 +
                                                                (piece % 8 ^ r % 8) * 16);
                w[4 * k] = x.x;
                w[4 * k + 1] = x.y;
                w[4 * k + 2] = x.z;
                w[4 * k + 3] = x.w;
            }
            if constexpr (DP == 128) tmem_st32(lanes + kQq + 32 * half, w);
            else tmem_st16(lanes + kQq + 16 * half, reinterpret_cast<const float(&)[16]>(w));
            // the loads above before the ring's next copy into this place
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            arrive_warp(&S.q_ready, lane);
        }
        for (int i = 0; i < steps && ok; ++i) {
            const int keys = min(kRows, t.len - i * kRows);
            ok = wait_warp(S, &S.s_full, i & 1);
            if (!ok) break;
            float p[64], g[64];
            tmem_ld64(lanes + kQs + 64 * half, p);
            tmem_ld64(lanes + kQg + 64 * half, g);
            release_warp(&S.taken, lane);
            const bool masked = keys < kRows || (a.causal && i + 1 == steps);
            // ds = 0 exactly for a row that sees one key only
            const int seen = ((a.causal ? row : t.len - 1) == 0 ? 0 : a.causal ? min(row + 1 - i * kRows, keys) : keys) -
                             64 * half;
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                float2 x = fma2(make_float2(p[k], p[k + 1]), c2, nl);
                x = mul2(make_float2(ex2(x.x), ex2(x.y)), add2(make_float2(g[k], g[k + 1]), nd));
                p[k] = x.x;
                p[k + 1] = x.y;
            }
            if (masked) {
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (k >= seen) p[k] = 0.0f;
            }
            if (keys < kRows) {
                // keys behind the sequence
                clear_rows<DP>(slots + (1 + 2 * i) % NS * kTile<DP>, keys, thread, 256);
            }
            // the product of the tile before has read ds
            if (i > 0) ok = wait_warp(S, &S.used, (i - 1) & 1);
            if (!ok) break;
            store_cols64(lanes + kQds + 32 * half, p);
            arrive_warp(&S.ds_ready, lane);
        }
        // a box of 64 columns each warpgroup
        if (64 * half < DP && ok && wait_warp(S, &S.done, 0)) {
            const int quarter = warp % 4;
            const int64_t out = t.begin + row0 + 32 * quarter;
            store_rows<1>(S.own[0] + half * kBox + quarter * 4096, kQdq + 64 * half + lanes, a.scale,
                          static_cast<__nv_bfloat16*>(a.out) + (out * a.heads + head) * a.dim + 64 * half,
                          static_cast<int64_t>(a.heads) * a.dim, t.len - row0 - 32 * quarter, a.dim - 64 * half, lane);
        }
    }
}

// ---------------------------------------------------------------- sequences of one tile

// A sequence of up to 128 tokens: one CTA per key head (or per part of its query heads)
// makes all three gradients, with s and dp formed once.  p and ds go through shared
// memory, where the products read them either way round: dq = ds k, dk = ds^T q, dv = p^T do.
// delta is the sum of p dp over the row at hand, not do . o: with few keys dp - delta
// is small beside dp, and the rounding of o to bf16 shows in it (2 to 16 keys: error of dq
// and dk 4e-3 to 5e-3 of their norm, with this 2.4e-3, which is that of ds and of the
// gradients themselves).
// TMEM: s, then dq; dp; dv; dk.  Shared memory: own = K, V; of the ring the last 64 KB hold p
// and ds, the others are slots for Q and dO of one head after the other.
template <int DP>
constexpr int kShortSlots = DP == 128 ? 3 : 4;

template <int DP, bool kElt>
__device__ __forceinline__ void short_side(const AttnArgs& a, Smem<DP>& S, const CUtensorMap* mq, const CUtensorMap* mk,
                                           const CUtensorMap* mv, const CUtensorMap* mo, const AttnTile& t, int kv,
                                           int part, int warp, int lane, uint32_t tmem) {
    constexpr int NS = kShortSlots<DP>;
    constexpr uint32_t kS = 0, kG = 128, kDv = 256, kDk = 256 + DP;
    const int token0 = static_cast<int>(t.begin);
    const int begin = attn_part(a.group, part, a.parts), steps = attn_part(a.group, part + 1, a.parts) - begin;
    const int head0 = kv * a.group + begin;
    uint8_t* p_tile = S.ring[kStages<DP> - 65536 / kTile<DP>];
    uint8_t* ds_tile = p_tile + 32768;
    if (!kElt && warp == 0) {
        const uint32_t e = elect_one();
        mbar_expect_tx_if(e, &S.own_full, 2 * kTile<DP>);
        load_tile<DP>(e, saddr(S.own[0]), mk, saddr(&S.own_full), kv, token0);
        load_tile<DP>(e, saddr(S.own[1]), mv, saddr(&S.own_full), kv, token0);
        produce<DP, NS>(S, e, S.ring[0], 2 * steps, [&](int i, const CUtensorMap*& map, int& head, int& token) {
            map = i & 1 ? mo : mq;
            head = head0 + i / 2;
            token = token0;
        });
    } else if (!kElt && warp == 1) {
        const uint32_t e = elect_one();
        const uint32_t own = saddr(S.own[0]), ring = saddr(S.ring[0]);
        const uint32_t p = saddr(p_tile), ds = saddr(ds_tile);
        bool ok = wait_warp(S, &S.own_full, 0);
        for (int i = 0; i < steps && ok; ++i) {
            const int nq = 2 * i, no = 2 * i + 1, sq = nq % NS, so = no % NS;
            // dq of the head before has been read
            ok = (i == 0 || wait_warp(S, &S.taken, (i - 1) & 1)) && wait_warp(S, &S.full[sq], (nq / NS) & 1);
            if (!ok) break;
            product_cols<DP>(e, tmem + kS, desc_k(ring + sq * kTile<DP>), desc_k(own));
            ok = wait_warp(S, &S.full[so], (no / NS) & 1);
            if (!ok) break;
            product_cols<DP>(e, tmem + kG, desc_k(ring + so * kTile<DP>), desc_k(own + kTile<DP>));
            umma_commit(e, saddr(&S.s_full));
            ok = wait_warp(S, &S.ds_ready, i & 1);
            if (!ok) break;
            product_tile<DP, true>(e, tmem + kDv, desc_mn(p), desc_mn(ring + so * kTile<DP>), i > 0);
            umma_commit(e, saddr(&S.empty[so]));
            product_tile<DP, true>(e, tmem + kDk, desc_mn(ds), desc_mn(ring + sq * kTile<DP>), i > 0);
            umma_commit(e, saddr(&S.empty[sq]));
            product_tile<DP, false>(e, tmem + kS, desc_k(ds), desc_mn(own), false);
            umma_commit(e, saddr(&S.used));
        }
        umma_commit(e, saddr(&S.done));
        mbar_wait<false>(&S.done, 0, &S.bad);
    } else if (kElt) {
        const int half = (warp - kEltWarp0) / 4, thread = threadIdx.x - 32 * kEltWarp0, r = thread % kRows;
        const int quarter = warp % 4;
        const uint32_t lanes = (static_cast<uint32_t>(quarter * 32) << 16) + tmem;
        const bool in = r < t.len;
        const int seen = (!in ? 0 : a.causal ? r + 1 : t.len) - 64 * half;  // columns of this half that row r sees
        // a row that sees one key only has ds = 0 exactly
        const int varied = (a.causal ? r : t.len - 1) == 0 ? 0 : seen;
        const float2 c2 = both(a.scale_log2);
        bool ok = wait_warp(S, &S.own_full, 0);
        if (ok && t.len < kRows) clear_rows<DP>(S.own[0], t.len, thread, 256);  // K: the rows of ds k
        for (int i = 0; i < steps && ok; ++i) {
            const int head = head0 + i;
            const float2 nl = both(in ? a.lse[head * a.tokens + t.begin + r] * -kLog2e : 0.0f);
            ok = wait_warp(S, &S.s_full, i & 1);
            if (!ok) break;
            float p[64], g[64];
            tmem_ld64(lanes + kS + 64 * half, p);
            tmem_ld64(lanes + kG + 64 * half, g);
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                const float2 x = fma2(make_float2(p[k], p[k + 1]), c2, nl);
                p[k] = ex2(x.x);
                p[k + 1] = ex2(x.y);
            }
            if (t.len < kRows || a.causal) {
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    if (k >= seen) p[k] = 0.0f;
                    if (k >= varied) g[k] = 0.0f;
                }
            }
            float2 sum2 = both(0.0f);
#pragma unroll
            for (int k = 0; k < 64; k += 2)
                sum2 = fma2(make_float2(p[k], p[k + 1]), make_float2(g[k], g[k + 1]), sum2);
            S.stat[i & 1][half][r] = sum2.x + sum2.y;
            release_warp(&S.p_ready, lane);  // both halves of every row's sum
            ok = wait_warp(S, &S.p_ready, i & 1);
            if (!ok) break;
            const float2 nd = both(-(S.stat[i & 1][0][r] + S.stat[i & 1][1][r]));
            // this row's 128 bytes of the half's box, in 16-byte pieces
            uint4* const prow = reinterpret_cast<uint4*>(p_tile + half * kBox + r * 128);
            uint4* const drow = reinterpret_cast<uint4*>(ds_tile + half * kBox + r * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t w[4], d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int n = 8 * c + 2 * k;
                    const float2 x = make_float2(p[n], p[n + 1]);
                    const float2 y = mul2(x, add2(make_float2(g[n], g[n + 1]), nd));
                    w[k] = pack_bf16x2(x.x, x.y);
                    d[k] = pack_bf16x2(y.x, y.y);
                }
                prow[c ^ (r % 8)] = make_uint4(w[0], w[1], w[2], w[3]);
                drow[c ^ (r % 8)] = make_uint4(d[0], d[1], d[2], d[3]);
            }
            if (t.len < kRows) {
                // rows behind the sequence, which meet zeros of p and ds
                clear_rows<DP>(S.ring[2 * i % NS], t.len, thread, 256);
                clear_rows<DP>(S.ring[(2 * i + 1) % NS], t.len, thread, 256);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            release_warp(&S.ds_ready, lane);
            ok = wait_warp(S, &S.used, i & 1);
            if (!ok) break;
            // p's rows of this warp are free again: dq passes through them
            if (64 * half < DP) {
                const int64_t out = t.begin + 32 * quarter;
                store_rows<1>(p_tile + half * kBox + quarter * 4096, lanes + kS + 64 * half, a.scale,
                              static_cast<__nv_bfloat16*>(a.out) + (out * a.heads + head) * a.dim + 64 * half,
                              static_cast<int64_t>(a.heads) * a.dim, t.len - 32 * quarter, a.dim - 64 * half, lane);
            }
            release_warp(&S.taken, lane);
        }
        if (ok && wait_warp(S, &S.done, 0)) store_keys<DP>(a, S, t, kv, part, half, quarter, kDk, kDv, lanes, lane);
    }
}

// The next of the launch's items that has something to do, by one warp: side of the keys,
// then of the queries, each with the heavy ones first, or (kWhole) sequences of one tile.
// A CTA begins with its own block index and then takes those of blocks not yet started.
template <int DP, bool kWhole>
__device__ __forceinline__ Item next_item(const AttnArgs& a, Smem<DP>& S, bool first, uint32_t& asked, int lane) {
    // tiles of the keys, tiles of the queries, rows to clear (once)
    const unsigned tiles = kWhole ? a.whole : a.slots;
    const unsigned keys_end = tiles * a.kv_heads * a.parts, tiles_end = keys_end + (kWhole ? 0 : tiles * a.heads);
    Item item;
    for (;;) {
        unsigned n = blockIdx.x;
        if (!first && !claim_block(&S.claim, &S.claimed, asked, n, &S.bad, lane)) return Item{NONE, 0, 0, 0, 0, 0};
        item = Item{NONE, 0, 0, 0, 0, 0};
        if (n >= tiles_end) {
            item.kind = CLEAR;
            item.tile = static_cast<int>(n - tiles_end);
            return item;
        }
        const bool keys = n < keys_end;
        const unsigned heads = keys ? a.kv_heads : a.heads, parts = keys ? a.parts : 1;
        n -= keys ? 0 : keys_end;
        const unsigned tile = n / parts, slot = tile / heads;
        item.part = static_cast<int>(n - tile * parts);
        item.head = static_cast<int>(tile - slot * heads);
        item.kind = kWhole ? WHOLE : keys ? KEYS : QUERIES;
        AttnTile t;
        bool any;
        if constexpr (kWhole) {
            t.begin = attn_offset(a, slot);
            t.len = static_cast<int32_t>(attn_offset(a, slot + 1) - t.begin);
            t.tile = 0;
            any = t.len > 0 && t.len <= kRows;
        } else {
            any = attn_find(a, static_cast<int>(slot), kRows, t) && (a.whole == 0 || t.len > kRows);
        }
        if (!any) {
            // a block that has nothing to do ends: the next of the grid follows it
            if (first) return Item{NONE, 0, 0, 0, 0, 0};
            continue;
        }
        item.begin = static_cast<int32_t>(t.begin);
        item.len = t.len;
        item.tile = t.tile;
        if (parts > 1 && part_begin(a, t, item.part) == part_begin(a, t, item.part + 1)) item.kind = CLEAR_PART;
        return item;
    }
}

template <int DP>
__device__ __forceinline__ void init_barriers(Smem<DP>& S, int lane, bool again) {
    // one barrier a lane, in the order of Smem
    uint64_t* bar = &S.own_full + lane;
    constexpr int n = static_cast<int>((offsetof(Smem<DP>, done) - offsetof(Smem<DP>, own_full)) / 8) + 1;
    static_assert(n <= 32, "a barrier a lane");
    if (lane >= n) return;
    if (again) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(saddr(bar)) : "memory");
    const bool warps = bar == &S.taken || bar == &S.p_ready || bar == &S.ds_ready || bar == &S.q_ready ||
                       (bar >= S.stat_empty && bar < S.stat_empty + 2);
    mbar_init(bar, warps ? kEltWarps : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// All items of a CTA, by the helper warps (kElt false) or the element-wise ones.
template <int DP, bool kElt, bool kWhole>
__device__ __forceinline__ void work(const AttnArgs& a, Smem<DP>& S, const CUtensorMap* mq, const CUtensorMap* mk,
                                     const CUtensorMap* mv, const CUtensorMap* mo, int warp, int lane, uint32_t tmem) {
    uint32_t asked = 0;  // requests for another block's index
    for (int n = 0;; ++n) {
        const Item& next = S.item[n & 1];
        // from one lane: uniform, as MMAs and copies take their operands
        const int kind = __shfl_sync(kFullMask, next.kind, 0), head = __shfl_sync(kFullMask, next.head, 0);
        const int part = __shfl_sync(kFullMask, next.part, 0);
        AttnTile t;
        t.begin = __shfl_sync(kFullMask, next.begin, 0);
        t.len = __shfl_sync(kFullMask, next.len, 0);
        t.tile = __shfl_sync(kFullMask, next.tile, 0);
        if (kind == NONE) return;
        if (kind == KEYS || kind == WHOLE || kind == QUERIES) {
            if constexpr (kWhole) short_side<DP, kElt>(a, S, mq, mk, mv, mo, t, head, part, warp, lane, tmem);
            else if (kind == KEYS) keys_side<DP, kElt>(a, S, mq, mk, mv, mo, t, head, part, warp, lane, tmem);
            else queries_side<DP, kElt>(a, S, mq, mk, mv, mo, t, head, warp, lane, tmem);
        } else if (kElt) {
            // rows of no sequence, or a part without steps
            if (kind == CLEAR_PART) {
                clear_part(a, t, head, part);
            } else {
                clear_rows_of(a, static_cast<__nv_bfloat16*>(a.out), a.heads, t.tile);
                if (a.parts > 1) {
                    for (int k = 0; k < 2 * a.parts; ++k) clear_rows_of(a, attn_partial(a, 0, k), a.kv_heads, t.tile);
                } else {
                    clear_rows_of(a, static_cast<__nv_bfloat16*>(a.dk), a.kv_heads, t.tile);
                    clear_rows_of(a, static_cast<__nv_bfloat16*>(a.dv), a.kv_heads, t.tile);
                }
            }
        }
        if (!kElt && warp == 0) {
            // not before this item's last loads are issued: an item taken early would wait here
            // while other SMs run dry
            const Item item = next_item<DP, kWhole>(a, S, false, asked, lane);
            if (lane == 0) S.item[(n + 1) & 1] = item;
        }
        // shared memory, TMEM and barriers pass to the next item
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        fence_before();
        __syncthreads();
        // from one lane, or the next item would run without uniform registers
        if (__shfl_sync(kFullMask, S.bad, 0) != 0) return;
        if (!kElt && warp == 2) init_barriers(S, lane, true);
        __syncthreads();
        fence_after();
    }
}

// kWhole: the sequences of one tile, in a launch of their own (as another kind of item
// of the other launch they slowed the others down by 3 to 10 %: the compiler's choices
// for one kind of loop suffer from the next).
template <int DP, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1)
    backward_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mo) {
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem<DP>& S = *reinterpret_cast<Smem<DP>*>(raw);
    const int warp = __shfl_sync(kFullMask, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    if (saddr(raw) % 1024 != 0) {  // no room was taken for aligning it here
        if (threadIdx.x == 0) atomicExch(&g_status, 1);
        return;
    }
    if (warp == 1) {
        tmem_alloc<kCols>(&S.tmem);
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
        uint32_t none = 0;
        const Item item = next_item<DP, kWhole>(a, S, true, none, lane);  // asks for no other block
        if (lane == 0) S.item[0] = item;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, S.tmem, 0);
    if (warp < kEltWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        work<DP, false, kWhole>(a, S, &mq, &mk, &mv, &mo, warp, lane, tmem);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsElt));
        work<DP, true, kWhole>(a, S, &mq, &mk, &mv, &mo, warp, lane, tmem);
    }
    fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && S.bad) atomicExch(&g_status, 1);
    if (warp == 1) {
        __syncwarp();
        fence_after();
        tmem_free<kCols>(tmem);
    }
}

template <int DP, bool kWhole>
cudaError_t attribute() {
    static_assert(sizeof(Smem<DP>) <= 232448, "shared memory of a block");
    return cudaFuncSetAttribute(backward_kernel<DP, kWhole>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(Smem<DP>)));
}

// Shared-memory attributes of all instances, once per device.
cudaError_t prepare() {
    static PerDevice cache;
    int dev = 0, ok = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cache.get(dev, &ok, [](int* out) {
        *out = 1;
        cudaError_t r = attribute<64, false>();
        if (r == cudaSuccess) r = attribute<64, true>();
        if (r == cudaSuccess) r = attribute<128, false>();
        if (r == cudaSuccess) r = attribute<128, true>();
        return r;
    });
}

template <int DP, bool kWhole>
cudaError_t launch(const AttnArgs& a, const AttnMaps& m, int64_t items, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(items));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem<DP>);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, backward_kernel<DP, kWhole>, a, m.q, m.k, m.v, m.d_o);
}

// Sequences of one tile have a launch of their own where the average one is no longer than this.  It is
// for delta's sake, not for time.  Measured, without -> with, by the average length (8192 tokens, 32/8
// heads of 128 | 12 of 64): 102 tokens 223 -> 222 us | 92 -> 95; 256: 210 -> 226 | 84 -> 95; 512: 242
// -> 247 | 91 -> 97; 683: 263 -> 267 | 96 -> 101; 1024: 347 -> 351 | 119 -> 124; 4096: 758 -> 762 | 231
// -> 238; four texts in 4096 tokens 61 -> 66 us with heads of 64.  Among longer sequences a short one takes
// delta from o like the others (two tokens: error of dq 4.6e-3 of its norm instead of 2.5e-3, more
// where one key has nearly all the weight), as the first rows of every causal sequence do.
constexpr int kShortAverage = 512;

template <int DP>
cudaError_t run(AttnArgs a, const AttnMaps& m, cudaStream_t s) {
    const int64_t longest = a.offsets ? a.tokens : a.length, average = a.offsets ? a.tokens / a.sequences : a.length;
    a.slots = longest <= kRows ? 0 : static_cast<int32_t>(attn_slots(a.tokens, a.sequences, kRows));
    a.whole = longest <= kRows || (a.offsets && average <= kShortAverage) ? a.sequences : 0;
    const int64_t keys = static_cast<int64_t>(a.kv_heads) * a.parts, both = a.heads + keys;
    cudaError_t e = cudaSuccess;
    if (a.whole > 0) e = launch<DP, true>(a, m, a.whole * keys + (a.slots > 0 ? 0 : a.fill), s);
    if (e == cudaSuccess && a.slots > 0) e = launch<DP, false>(a, m, a.slots * both + a.fill, s);
    return e;
}

}  // namespace
}  // namespace attn

cudaError_t attn_bwd_status_word(void** p) { return cudaGetSymbolAddress(p, attn::g_status); }

bool attn_tc_needs_delta(const AttnArgs& a) { return (a.offsets ? a.tokens : a.length) > attn::kRows; }

cudaError_t attn_tc_backward(const AttnArgs& a, const AttnMaps& m, cudaStream_t s) {
    const cudaError_t e = attn::prepare();
    if (e != cudaSuccess) return e;
    return a.dim <= 64 ? attn::run<64>(a, m, s) : attn::run<128>(a, m, s);
}

}  // namespace dmuon
