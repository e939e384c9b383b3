// Host side of attention: argument checks, workspace layout, choice of kernels.
#include <algorithm>
#include <cmath>

#include "act.cuh"
#include "attn.h"
#include "checks.h"

namespace dmuon {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxSequences = int64_t(1) << 20;
constexpr int kMaxHeads = 1024, kMaxDim = 128;
// Blocks of a launch: 2^31 - 1, less those that clear rows.  (Key tiles shared by several
// blocks make fewer: there are at most 121 sequences then.)
constexpr int64_t kMaxBlocks = (int64_t(1) << 31) - 256;

bool sizes_ok(int64_t tokens, int64_t sequences, int64_t heads, int64_t kv_heads, int64_t dim) {
    return in_range(tokens, 0, kMaxTokens) && in_range(sequences, 1, kMaxSequences) && in_range(heads, 1, kMaxHeads) &&
           in_range(kv_heads, 1, heads) && heads % kv_heads == 0 && in_range(dim, 1, kMaxDim) &&
           (tokens / 32 + sequences) * (heads + kv_heads) < kMaxBlocks;
}

int set_heads(AttnHeads& h, const dmuon_heads_t* t, int64_t tokens, int64_t heads, int64_t dim, int es,
              const char* name, const char* where) {
    if (!t) return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": " + name + " is NULL");
    OPS_TRY(check_ptr(t->p, name, where, static_cast<size_t>(es)));
    const int64_t most = int64_t(1) << 36;
    if ((tokens > 1 && !in_range(t->token_stride, dim, most)) || (heads > 1 && !in_range(t->head_stride, dim, most)))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": strides of " + name + " must be at least dim, and at most 2^36");
    h.p = t->p;
    // a stride that no access uses has any value
    h.token = tokens > 1 ? t->token_stride : dim;
    h.head = heads > 1 ? t->head_stride : dim;
    return DMUON_OK;
}

// What both directions check, and the arguments they share.
int common(AttnArgs& a, const dmuon_heads_t* q, const dmuon_heads_t* k, const dmuon_heads_t* v,
           const int64_t* offsets, int64_t sequences, int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim,
           int32_t dtype, int32_t causal, float scale, const char* where) {
    if (!sizes_ok(tokens, sequences, heads, kv_heads, dim))
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": tokens must be in [0, 2^24], sequences in [1, 2^20], heads in [1, 1024] and "
                                         "a multiple of kv_heads, dim in [1, 128], and "
                                         "(tokens / 32 + sequences) * (heads + kv_heads) below 2^31 - 256");
    OPS_TRY(check_dtype(dtype, where));
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": scale must be finite and > 0");
    if (!offsets && tokens % sequences != 0)
        return fail(DMUON_ERR_INVALID_ARG,
                    std::string(where) + ": without offsets tokens must be a multiple of sequences");
    if (offsets) OPS_TRY(check_ptr(offsets, "offsets", where, 8));
    a.offsets = offsets;
    a.tokens = tokens;
    a.length = tokens / sequences;
    a.sequences = static_cast<int32_t>(sequences);
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.group = heads / kv_heads;
    a.dim = dim;
    a.causal = causal != 0;
    // Blocks that clear the rows of no sequence: one per SM where there are 128 rows for each.  Measured, 38 |
    // 152 | 608 blocks, backward, 32/8 heads of 128: 1384 of 16384 tokens in sequences 158 | 119 | 111 us, half
    // of 8192 326 | 318 | 313; without such rows they cost nothing that shows.
    a.fill = offsets ? static_cast<int32_t>(std::min<int64_t>(ceil_div(tokens, 128), 152)) : 0;
    a.scale = scale;
    a.scale_log2 = scale * kLog2e;
    if (tokens == 0) return DMUON_OK;
    const int es = dtype == DMUON_FP32 ? 4 : 2;
    OPS_TRY(set_heads(a.q, q, tokens, heads, dim, es, "q", where));
    OPS_TRY(set_heads(a.k, k, tokens, kv_heads, dim, es, "k", where));
    OPS_TRY(set_heads(a.v, v, tokens, kv_heads, dim, es, "v", where));
    return DMUON_OK;
}

// Whether TMA reads the rows in place.
bool tma_rows(const AttnHeads& h) {
    return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.token % 8 == 0 && h.head % 8 == 0;
}

// The tensor-core kernels take what TMA reads.
bool tensor_cores(const AttnArgs& a, int32_t dtype, bool backward) {
    return dtype == DMUON_BF16 && a.dim % 8 == 0 && tma_rows(a.q) && tma_rows(a.k) && tma_rows(a.v) &&
           (!backward || tma_rows(a.d_o));
}

// bf16 rows whose length is no multiple of 16 bytes are copied to rows padded with zeros for
// the tensor cores.  Measured, FFMA kernels -> copies, forward | backward: 8192 tokens, 8 heads of
// 50: 2526 -> 86 us | 9007 -> 277; 512 tokens, 8 heads of 50: 59 -> 18 | 144 -> 29; 100
// tokens, 12 heads of 50: 18 -> 16 | 58 -> 23; 37 tokens: 12 -> 16 | 40 -> 23.
bool packs(int64_t dim, int32_t dtype) { return dtype == DMUON_BF16 && dim % 8 != 0; }

int encode(CUtensorMap* map, const AttnHeads& h, int64_t tokens, int heads, int dim) {
    const auto enc = tensor_map_encoder();
    if (!enc) return fail(DMUON_ERR_CUDA, "cuTensorMapEncodeTiled entry point not found");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(h.head * 2), static_cast<cuuint64_t>(h.token * 2)};
    const cuuint32_t box[3] = {64, 1, 128}, estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(h.p), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(DMUON_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
    return DMUON_OK;
}

int set_maps(AttnMaps& m, const AttnArgs& a) {
    OPS_TRY(encode(&m.q, a.q, a.tokens, a.heads, a.dim));
    OPS_TRY(encode(&m.k, a.k, a.tokens, a.kv_heads, a.dim));
    OPS_TRY(encode(&m.v, a.v, a.tokens, a.kv_heads, a.dim));
    if (a.d_o.p) OPS_TRY(encode(&m.d_o, a.d_o, a.tokens, a.heads, a.dim));
    return DMUON_OK;
}

// The same of padded copies, which a launch makes in the workspace.
int set_packed_maps(AttnMaps& m, const AttnArgs& a, __nv_bfloat16* space, cudaStream_t s, const char* where) {
    AttnArgs b = a;
    b.dim = static_cast<int32_t>(up(a.dim, 8));
    for (AttnHeads* h : {&b.q, &b.k, &b.v, &b.d_o}) {
        if (!h->p) continue;
        const int64_t heads = h == &b.q || h == &b.d_o ? a.heads : a.kv_heads;
        *h = AttnHeads{space, heads * b.dim, b.dim};
        space += a.tokens * heads * b.dim;
    }
    OPS_CUDA(attn_pack(a, b, s));
    return set_maps(m, b);
}

// Blocks that share a key tile's queries.  The longest of them must not outlast the rest
// of the launch: about group * tiles steps, against the whole backward pass's steps over
// all SMs (a query tile's step costs 0.8 of a key tile's).  With sequences of the average
// length.  Measured, one part -> as chosen: 2048 tokens, 32 / 1 heads of 128: 640 -> 110 us;
// 1024 tokens, 16 / 2 heads of 128: 96 -> 38 us; fp32, 777 tokens, 6 / 2 heads of 80: 238 ->
// 72 us; 4096 tokens, 8 / 1 heads of 64: 3583 -> 1406 us.
constexpr int kMaxParts = 16;

int parts_of(int64_t sequences, int64_t tokens, int64_t heads, int64_t kv_heads, bool causal, bool tc) {
    const int64_t tile = tc ? 128 : 64, sms = 152;
    const double length = static_cast<double>(tokens) / static_cast<double>(sequences);
    const double tiles = std::max(1.0, std::ceil(length / static_cast<double>(tile)));
    const double pairs = causal ? tiles * (tiles + 1.0) / 2.0 : tiles * tiles;
    // FFMA: the factor that does best over all sizes (0.5 | 1.0 | 2.0, fp32: 2048 tokens, 32 / 4 heads of 64
    // 1414 | 1816 | 1815 us; 4096, 8 / 1 of 64 1406 | 1393 | 3584; 1024, 8 / 8 of 128 233 | 222 | 222)
    const double share = (tc ? 1.8 : 0.5) * static_cast<double>(heads * sequences) * pairs / sms;
    const double longest = static_cast<double>(heads / kv_heads) * tiles;
    // below 2.5 the partial sums cost more than the wait (2048 tokens, 8 heads of 128: 37 -> 60 us)
    const double ratio = longest / std::max(share, 2.0);
    return ratio < 2.5 ? 1 : static_cast<int>(std::min<double>({std::ceil(ratio), longest, kMaxParts}));
}

struct Layout {
    float* delta = nullptr;
    float* partial = nullptr;
    __nv_bfloat16* packed = nullptr;  // copies of q, k, v and d_o, where they are made
    int parts = 1;
    size_t bytes = 0;
    // the workspace serves either kind of kernels, causal or not
    Layout(char* base, int64_t sequences, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim, int32_t dtype,
           bool backward) {
        Arena a{base};
        if (backward) {
            delta = a.take<float>(tokens * heads);
            for (int k = 0; k < 4; ++k)
                parts = std::max(parts, parts_of(sequences, tokens, heads, kv_heads, (k & 1) != 0, (k & 2) != 0));
            if (parts > 1) partial = a.take<float>(2 * parts * tokens * kv_heads * dim);
        }
        if (packs(dim, dtype))
            packed = a.take<__nv_bfloat16>(tokens * ((backward ? 2 : 1) * heads + 2 * kv_heads) * up(dim, 8));
        bytes = a.off;
    }
};

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" size_t dmuon_attention_workspace_bytes(int64_t sequences, int64_t tokens, int32_t heads, int32_t kv_heads,
                                                  int32_t dim, int32_t dtype, int32_t backward) {
    if (!sizes_ok(tokens, sequences, heads, kv_heads, dim) ||
        check_dtype(dtype, "dmuon_attention_workspace_bytes") != DMUON_OK)
        return 0;
    return tokens == 0 ? 0 : Layout(nullptr, sequences, tokens, heads, kv_heads, dim, dtype, backward != 0).bytes;
}

extern "C" int dmuon_attention_forward(const dmuon_heads_t* q, const dmuon_heads_t* k, const dmuon_heads_t* v,
                                       const int64_t* offsets, int64_t sequences, void* o, float* lse, int64_t tokens,
                                       int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype, int32_t causal,
                                       float scale, void* workspace, size_t workspace_bytes, void* stream) {
    const char* where = "dmuon_attention_forward";
    AttnArgs a = {};
    OPS_TRY(common(a, q, k, v, offsets, sequences, tokens, heads, kv_heads, dim, dtype, causal, scale, where));
    if (tokens == 0) return DMUON_OK;
    OPS_TRY(check_ptr(o, "o", where));
    OPS_TRY(check_ptr(lse, "lse", where));
    const Layout L(static_cast<char*>(workspace), sequences, tokens, heads, kv_heads, dim, dtype, false);
    OPS_TRY(check_workspace(workspace, workspace_bytes, L.bytes, where));
    OPS_TRY(check_device(where));
    a.out = o;
    a.lse = lse;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pack = packs(dim, dtype);
    if (pack || tensor_cores(a, dtype, false)) {
        AttnMaps m = {};
        OPS_TRY(pack ? set_packed_maps(m, a, L.packed, s, where) : set_maps(m, a));
        OPS_CUDA(attn_tc_forward(a, m, s));
    } else {
        OPS_CUDA(attn_simt_forward(a, dtype == DMUON_FP32, s));
    }
    return DMUON_OK;
}

extern "C" int dmuon_attention_backward(const dmuon_heads_t* d_o, const dmuon_heads_t* q, const dmuon_heads_t* k,
                                        const dmuon_heads_t* v, const void* o, const float* lse,
                                        const int64_t* offsets, int64_t sequences, void* dq, void* dk, void* dv,
                                        int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                                        int32_t causal, float scale, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    const char* where = "dmuon_attention_backward";
    AttnArgs a = {};
    OPS_TRY(common(a, q, k, v, offsets, sequences, tokens, heads, kv_heads, dim, dtype, causal, scale, where));
    if (tokens == 0) return DMUON_OK;
    const bool f32 = dtype == DMUON_FP32;
    OPS_TRY(set_heads(a.d_o, d_o, tokens, heads, dim, f32 ? 4 : 2, "d_o", where));
    OPS_TRY(check_ptr(o, "o", where));
    OPS_TRY(check_ptr(lse, "lse", where));
    OPS_TRY(check_ptr(dq, "dq", where));
    OPS_TRY(check_ptr(dk, "dk", where));
    OPS_TRY(check_ptr(dv, "dv", where));
    const Layout L(static_cast<char*>(workspace), sequences, tokens, heads, kv_heads, dim, dtype, true);
    OPS_TRY(check_workspace(workspace, workspace_bytes, L.bytes, where));
    OPS_TRY(check_device(where));
    a.o = o;
    a.lse = const_cast<float*>(lse);
    a.delta = L.delta;
    a.out = dq;
    a.dk = dk;
    a.dv = dv;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pack = packs(dim, dtype), tc = pack || tensor_cores(a, dtype, true);
    a.parts = parts_of(sequences, tokens, heads, kv_heads, a.causal != 0, tc);
    a.partial = L.partial;
    // (bf16 rows of the FFMA kernels and sequences of one tile: made there)
    if (tc ? attn_tc_needs_delta(a) : f32) OPS_CUDA(attn_delta(a, f32, s));
    if (tc) {
        AttnMaps m = {};
        OPS_TRY(pack ? set_packed_maps(m, a, L.packed, s, where) : set_maps(m, a));
        OPS_CUDA(attn_tc_backward(a, m, s));
    } else {
        OPS_CUDA(attn_simt_backward(a, f32, s));
    }
    if (a.parts > 1) OPS_CUDA(attn_join(a, f32, s));
    return DMUON_OK;
}
