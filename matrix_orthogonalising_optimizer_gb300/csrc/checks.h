// Argument checks and workspace layout that the operators' entry points share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>
#include <string>

#include "dmuon.h"
#include "internal.h"
#include "ops.h"

namespace dmuon {
namespace {

[[maybe_unused]] int fail(int code, const std::string& msg) {
    set_last_error(msg);
    return code;
}

#define OPS_CUDA(call)                                                                                       \
    do {                                                                                                     \
        const cudaError_t e_ = (call);                                                                       \
        if (e_ != cudaSuccess) return fail(DMUON_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e_)); \
    } while (0)
#define OPS_TRY(call)                       \
    do {                                    \
        const int r_ = (call);              \
        if (r_ != DMUON_OK) return r_;      \
    } while (0)

[[maybe_unused]] int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
[[maybe_unused]] int64_t ceil_div(int64_t v, int64_t a) { return (v + a - 1) / a; }

struct Arena {
    char* base;
    size_t off = 0;
    template <typename T>
    T* take(int64_t count) {
        T* p = reinterpret_cast<T*>(base + off);  // only offsets are used when base is null
        off += static_cast<size_t>(up(count * static_cast<int64_t>(sizeof(T)), 256));
        return p;
    }
};

[[maybe_unused]] int check_dtype(int32_t dtype, const char* where) {
    if (dtype != DMUON_BF16 && dtype != DMUON_FP32)
        return fail(DMUON_ERR_UNSUPPORTED_DTYPE, std::string(where) + ": dtype must be DMUON_BF16 or DMUON_FP32");
    return DMUON_OK;
}

[[maybe_unused]] int check_ptr(const void* p, const char* name, const char* where, size_t align = 16) {
    if (!p) return fail(DMUON_ERR_INVALID_ARG, std::string(where) + ": " + name + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) % align)
        return fail(DMUON_ERR_ALIGN,
                    std::string(where) + ": " + name + " is not " + std::to_string(align) + "-byte aligned");
    return DMUON_OK;
}

[[maybe_unused]] int check_workspace(const void* ws, size_t have, size_t need, const char* where) {
    if (need == 0) return DMUON_OK;
    if (!ws) return fail(DMUON_ERR_NO_WORKSPACE, std::string(where) + ": workspace is NULL");
    if (reinterpret_cast<uintptr_t>(ws) % 256)
        return fail(DMUON_ERR_ALIGN, std::string(where) + ": workspace is not 256-byte aligned");
    if (have < need)
        return fail(DMUON_ERR_WORKSPACE_TOO_SMALL, std::string(where) + ": workspace of " + std::to_string(have) +
                                                       " bytes, " + std::to_string(need) + " needed");
    return DMUON_OK;
}

[[maybe_unused]] bool in_range(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

// The driver's tensor-map encoder; NULL if it has none.
[[maybe_unused]] PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)
                   : nullptr;
    }();
    return enc;
}

[[maybe_unused]] int check_device(const char* where) {
    static PerDevice cache;  // compute capability, 10 major + minor
    int dev = 0, cc = 0;
    OPS_CUDA(cudaGetDevice(&dev));
    OPS_CUDA(cache.get(dev, &cc, [&](int* out) {
        int major = 0, minor = 0;
        cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        *out = 10 * major + minor;
        return e;
    }));
    if (cc != 103) return fail(DMUON_ERR_UNSUPPORTED_DEVICE, std::string(where) + ": needs an sm_103 GPU");
    return DMUON_OK;
}

}  // namespace
}  // namespace dmuon
