// Argument checks and error reporting shared by the C-ABI files (gdn_api.cpp, gdn_linear_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <string>
#include <utility>

#include "gdn.h"
#include "gdn_launch.h"

namespace gdn {

// The calling thread's error text (gdn_last_error).
std::string& last_error();

namespace api {

inline gdn_status fail(gdn_status s, const std::string& msg) {
    last_error() = msg;
    return s;
}

inline gdn_status fail_hip(const char* what, hipError_t e) {
    last_error() = std::string(what) + ": " + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")";
    return GDN_ERR_HIP;
}

inline bool supported_dim(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool valid_dtype(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16 || t == GDN_F16; }
inline size_t dtype_bytes(gdn_dtype t) { return t == GDN_F32 ? 4 : 2; }
inline gdn::DType to_dtype(gdn_dtype t) {
    return t == GDN_F32 ? gdn::DType::F32 : (t == GDN_BF16 ? gdn::DType::BF16 : gdn::DType::F16);
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// a * b with overflow detection on size_t.
inline bool mul_ok(size_t a, size_t b, size_t* out) { return !__builtin_mul_overflow(a, b, out); }

struct Range {
    const char* name;
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range(const char* name, const void* p, size_t bytes) {
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, lo + bytes};
}

inline bool overlaps(const Range& a, const Range& b) {
    return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

// Shape checks shared by the two step functions. Returns GDN_OK, or a failure with message.
inline gdn_status check_shape(const char* fn, int64_t B, int32_t T, int32_t H, int32_t dk, int32_t dv) {
    if (B < 0 || T < 0) return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": B and T must be >= 0");
    if (H < 1) return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": H must be >= 1");
    if (dk < 1 || dv < 1) return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": dk and dv must be >= 1");
    if (dk != dv || !supported_dim(dk))
        return fail(GDN_ERR_UNSUPPORTED,
                    std::string(fn) + ": supported head dims are dk == dv in {16, 32, 64, 128}, got dk=" +
                        std::to_string(dk) + " dv=" + std::to_string(dv));
    if (B * (int64_t)H >= (int64_t(1) << 31))
        return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": B * H must be < 2^31");
    if (B * (int64_t)H * gdn::kThreadsPerHeadPerDim * dk >= gdn::kMaxWorkItems)
        return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": B * H * 8 * dk must be < 2^32 (one dispatch)");
    return GDN_OK;
}

inline gdn_status check_ptrs(const char* fn, std::initializer_list<std::pair<const char*, const void*>> ps) {
    for (auto& p : ps) {
        if (p.second == nullptr)
            return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + p.first + " is NULL");
        if (!aligned16(p.second))
            return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + p.first + " is not 16-byte aligned");
    }
    return GDN_OK;
}

inline gdn_status check_disjoint(const char* fn, const Range& out, std::initializer_list<Range> others) {
    for (auto& r : others)
        if (overlaps(out, r))
            return fail(GDN_ERR_INVALID_ARGUMENT,
                        std::string(fn) + ": " + out.name + " overlaps " + r.name);
    return GDN_OK;
}

}  // namespace api
}  // namespace gdn
