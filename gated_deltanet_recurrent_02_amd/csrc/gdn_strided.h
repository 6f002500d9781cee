// Checks of strided tensors of a call (gdn_rotary_api.cpp, gdn_scan_api.cpp): sizes, distinct elements
// of an output, and whether two tensors share bytes.
#pragma once

#include <cstdint>
#include <string>

#include "gdn_api_common.h"

namespace gdn {
namespace api {

// A tensor of up to three strided dimensions over rows of dense bytes. Dimensions of one element have no stride.
struct Strided {
    const char* name;
    uintptr_t base;
    int64_t n[3], stride[3];  // elements of each dimension, and its stride in bytes
    int64_t row;              // bytes of a row
    bool wanted;              // false: an absent optional tensor; it shares bytes with nothing

    bool empty() const { return !wanted || row == 0 || n[0] == 0 || n[1] == 0 || n[2] == 0; }
    // Bytes from the first element's start to the last one's end, over the strides below `limit`.
    int64_t span(int64_t limit) const {
        int64_t s = row;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && stride[i] < limit) s += (n[i] - 1) * stride[i];
        return s;
    }
};

constexpr int64_t kNoLimit = INT64_MAX;

// `strides` in elements of es bytes (nullptr: dense) of a tensor [n0][n1][n2][row]. Refuses negative strides,
// pointers off the element's alignment, NULL, and extents of 2^61 bytes or more.
inline gdn_status strided(const char* fn, const char* name, const void* p, const int64_t* strides, int dims, int64_t n0,
                          int64_t n1, int64_t n2, int64_t row, size_t es, Strided* out) {
    Strided& t = *out;
    t.name = name;
    t.base = reinterpret_cast<uintptr_t>(p);
    t.n[0] = n0; t.n[1] = n1; t.n[2] = n2;
    t.row = row * (int64_t)es;
    t.wanted = true;
    int64_t dense[3] = {n1 * n2 * row, n2 * row, row};
    int64_t total = t.row;
    for (int i = 0; i < 3; ++i) {
        const int64_t s = strides && i < dims ? strides[i] : dense[i];
        int64_t step = 0;
        if (t.n[i] <= 1) { t.stride[i] = 0; continue; }
        if (s < 0) return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + name + " has a negative stride");
        if (__builtin_mul_overflow(s, (int64_t)es, &t.stride[i]) || __builtin_mul_overflow(t.stride[i], t.n[i] - 1, &step) ||
            __builtin_add_overflow(total, step, &total) || total >= (int64_t(1) << 61))
            return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": size of " + name + " overflows");
    }
    if (t.empty()) return GDN_OK;
    if (!p) return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + name + " is NULL");
    if (t.base % es != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + name + " is not aligned to its element");
    return GDN_OK;
}

inline Strided absent(const char* name) { return Strided{name, 0, {0, 0, 0}, {0, 0, 0}, 0, false}; }

// A dense run of bytes as such a tensor.
inline Strided run_of(const char* name, const void* p, size_t bytes) {
    return Strided{name, reinterpret_cast<uintptr_t>(p), {1, 1, 1}, {0, 0, 0}, (int64_t)bytes, p != nullptr};
}

inline bool same_elements(const Strided& a, const Strided& b) {
    if (a.base != b.base || a.row != b.row) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || a.stride[i] != b.stride[i]) return false;
    return true;
}

// Whether a's elements are proved distinct: every stride covers all that the smaller ones reach.
inline bool distinct(const Strided& a) {
    if (a.empty()) return true;
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] <= 1) continue;
        if (a.stride[i] < a.span(a.stride[i])) return false;
        for (int j = 0; j < i; ++j)
            if (a.n[j] > 1 && a.stride[j] == a.stride[i]) return false;
    }
    return true;
}

// Whether a and b may share bytes. They do not where their ranges are apart, or where both repeat with one
// period (a stride that divides all larger ones) and occupy different parts of it: the q and k parts of a
// packed tensor.
inline bool may_share(const Strided& a, const Strided& b) {
    if (a.empty() || b.empty()) return false;
    if (a.base + (uintptr_t)a.span(kNoLimit) <= b.base || b.base + (uintptr_t)b.span(kNoLimit) <= a.base) return false;
    for (int c = 0; c < 6; ++c) {
        const Strided& of = c < 3 ? a : b;
        const int64_t period = of.n[c % 3] > 1 ? of.stride[c % 3] : 0;
        if (period <= 0) continue;
        auto repeats = [&](const Strided& t) {
            for (int i = 0; i < 3; ++i)
                if (t.n[i] > 1 && t.stride[i] >= period && t.stride[i] % period != 0) return false;
            return t.span(period) <= period;
        };
        if (!repeats(a) || !repeats(b)) continue;
        // b's start within a period that begins at a's
        const uint64_t up = (uint64_t)period;
        const uint64_t off = b.base >= a.base ? (b.base - a.base) % up : (up - (a.base - b.base) % up) % up;
        if (off >= (uint64_t)a.span(period) && off + (uint64_t)b.span(period) <= up) return false;
    }
    return true;
}

// `out` must have distinct elements and share none with the `count` others, apart from `in_place`, which it
// may be exactly.
inline gdn_status check_output(const char* fn, const Strided& out, const Strided* const* others, int count,
                               const Strided* in_place = nullptr) {
    if (out.empty()) return GDN_OK;
    if (!distinct(out))
        return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": elements of " + out.name + " overlap each other");
    for (int i = 0; i < count; ++i) {
        const Strided& o = *others[i];
        if (&o == &out || (&o == in_place && same_elements(out, o))) continue;
        if (may_share(out, o))
            return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + out.name + " overlaps " + o.name);
    }
    return GDN_OK;
}

}  // namespace api
}  // namespace gdn
