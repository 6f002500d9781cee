// Device helpers shared by gdn_linear.hip, gdn_norm.hip, gdn_rotary.hip and gdn_scan.hip: element types, vector
// memory access and sums over lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Storage element types: float (fp32), uint16_t (bf16 bits), _Float16 (fp16). get widens exactly;
// pack rounds two floats to nearest even (v_cvt_pk_bf16_f32, v_cvt_pk_f16_f32).
template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float get(const uint32_t* w, int e) { return __uint_as_float(w[e]); }
};
template <> struct Elem<uint16_t> {
    static __device__ __forceinline__ float get(const uint32_t* w, int e) {
        const uint32_t x = w[e >> 1];
        return __uint_as_float((e & 1) ? (x & 0xffff0000u) : (x << 16));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const f32x2_t v = {lo, hi};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
    }
};
template <> struct Elem<_Float16> {
    static __device__ __forceinline__ float get(const uint32_t* w, int e) {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, w[e >> 1]);
        return (float)((e & 1) ? h.y : h.x);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const f32x2_t v = {lo, hi};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
    }
};

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<uint16_t>(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
template <> __device__ __forceinline__ float to_f32<_Float16>(_Float16 x) { return (float)x; }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t from_f32<uint16_t>(float x) {
    return (uint16_t)(Elem<uint16_t>::pack(x, 0.0f) & 0xffffu);
}
template <> __device__ __forceinline__ _Float16 from_f32<_Float16>(float x) {
    return __builtin_bit_cast(_Float16, (uint16_t)(Elem<_Float16>::pack(x, 0.0f) & 0xffffu));
}

// N contiguous elements of T as raw words; p is aligned to min(16, N * sizeof(T)) bytes.
template <typename T, int N>
struct Run {
    static constexpr int BYTES = N * (int)sizeof(T);
    static constexpr int WORDS = (BYTES + 3) / 4;
    uint32_t w[WORDS];

    template <bool NT = false>
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (BYTES >= 16) {
            static_assert(BYTES % 16 == 0, "run length");
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const u32x4* a = (const u32x4*)p + i;
                const u32x4 x = NT ? __builtin_nontemporal_load(a) : *a;
                w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
            }
        } else if constexpr (BYTES == 8) {
            const u32x2* a = (const u32x2*)p;
            const u32x2 x = NT ? __builtin_nontemporal_load(a) : *a;
            w[0] = x.x; w[1] = x.y;
        } else if constexpr (BYTES == 4) {
            w[0] = NT ? __builtin_nontemporal_load((const uint32_t*)p) : *(const uint32_t*)p;
        } else {
            static_assert(BYTES == 2, "run length");
            w[0] = NT ? __builtin_nontemporal_load((const uint16_t*)p) : *(const uint16_t*)p;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int e) const { return Elem<T>::get(w, e); }
    __device__ __forceinline__ void set(const float* x) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = __float_as_uint(x[e]);
        } else if constexpr (N == 1) {
            w[0] = Elem<T>::pack(x[0], 0.0f) & 0xffffu;
        } else {
#pragma unroll
            for (int e = 0; e < N; e += 2) w[e / 2] = Elem<T>::pack(x[e], x[e + 1]);
        }
    }
    template <bool NT = false>
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const u32x4 v = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
                if (NT) __builtin_nontemporal_store(v, (u32x4*)p + i); else ((u32x4*)p)[i] = v;
            }
        } else if constexpr (BYTES == 8) {
            const u32x2 v = {w[0], w[1]};
            if (NT) __builtin_nontemporal_store(v, (u32x2*)p); else *(u32x2*)p = v;
        } else if constexpr (BYTES == 4) {
            *(uint32_t*)p = w[0];
        } else {
            *(uint16_t*)p = (uint16_t)w[0];
        }
    }
};

// ------------------------------------------------------------------------ sums over lanes

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float x) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

// Sum over aligned groups of N lanes (a power of two up to 64); every lane gets the same value, in
// an order that does not depend on the lane.
template <int N>
__device__ __forceinline__ float lane_sum(float x) {
    if constexpr (N >= 2) x += dpp_mov<0xB1>(x);    // quad_perm [1,0,3,2]: lane ^ 1
    if constexpr (N >= 4) x += dpp_mov<0x4E>(x);    // quad_perm [2,3,0,1]: lane ^ 2
    if constexpr (N >= 8) x += dpp_mov<0x141>(x);   // row_half_mirror: i <- 7 - i in 8 lanes
    if constexpr (N >= 16) x += dpp_mov<0x140>(x);  // row_mirror: i <- 15 - i in 16 lanes
    if constexpr (N >= 32) x += __shfl_xor(x, 16);
    if constexpr (N >= 64) x += __shfl_xor(x, 32);
    return x;
}

// Tokens of sequence b, clamped to [0, T].
__device__ __forceinline__ int tokens_of(const int32_t* lengths, int64_t b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace
}  // namespace gdn
