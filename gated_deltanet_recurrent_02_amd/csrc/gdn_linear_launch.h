// Internal interface between the C-ABI layer (gdn_linear_api.cpp) and the kernels of linear
// attention (gdn_linear.hip) and layer norm (gdn_norm.hip). Arguments are validated by the caller;
// the launchers select kernel instances and enqueue them on the given stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_launch.h"

namespace gdn {

struct LinearArgs {
    int64_t B;
    int32_t T, H, Hk, D;      // D = dk = dv
    const void* q;            // act [B][T][Hk][D]
    const void* k;            // act [B][T][Hk][D]
    const void* v;            // act [B][T][H][D]
    DType act;
    const float* decay;       // [H]
    const int32_t* lengths;   // [B] or nullptr (T for all)
    void* state;              // state dtype [B][H][D][D]
    DType state_dtype;
    void* o;                  // act [B][T][H][D]
    float scale;
    float* ws;                // workspace (prefill)
};

struct LinearBackwardArgs {
    int64_t B;
    int32_t T, H, Hk, D;
    const void* q;
    const void* k;
    const void* v;
    DType act;
    const float* decay;
    const int32_t* lengths;
    const void* state0;       // state dtype [B][H][D][D] or nullptr
    const void* d_o;          // act [B][T][H][D]
    const void* dstate;       // state dtype [B][H][D][D] or nullptr
    DType state_dtype;
    void* dq;                 // act [B][T][Hk][D]
    void* dk;                 // act [B][T][Hk][D]
    void* dv;                 // act [B][T][H][D]
    void* dstate0;            // state dtype [B][H][D][D] or nullptr
    float* ddecay;            // [H] or nullptr
    float scale;
    float* ws;                // workspace
};

// One sweep of linear attention (see gdn_linear.hip): N <- decay N + zscale z y^T, out = oscale N x, over
// the tensors [B][T][H / g][D] (head h reads head h / g of a tensor with group g).
struct Sweep {
    int32_t T, H;
    int32_t gx, gy, gz;
    const void* x;
    const void* y;
    const void* z;
    const float* decay;       // [H]
    const int32_t* lengths;   // [B] or nullptr
    const void* first;        // state before the sweep [B][H][D][D], or nullptr (zero)
    void* last;               // state after it, or nullptr (not wanted)
    void* out;                // [B][T][H][D]
    float zscale, oscale;
    bool reverse;             // backward in time
    bool transposed;          // `first` is read transposed
    bool out_f32;             // out is fp32 (else the activations' type)
    DType state_dtype;        // of first and last
};

// The chunked form of up to three sweeps over the same B, T, H and D, in one set of launches. Of three,
// sweep 1 has sweep 2's y and z exchanged and its first state transposed (dk and dv).
hipError_t launch_linear_chunk(const Sweep* sweeps, int n, int64_t B, int D, DType act, float* ws,
                               hipStream_t stream);

// The decay's gradient of a chunked call: partial sums, *parts of them per head and sequence, [*parts][B * H]
// after the states in ws (linear_tangent_state_floats).
hipError_t launch_linear_tangent(const LinearBackwardArgs& a, float* ws, int64_t* parts, hipStream_t stream);

// Which calls take the chunked form: runs of at least kLinearChunkMinTokens tokens whose rows of a
// chunk lie within 32 bits of each other (64 rows of H * D elements of 4 bytes); others go token by
// token. Token by token against chunked, H = 48, D = 128, bf16: prefill B = 1 T = 8 10.6 and 11.8 us,
// T = 12 14.0 and 11.9, T = 32 31.5 and 11.9; B = 64 T = 8 99 and 102 (fp32 98 and 100; fp16, D = 64 37 and
// 28), T = 32 235 and 114; backward B = 1 T = 8 19.1 and 13.5, B = 64 T = 8 195 and 153 (fp32 190 and 157).
constexpr int32_t kLinearChunkMinTokens = 8;
inline bool linear_chunked(int32_t T, int32_t H, int32_t D) {
    return T >= kLinearChunkMinTokens && (int64_t)H * D <= (int64_t(1) << 23);
}

// Pieces a sequence is split into when there are few heads: each starts from a state that a first
// pass over the pieces before it provides, at a little more than half the cost of the sweep itself. The
// pieces of all sweeps are to fill the 512 places of workgroups (two a CU), with at least two chunks
// each. Split against whole, D = 128, bf16, T = 4096: prefill of 48 heads in all 120 and 314 us, of 128
// 233 and 312, of 160 290 and 313; backward of 48 (144 sweeps) 243 and 310, of 56 (168) 264 and 310; fp16
// prefill of 160 419 and 516. Two pieces do not pay for the first pass: prefill of 176 heads 332 and 314
// (fp16 532 and 516), of 192 341 and 315, at T = 1000 111 and 87; backward of 60 326 and 310; 48 heads at
// T = 256 33 and 27 (fp32 47.5 and 47.3), backward 44 and 25. Narrow heads, of
// which a CU holds more, take the same rule though two would pay (192 of D = 16: 144 and 224; of D = 64,
// fp16: 274 and 318).
inline int32_t linear_segments(int64_t B, int32_t T, int32_t H, int sweeps) {
    const int64_t wgs = B * H * sweeps, chunks = ((int64_t)T + 63) / 64;
    int64_t n = 512 / wgs;
    if (n > chunks / 2) n = chunks / 2;
    return (int32_t)(n < 3 ? 1 : n);
}

struct NormArgs {
    int64_t rows;
    int32_t G, C;
    const void* x;
    DType dtype;
    const float* weight;      // [G][C] or nullptr
    const float* bias;        // [G][C] or nullptr
    void* y;
    float* mean;              // [rows] or nullptr
    float* rstd;              // [rows] or nullptr
    float eps;
};

struct NormBackwardArgs {
    int64_t rows;
    int32_t G, C;
    const void* dy;
    const void* x;
    DType dtype;
    const float* weight;      // [G][C] or nullptr
    const float* mean;        // [rows]
    const float* rstd;        // [rows]
    void* dx;
    float* dweight;           // [G][C] or nullptr
    float* dbias;             // [G][C] or nullptr
    float* ws;                // workspace, where dweight or dbias is wanted
};

// Workspace floats of the calls (host arithmetic only; no overflow below the callers' limits).
// A chunked call keeps a state for each sweep and segment where it has several segments or several
// sweeps (the gradients', which read states transposed).
inline size_t linear_segment_floats(int64_t B, int32_t T, int32_t H, int32_t D, int sweeps) {
    if (B == 0 || !linear_chunked(T, H, D)) return 0;
    const int32_t n = linear_segments(B, T, H, sweeps);
    return n > 1 || sweeps > 1 ? (size_t)sweeps * B * H * n * D * D : 0;
}

inline size_t linear_prefill_ws_floats(int64_t B, int32_t T, int32_t H, int32_t D) {
    return linear_segment_floats(B, T, H, D, 1);
}

// The chunked decay gradient's states (S and M of every segment); its partial sums lie after them.
inline size_t linear_tangent_state_floats(int64_t B, int32_t T, int32_t H, int32_t D) {
    return 2 * linear_segment_floats(B, T, H, D, 1);
}

// The fp32 dq and dk of every head where heads share q and k; then, one after the other in the same
// place, the sweeps' segment states and the decay gradient's states and partial sums (one a wave token by
// token; one a segment and head chunked).
inline size_t linear_backward_ws_floats(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t D) {
    const size_t partial = H != Hk ? 2 * (size_t)B * T * H * D : 0;
    const size_t states = linear_segment_floats(B, T, H, D, 3);
    const size_t segs = B > 0 ? linear_segments(B, T, H, 1) : 1, per = segs > (size_t)D / 8 ? segs : (size_t)D / 8;
    const size_t sums = linear_tangent_state_floats(B, T, H, D) + (size_t)B * H * per + 4;
    return partial + (sums > states ? sums : states);
}

// Slabs of rows that layer norm's parameter gradients are summed over before they are joined: no more
// than there are rows of a group, and slabs * G * C < 2^32 (a launch of one work-item each). Short
// affines take up to 1024 slabs, for enough workgroups (with 1024 against 256, 2^26 bf16 values in
// rows of 128: 85 and 181 us, of 1024: 85 and 150, of 4096: 98 and 133), long ones 256, so that the slabs'
// own traffic stays small (rows of 12288: 140 and 103 us).
constexpr int64_t kNormSlabs = 1024, kNormSlabsLong = 256, kNormSlabFloats = 1 << 22;
inline int32_t norm_slabs(int64_t rows, int32_t G, int32_t C) {
    const int64_t tokens = rows / G, GC = (int64_t)G * C, fit = kNormSlabFloats / GC;
    int64_t n = fit > kNormSlabs ? kNormSlabs : fit < kNormSlabsLong ? kNormSlabsLong : fit;
    if (n > (int64_t(1) << 31) / GC) n = (int64_t(1) << 31) / GC;  // G * C < 2^31
    return (int32_t)(tokens < n ? tokens : n);
}

inline size_t norm_backward_ws_floats(int64_t rows, int32_t G, int32_t C) {
    return 2 * (size_t)norm_slabs(rows, G, C) * G * C;
}

// All return hipSuccess or the launch error; nothing is synchronised.
hipError_t launch_linear_decode(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_prefill(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t stream);
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_layer_norm_backward(const NormBackwardArgs& a, hipStream_t stream);

}  // namespace gdn
