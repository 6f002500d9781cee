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
size_t linear_prefill_ws_floats(int64_t B, int32_t T, int32_t H, int32_t D);
size_t linear_backward_ws_floats(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t D);
size_t norm_backward_ws_floats(int64_t rows, int32_t G, int32_t C);

// All return hipSuccess or the launch error; nothing is synchronised.
hipError_t launch_linear_decode(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_prefill(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t stream);
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_layer_norm_backward(const NormBackwardArgs& a, hipStream_t stream);

}  // namespace gdn
