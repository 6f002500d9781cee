// Internal interface between the C-ABI layer (gdn_rotary_api.cpp) and the kernels of the rotation and the
// norm of queries and keys (gdn_rotary.hip). Arguments are validated by the caller; the launchers select
// kernel instances and enqueue them on the given stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_launch.h"

namespace gdn {

// A tensor [B][T][H][D] with strides in elements, the last one 1.
struct HeadsView {
    const void* p;
    int64_t sb, st, sh;
};

// Everything one of q and k has in a call.
struct RotarySet {
    HeadsView x;         // q or k (in rope's backward, the gradient to turn back)
    HeadsView dy;        // the gradient of the output (norm's backward)
    HeadsView y;         // written
    const float* w;      // weight or nullptr
    float* dw;           // its gradient or nullptr
};

struct RotaryArgs {
    int64_t B;
    int32_t T, Hq, Hk, D, R;
    DType dtype;
    RotarySet q, k;
    int32_t per_head;          // weights [H][D] rather than [D]
    float eps;
    const int32_t* positions;  // [B][T] or nullptr (0, 1, ...)
    const double* freqs;       // [R/2]
    float amplitude;
    int32_t interleaved, transposed;
    const int32_t* lengths;    // [B] or nullptr (T for all)
    float* ws;                 // workspace (norm's backward, where a dw is wanted)
};

// Slabs of tokens whose weight gradients are summed apart, and the workspace they take in all: enough to fill
// the card with few heads, and no more than 256 with many, whose workgroups lie along the heads too.
inline int64_t rotary_slabs(int64_t tokens, int64_t heads) {
    int64_t n = 16384 / heads;
    n = n < 256 ? 256 : (n > 1024 ? 1024 : n);
    return tokens < n ? tokens : n;
}
inline size_t rotary_backward_ws_floats(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D) {
    // every slab's sums of every head; one slab more than the kernels write, the size that callers have allocated so far
    const int64_t heads = (int64_t)Hq + Hk;
    return B * T == 0 ? 0 : (size_t)(rotary_slabs(B * T, heads) + 1) * (size_t)heads * (size_t)D;
}

hipError_t launch_rope(const RotaryArgs& a, hipStream_t stream);
hipError_t launch_qk_norm_rope(const RotaryArgs& a, hipStream_t stream);
hipError_t launch_qk_norm_rope_backward(const RotaryArgs& a, hipStream_t stream);

}  // namespace gdn
