// Internal interface between the C-ABI layer (gdn_scan_api.cpp) and the kernels of the gated linear recurrence
// (gdn_scan.hip). Arguments are validated by the caller; the launchers select kernel instances and enqueue
// them on the given stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_launch.h"

namespace gdn {

// A tensor [B][T][C] with strides in elements, the last one 1.
struct RowsView {
    void* p;
    int64_t sb, st;
};

struct ScanArgs {
    int64_t B;
    int32_t T, C;
    DType act, state_dtype;
    RowsView x, a, b;          // b.p nullptr: beta = 1 - alpha
    const float* rate;         // [C] or nullptr (1)
    const int32_t* lengths;    // [B] or nullptr (T for all)
    void* state;               // forward: [B][C], in place
    RowsView o;
    float* checkpoints;        // [B][chunks][C] or nullptr; backward: read
    // backward
    const void* state0;
    const void* dstate;
    RowsView d_o, dx, da, db;
    void* dstate0;
    float* drate;
    float* ws;
};

constexpr int kScanChunk = 64;  // tokens from one kept state to the next, and of a workgroup's tile

inline int64_t scan_chunks(int32_t T) { return ((int64_t)T + kScanChunk - 1) / kScanChunk; }

// The workspace: eight counters for each direction, 128 bytes apart; values per sequence, chunk and channel at the tiles'
// edges (in rows of 16 bytes), the states unless the caller's checkpoints take them; and the maps of the tiles, two values
// per sequence, tile of at least 64 tokens and channel.
constexpr int kScanCounterStride = 32, kScanCounterFloats = 16 * kScanCounterStride;
inline size_t scan_values(int64_t B, int32_t T, int32_t C) { return ((size_t)B * scan_chunks(T) * C + 3) / 4 * 4; }
inline size_t scan_prefill_ws_floats(int64_t B, int32_t T, int32_t C) {
    return B == 0 || scan_chunks(T) <= 1 ? 0 : kScanCounterFloats + 3 * scan_values(B, T, C);
}
// The adjoints and the states at the edges, the maps of both directions, and the rates' gradient of every chunk.
inline size_t scan_backward_ws_floats(int64_t B, int32_t T, int32_t C) {
    return B == 0 || T == 0 ? 0 : kScanCounterFloats + 7 * scan_values(B, T, C);
}

hipError_t launch_scan_decode(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_prefill(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t stream);

}  // namespace gdn
