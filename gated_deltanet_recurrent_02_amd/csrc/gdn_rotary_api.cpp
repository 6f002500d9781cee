// C-ABI entry points declared in include/gdn_rotary.h (the rotation and the norm of queries and keys): host-side
// validation, then kernel launches on the caller's stream. Nothing here synchronises or allocates device memory.

#include "gdn_rotary.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "gdn_api_common.h"
#include "gdn_rotary_launch.h"
#include "gdn_strided.h"

using namespace gdn::api;

namespace {

constexpr int32_t kMaxHeadDim = 512;
constexpr int64_t kMaxHeads = 1 << 14;

enum class Kind { ROPE, NORM, NORM_BACKWARD };

// One tensor as a caller passes it.
struct Raw {
    const char* name;
    const void* p;
    const int64_t* strides;
};

// One of q and k as a caller passes it.
struct RawSet {
    Raw x, dy, y;
    const char *weight_name, *grad_name;
    const float* weight;
    float* grad;
};

struct Call {
    const char* fn;
    Kind kind;
    int64_t B;
    int32_t T, Hq, Hk, D, R;
    int dtype;
    RawSet set[2];
    int32_t per_head;
    float eps;
    const int32_t* positions;
    const double* freqs;
    float amplitude;
    int32_t interleaved;
    bool transposed;
    const int32_t* lengths;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
};

gdn_status check_sizes(const char* fn, int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D) {
    if (B < 0 || T < 0) return invalid(fn, "B and T must be >= 0");
    if (Hq < 1 || Hk < 0) return invalid(fn, "Hq must be >= 1 and Hk >= 0");
    if (D < 1) return invalid(fn, "D must be >= 1");
    if (D > kMaxHeadDim) return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": D must be <= 512");
    if ((int64_t)Hq + Hk > kMaxHeads) return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": Hq + Hk must be <= 16384");
    if (B >= (int64_t(1) << 31) || B * T >= (int64_t(1) << 31))
        return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": B * T must be < 2^31");
    return GDN_OK;
}

gdn::HeadsView view(const Strided& t, size_t es) {
    return gdn::HeadsView{reinterpret_cast<const void*>(t.base), t.stride[0] / (int64_t)es, t.stride[1] / (int64_t)es,
                          t.stride[2] / (int64_t)es};
}

gdn_status run(const Call& c) {
    const char* fn = c.fn;
    gdn_status s = check_sizes(fn, c.B, c.T, c.Hq, c.Hk, c.D);
    if (s != GDN_OK) return s;
    if (c.R < 0 || c.R > c.D || c.R % 2 != 0) return invalid(fn, "R must be even and in [0, D]");
    if (!valid_code(c.dtype)) return invalid(fn, "bad dtype");
    if (c.kind != Kind::ROPE && !(c.eps >= 0.0f)) return invalid(fn, "eps must be >= 0");
    if (!std::isfinite(c.amplitude)) return invalid(fn, "amplitude must be finite");
    const bool empty = c.B == 0 || c.T == 0, backward = c.kind == Kind::NORM_BACKWARD;
    const int sets = c.Hk ? 2 : 1;
    bool grads = false;
    for (int i = 0; i < sets; ++i) grads = grads || c.set[i].grad;
    if (empty && !grads) return GDN_OK;

    const size_t es = c.dtype == GDN_F32 ? 4 : 2;
    const size_t need = grads && !empty ? gdn::rotary_backward_ws_floats(c.B, c.T, c.Hq, c.Hk, c.D) * sizeof(float) : 0;
    Strided x[2], dy[2], y[2], weight[2], grad[2];
    for (int i = 0; i < 2; ++i) {
        const RawSet& r = c.set[i];
        x[i] = absent(r.x.name); dy[i] = absent(r.dy.name); y[i] = absent(r.y.name);
        weight[i] = absent(r.weight_name); grad[i] = absent(r.grad_name);
        if (i >= sets) continue;
        const int32_t H = i ? c.Hk : c.Hq;
        const size_t params = (size_t)(c.per_head ? H : 1) * c.D * sizeof(float);
        if (!empty) {
            s = strided(fn, r.x.name, r.x.p, r.x.strides, 3, c.B, c.T, H, c.D, es, &x[i]);
            if (s != GDN_OK) return s;
            if (backward) {
                s = strided(fn, r.dy.name, r.dy.p, r.dy.strides, 3, c.B, c.T, H, c.D, es, &dy[i]);
                if (s != GDN_OK) return s;
            }
            s = strided(fn, r.y.name, r.y.p, r.y.strides, 3, c.B, c.T, H, c.D, es, &y[i]);
            if (s != GDN_OK) return s;
        }
        s = check_optional(fn, r.weight_name, r.weight);
        if (s != GDN_OK) return s;
        s = check_optional(fn, r.grad_name, r.grad);
        if (s != GDN_OK) return s;
        weight[i] = run_of(r.weight_name, r.weight, params);
        grad[i] = run_of(r.grad_name, r.grad, params);
    }
    s = check_optional(fn, "positions", c.positions);
    if (s != GDN_OK) return s;
    if (c.R > 0 && !empty) {
        s = check_ptrs(fn, {{"freqs", c.freqs}});
        if (s != GDN_OK) return s;
    }
    s = check_optional(fn, "lengths", c.lengths);
    if (s != GDN_OK) return s;
    s = check_workspace(fn, c.workspace, c.workspace_bytes, need);
    if (s != GDN_OK) return s;

    const Strided positions = run_of("positions", c.positions, empty ? 0 : (size_t)c.B * c.T * 4);
    const Strided freqs = run_of("freqs", c.R > 0 ? c.freqs : nullptr, (size_t)c.R / 2 * 8);
    const Strided lengths = run_of("lengths", c.lengths, (size_t)c.B * 4);
    const Strided workspace = run_of("workspace", need ? c.workspace : nullptr, need);
    const Strided* all[] = {&x[0], &x[1], &dy[0], &dy[1], &weight[0], &weight[1], &positions, &freqs, &lengths,
                            &y[0], &y[1], &grad[0], &grad[1], &workspace};
    const int count = sizeof(all) / sizeof(all[0]);
    for (int i = 0; i < 2; ++i) {
        s = check_output(fn, y[i], all, count, backward ? &dy[i] : &x[i]);
        if (s != GDN_OK) return s;
        s = check_output(fn, grad[i], all, count);
        if (s != GDN_OK) return s;
    }
    s = check_output(fn, workspace, all, count);
    if (s != GDN_OK) return s;

    gdn::RotaryArgs a{};
    a.B = c.B; a.T = c.T; a.Hq = c.Hq; a.Hk = c.Hk; a.D = c.D; a.R = c.R;
    a.dtype = to_dtype((gdn_dtype)c.dtype);
    for (int i = 0; i < sets; ++i) {
        gdn::RotarySet& t = i ? a.k : a.q;
        t.x = view(x[i], es); t.dy = view(dy[i], es); t.y = view(y[i], es);
        t.w = c.set[i].weight; t.dw = c.set[i].grad;
    }
    a.per_head = c.per_head != 0;
    a.eps = c.eps;
    a.positions = c.positions; a.freqs = c.freqs; a.amplitude = c.amplitude;
    a.interleaved = c.interleaved != 0; a.transposed = c.transposed;
    a.lengths = c.lengths;
    a.ws = static_cast<float*>(c.workspace);
    hipStream_t st = reinterpret_cast<hipStream_t>(c.stream);
    hipError_t e;
    switch (c.kind) {
        case Kind::ROPE: e = gdn::launch_rope(a, st); break;
        case Kind::NORM: e = gdn::launch_qk_norm_rope(a, st); break;
        default: e = gdn::launch_qk_norm_rope_backward(a, st); break;
    }
    if (e != hipSuccess) return fail_hip((std::string(fn) + ": kernel launch").c_str(), e);
    return GDN_OK;
}

RawSet set_of(const char* x_name, const void* x, const int64_t* xs, const char* y_name, const void* y, const int64_t* ys) {
    return RawSet{{x_name, x, xs}, {"", nullptr, nullptr}, {y_name, y, ys}, "", "", nullptr, nullptr};
}

}  // namespace

extern "C" {

gdn_status gdn_rope(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                    gdn_dtype dtype, const void* q, const int64_t* q_strides, const void* k,
                    const int64_t* k_strides, const int32_t* positions, const double* freqs,
                    float amplitude, int32_t interleaved, const int32_t* lengths, void* q_out,
                    const int64_t* q_out_strides, void* k_out, const int64_t* k_out_strides,
                    void* stream) {
    const int code = dtype_code(dtype);
    return guarded([&] {
        return run(Call{"gdn_rope", Kind::ROPE, B, T, Hq, Hk, D, R, code,
                        {set_of("q", q, q_strides, "q_out", q_out, q_out_strides),
                         set_of("k", k, k_strides, "k_out", k_out, k_out_strides)},
                        0, 0.0f, positions, freqs, amplitude, interleaved, false, lengths, nullptr, 0, stream});
    });
}

gdn_status gdn_rope_backward(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                             gdn_dtype dtype, const void* dq, const int64_t* dq_strides,
                             const void* dk, const int64_t* dk_strides, const int32_t* positions,
                             const double* freqs, float amplitude, int32_t interleaved,
                             const int32_t* lengths, void* q_out, const int64_t* q_out_strides,
                             void* k_out, const int64_t* k_out_strides, void* stream) {
    const int code = dtype_code(dtype);
    return guarded([&] {
        return run(Call{"gdn_rope_backward", Kind::ROPE, B, T, Hq, Hk, D, R, code,
                        {set_of("dq", dq, dq_strides, "q_out", q_out, q_out_strides),
                         set_of("dk", dk, dk_strides, "k_out", k_out, k_out_strides)},
                        0, 0.0f, positions, freqs, amplitude, interleaved, true, lengths, nullptr, 0, stream});
    });
}

gdn_status gdn_qk_norm_rope(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                            gdn_dtype dtype, const void* q, const int64_t* q_strides, const void* k,
                            const int64_t* k_strides, const float* q_weight, const float* k_weight,
                            int32_t per_head, float eps, const int32_t* positions,
                            const double* freqs, float amplitude, int32_t interleaved,
                            const int32_t* lengths, void* q_out, const int64_t* q_out_strides,
                            void* k_out, const int64_t* k_out_strides, void* stream) {
    const int code = dtype_code(dtype);
    return guarded([&] {
        Call c{"gdn_qk_norm_rope", Kind::NORM, B, T, Hq, Hk, D, R, code,
               {set_of("q", q, q_strides, "q_out", q_out, q_out_strides),
                set_of("k", k, k_strides, "k_out", k_out, k_out_strides)},
               per_head, eps, positions, freqs, amplitude, interleaved, false, lengths, nullptr, 0, stream};
        c.set[0].weight_name = "q_weight"; c.set[0].weight = q_weight;
        c.set[1].weight_name = "k_weight"; c.set[1].weight = k_weight;
        return run(c);
    });
}

gdn_status gdn_qk_norm_rope_backward_workspace_size(int64_t B, int32_t T, int32_t Hq, int32_t Hk,
                                                    int32_t D, size_t* bytes) {
    return guarded([&] {
        static const char* fn = "gdn_qk_norm_rope_backward_workspace_size";
        if (!bytes) return invalid(fn, "bytes is NULL");
        *bytes = 0;
        gdn_status s = check_sizes(fn, B, T, Hq, Hk, D);
        if (s != GDN_OK) return s;
        *bytes = gdn::rotary_backward_ws_floats(B, T, Hq, Hk, D) * sizeof(float);
        return GDN_OK;
    });
}

gdn_status gdn_qk_norm_rope_backward(
    int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, gdn_dtype dtype,
    const void* dq, const int64_t* dq_strides, const void* dk, const int64_t* dk_strides,
    const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
    const float* q_weight, const float* k_weight, int32_t per_head, float eps,
    const int32_t* positions, const double* freqs, float amplitude, int32_t interleaved,
    const int32_t* lengths, void* q_out, const int64_t* q_out_strides, void* k_out,
    const int64_t* k_out_strides, float* dq_weight, float* dk_weight, void* workspace,
    size_t workspace_bytes, void* stream) {
    const int code = dtype_code(dtype);
    return guarded([&] {
        return run(Call{"gdn_qk_norm_rope_backward", Kind::NORM_BACKWARD, B, T, Hq, Hk, D, R, code,
                        {RawSet{{"q", q, q_strides}, {"dq", dq, dq_strides}, {"q_out", q_out, q_out_strides},
                                "q_weight", "dq_weight", q_weight, dq_weight},
                         RawSet{{"k", k, k_strides}, {"dk", dk, dk_strides}, {"k_out", k_out, k_out_strides},
                                "k_weight", "dk_weight", k_weight, dk_weight}},
                        per_head, eps, positions, freqs, amplitude, interleaved, true, lengths, workspace,
                        workspace_bytes, stream});
    });
}

}  // extern "C"
