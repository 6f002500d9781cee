// C-ABI entry points declared in include/gdn_linear.h (linear attention with a decay for each head,
// its gradients, layer norm): host-side validation, then kernel launches on the caller's stream.
// Nothing here synchronises or allocates device memory.

#include "gdn_linear.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <new>
#include <string>

#include "gdn_api_common.h"
#include "gdn_linear_launch.h"

using namespace gdn::api;

namespace {

constexpr size_t kMaxElements = size_t(1) << 60;  // of one tensor: byte counts stay far from 2^64

// Runs an entry point's body; no C++ exception (a failed host allocation) leaves the C ABI.
template <typename F>
gdn_status guarded(F&& body) {
    try {
        gdn::last_error().clear();
        return body();
    } catch (const std::bad_alloc&) {
        return GDN_ERR_OUT_OF_MEMORY;
    } catch (...) {
        return GDN_ERR_HIP;
    }
}

// A dtype argument as the number that was passed: a C caller may pass any, and to load one that is no
// enumerator as the enum is undefined.
int dtype_code(const gdn_dtype& t) {
    int c;
    static_assert(sizeof(c) == sizeof(t), "dtype");
    memcpy(&c, &t, sizeof(c));
    return c;
}
bool valid_code(int c) { return c == GDN_F32 || c == GDN_BF16 || c == GDN_F16; }

gdn_status invalid(const char* fn, const char* msg) {
    return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + msg);
}

// Sizes of a linear-attention call; Hk is checked against H.
gdn_status check_linear(const char* fn, int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                        int32_t dv) {
    if (B >= (int64_t(1) << 31)) return invalid(fn, "B * H must be < 2^31");
    gdn_status s = check_shape(fn, B, T, H, dk, dv);
    if (s != GDN_OK) return s;
    if (Hk < 1 || H % Hk != 0) return invalid(fn, "Hk must be >= 1 and divide H");
    if (T >= (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": T must be < 2^30");
    size_t n = 0;
    if (!mul_ok((size_t)B * H, (size_t)T, &n) || !mul_ok(n, (size_t)dk, &n) || n >= kMaxElements)
        return invalid(fn, "size overflows");
    return GDN_OK;
}

gdn_status check_optional(const char* fn, const char* name, const void* p) {
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": " + name + " is not 16-byte aligned");
    return GDN_OK;
}

gdn_status check_workspace(const char* fn, const void* workspace, size_t bytes, size_t need) {
    if (need == 0) return GDN_OK;
    gdn_status s = check_ptrs(fn, {{"workspace", workspace}});
    if (s != GDN_OK) return s;
    if (bytes < need)
        return fail(GDN_ERR_INVALID_ARGUMENT, std::string(fn) + ": workspace has " + std::to_string(bytes) +
                                                  " bytes, " + std::to_string(need) + " needed");
    return GDN_OK;
}

gdn_status forward(const char* fn, bool prefill, int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                   int32_t dv, const void* q, const void* k, const void* v, int act_code,
                   const float* decay, const int32_t* lengths, void* state, int state_code, void* o,
                   float scale, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status s = check_linear(fn, B, T, H, Hk, dk, dv);
    if (s != GDN_OK) return s;
    if (!valid_code(act_code) || !valid_code(state_code)) return invalid(fn, "bad dtype");
    const gdn_dtype act_dtype = (gdn_dtype)act_code, state_dtype = (gdn_dtype)state_code;
    if (B == 0 || T == 0) return GDN_OK;
    s = check_ptrs(fn, {{"q", q}, {"k", k}, {"v", v}, {"decay", decay}, {"state", state}, {"o", o}});
    if (s != GDN_OK) return s;
    s = check_optional(fn, "lengths", lengths);
    if (s != GDN_OK) return s;
    const size_t need = prefill ? gdn::linear_prefill_ws_floats(B, T, H, dk) * sizeof(float) : 0;
    s = check_workspace(fn, workspace, workspace_bytes, need);
    if (s != GDN_OK) return s;
    const size_t ab = dtype_bytes(act_dtype);
    const size_t kv = (size_t)B * T * Hk * dk * ab, vo = (size_t)B * T * H * dv * ab;
    const Range r_q = range("q", q, kv), r_k = range("k", k, kv), r_v = range("v", v, vo);
    const Range r_d = range("decay", decay, (size_t)H * 4);
    const Range r_l = range("lengths", lengths, lengths ? (size_t)B * 4 : 0);
    const Range r_s = range("state", state, (size_t)B * H * dk * dv * dtype_bytes(state_dtype));
    const Range r_o = range("o", o, vo), r_w = range("workspace", workspace, need);
    s = check_disjoint(fn, r_o, {r_q, r_k, r_v, r_d, r_l, r_s, r_w});
    if (s != GDN_OK) return s;
    s = check_disjoint(fn, r_s, {r_q, r_k, r_v, r_d, r_l, r_w});
    if (s != GDN_OK) return s;
    s = check_disjoint(fn, r_w, {r_q, r_k, r_v, r_d, r_l});
    if (s != GDN_OK) return s;

    gdn::LinearArgs a;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.D = dk;
    a.q = q; a.k = k; a.v = v; a.act = to_dtype(act_dtype);
    a.decay = decay; a.lengths = lengths;
    a.state = state; a.state_dtype = to_dtype(state_dtype);
    a.o = o; a.scale = scale;
    a.ws = static_cast<float*>(workspace);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = prefill ? gdn::launch_linear_prefill(a, st) : gdn::launch_linear_decode(a, st);
    if (e != hipSuccess) return fail_hip((std::string(fn) + ": kernel launch").c_str(), e);
    return GDN_OK;
}

// Sizes of a layer-norm call.
gdn_status check_norm(const char* fn, int64_t rows, int32_t G, int32_t C) {
    if (rows < 0) return invalid(fn, "rows must be >= 0");
    if (G < 1 || C < 1) return invalid(fn, "G and C must be >= 1");
    if (rows % G != 0) return invalid(fn, "rows must be a multiple of G");
    size_t n = 0;
    if (!mul_ok((size_t)rows, (size_t)C, &n) || n >= kMaxElements) return invalid(fn, "size overflows");
    if ((int64_t)G * C >= (int64_t(1) << 31)) return invalid(fn, "G * C must be < 2^31");
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_linear_attn_decode_step(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                                       int32_t dv, const void* q, const void* k, const void* v,
                                       gdn_dtype act_dtype, const float* decay,
                                       const int32_t* lengths, void* state,
                                       gdn_dtype state_dtype, void* o, float scale, void* stream) {
    const int act = dtype_code(act_dtype), st = dtype_code(state_dtype);
    return guarded([&] {
        return forward("gdn_linear_attn_decode_step", false, B, T, H, Hk, dk, dv, q, k, v, act, decay,
                       lengths, state, st, o, scale, nullptr, 0, stream);
    });
}

gdn_status gdn_linear_attn_prefill_workspace_size(int64_t B, int32_t T, int32_t H, int32_t dk,
                                                  int32_t dv, size_t* bytes) {
    return guarded([&] {
        static const char* fn = "gdn_linear_attn_prefill_workspace_size";
        if (!bytes) return invalid(fn, "bytes is NULL");
        *bytes = 0;
        gdn_status s = check_linear(fn, B, T, H, H, dk, dv);
        if (s != GDN_OK) return s;
        *bytes = gdn::linear_prefill_ws_floats(B, T, H, dk) * sizeof(float);
        return GDN_OK;
    });
}

gdn_status gdn_linear_attn_prefill(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                                   int32_t dv, const void* q, const void* k, const void* v,
                                   gdn_dtype act_dtype, const float* decay,
                                   const int32_t* lengths, void* state, gdn_dtype state_dtype,
                                   void* o, float scale, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    const int act = dtype_code(act_dtype), st = dtype_code(state_dtype);
    return guarded([&] {
        return forward("gdn_linear_attn_prefill", true, B, T, H, Hk, dk, dv, q, k, v, act, decay,
                       lengths, state, st, o, scale, workspace, workspace_bytes, stream);
    });
}

gdn_status gdn_linear_attn_backward_workspace_size(int64_t B, int32_t T, int32_t H, int32_t Hk,
                                                   int32_t dk, int32_t dv, size_t* bytes) {
    return guarded([&] {
        static const char* fn = "gdn_linear_attn_backward_workspace_size";
        if (!bytes) return invalid(fn, "bytes is NULL");
        *bytes = 0;
        gdn_status s = check_linear(fn, B, T, H, Hk, dk, dv);
        if (s != GDN_OK) return s;
        *bytes = gdn::linear_backward_ws_floats(B, T, H, Hk, dk) * sizeof(float);
        return GDN_OK;
    });
}

gdn_status gdn_linear_attn_backward(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                                    int32_t dv, const void* q, const void* k, const void* v,
                                    gdn_dtype act_dtype, const float* decay,
                                    const int32_t* lengths, const void* state0,
                                    const void* d_o, const void* dstate, gdn_dtype state_dtype,
                                    void* dq, void* dk_out, void* dv_out, void* dstate0,
                                    float* ddecay, float scale, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const int act_code = dtype_code(act_dtype), state_code = dtype_code(state_dtype);
    return guarded([&] {
        static const char* fn = "gdn_linear_attn_backward";
        gdn_status s = check_linear(fn, B, T, H, Hk, dk, dv);
        if (s != GDN_OK) return s;
        if (!valid_code(act_code) || !valid_code(state_code)) return invalid(fn, "bad dtype");
        const gdn_dtype act = (gdn_dtype)act_code, state = (gdn_dtype)state_code;
        // With no tokens the states' gradients remain: dstate0 = dstate, ddecay = 0.
        const bool empty = B == 0 || T == 0;
        if (empty && (B == 0 || !dstate0) && !ddecay) return GDN_OK;
        if (!empty) {
            s = check_ptrs(fn, {{"q", q}, {"k", k}, {"v", v}, {"d_o", d_o}, {"dq", dq}, {"dk_out", dk_out},
                                {"dv_out", dv_out}});
            if (s != GDN_OK) return s;
        }
        if (B > 0) {
            s = check_ptrs(fn, {{"decay", decay}});
            if (s != GDN_OK) return s;
        }
        const std::pair<const char*, const void*> optional[] = {
            {"lengths", lengths}, {"state0", state0}, {"dstate", dstate}, {"dstate0", dstate0}, {"ddecay", ddecay}};
        for (auto& p : optional) {
            s = check_optional(fn, p.first, p.second);
            if (s != GDN_OK) return s;
        }
        const size_t need = gdn::linear_backward_ws_floats(B, T, H, Hk, dk) * sizeof(float);
        s = check_workspace(fn, workspace, workspace_bytes, need);
        if (s != GDN_OK) return s;
        const size_t ab = dtype_bytes(act);
        const size_t kv = (size_t)B * T * Hk * dk * ab, vo = (size_t)B * T * H * dv * ab;
        const size_t st = (size_t)B * H * dk * dv * dtype_bytes(state);
        const Range in[] = {range("q", q, kv), range("k", k, kv), range("v", v, vo), range("d_o", d_o, vo),
                            range("decay", decay, (size_t)H * 4),
                            range("lengths", lengths, lengths ? (size_t)B * 4 : 0),
                            range("state0", state0, state0 ? st : 0), range("dstate", dstate, dstate ? st : 0)};
        const Range out[] = {range("dq", dq, kv), range("dk_out", dk_out, kv), range("dv_out", dv_out, vo),
                             range("dstate0", dstate0, dstate0 ? st : 0),
                             range("ddecay", ddecay, ddecay ? (size_t)H * 4 : 0),
                             range("workspace", workspace, need)};
        for (size_t i = 0; i < sizeof(out) / sizeof(out[0]); ++i) {
            for (auto& r : in) {
                s = check_disjoint(fn, out[i], {r});
                if (s != GDN_OK) return s;
            }
            for (size_t j = 0; j < i; ++j) {
                s = check_disjoint(fn, out[i], {out[j]});
                if (s != GDN_OK) return s;
            }
        }

        gdn::LinearBackwardArgs a;
        a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.D = dk;
        a.q = q; a.k = k; a.v = v; a.act = to_dtype(act);
        a.decay = decay; a.lengths = lengths;
        a.state0 = state0; a.d_o = d_o; a.dstate = dstate; a.state_dtype = to_dtype(state);
        a.dq = dq; a.dk = dk_out; a.dv = dv_out; a.dstate0 = dstate0; a.ddecay = ddecay;
        a.scale = scale;
        a.ws = static_cast<float*>(workspace);
        hipError_t e = gdn::launch_linear_backward(a, reinterpret_cast<hipStream_t>(stream));
        if (e != hipSuccess) return fail_hip("gdn_linear_attn_backward: kernel launch", e);
        return GDN_OK;
    });
}

gdn_status gdn_layer_norm(int64_t rows, int32_t G, int32_t C, const void* x, gdn_dtype dtype,
                          const float* weight, const float* bias, void* y, float* mean,
                          float* rstd, float eps, void* stream) {
    const int code = dtype_code(dtype);
    return guarded([&] {
        static const char* fn = "gdn_layer_norm";
        gdn_status s = check_norm(fn, rows, G, C);
        if (s != GDN_OK) return s;
        if (!valid_code(code)) return invalid(fn, "bad dtype");
        const gdn_dtype type = (gdn_dtype)code;
        if (!(eps >= 0.0f)) return invalid(fn, "eps must be >= 0");
        if ((mean == nullptr) != (rstd == nullptr)) return invalid(fn, "mean and rstd are wanted together or not at all");
        if (rows == 0) return GDN_OK;
        s = check_ptrs(fn, {{"x", x}, {"y", y}});
        if (s != GDN_OK) return s;
        const std::pair<const char*, const void*> optional[] = {
            {"weight", weight}, {"bias", bias}, {"mean", mean}, {"rstd", rstd}};
        for (auto& p : optional) {
            s = check_optional(fn, p.first, p.second);
            if (s != GDN_OK) return s;
        }
        const size_t n = (size_t)rows * C * dtype_bytes(type), p = (size_t)G * C * 4, st = (size_t)rows * 4;
        const Range r_x = range("x", x, n), r_y = range("y", y, n);
        const Range r_w = range("weight", weight, weight ? p : 0), r_b = range("bias", bias, bias ? p : 0);
        const Range r_m = range("mean", mean, mean ? st : 0), r_r = range("rstd", rstd, rstd ? st : 0);
        if (x != y) {
            s = check_disjoint(fn, r_y, {r_x});
            if (s != GDN_OK) return s;
        }
        s = check_disjoint(fn, r_y, {r_w, r_b, r_m, r_r});
        if (s != GDN_OK) return s;
        s = check_disjoint(fn, r_m, {r_x, r_w, r_b, r_r});
        if (s != GDN_OK) return s;
        s = check_disjoint(fn, r_r, {r_x, r_w, r_b});
        if (s != GDN_OK) return s;

        gdn::NormArgs a;
        a.rows = rows; a.G = G; a.C = C;
        a.x = x; a.dtype = to_dtype(type);
        a.weight = weight; a.bias = bias;
        a.y = y; a.mean = mean; a.rstd = rstd; a.eps = eps;
        hipError_t e = gdn::launch_layer_norm(a, reinterpret_cast<hipStream_t>(stream));
        if (e != hipSuccess) return fail_hip("gdn_layer_norm: kernel launch", e);
        return GDN_OK;
    });
}

gdn_status gdn_layer_norm_backward_workspace_size(int64_t rows, int32_t G, int32_t C, size_t* bytes) {
    return guarded([&] {
        static const char* fn = "gdn_layer_norm_backward_workspace_size";
        if (!bytes) return invalid(fn, "bytes is NULL");
        *bytes = 0;
        gdn_status s = check_norm(fn, rows, G, C);
        if (s != GDN_OK) return s;
        *bytes = gdn::norm_backward_ws_floats(rows, G, C) * sizeof(float);
        return GDN_OK;
    });
}

gdn_status gdn_layer_norm_backward(int64_t rows, int32_t G, int32_t C, const void* dy,
                                   const void* x, gdn_dtype dtype, const float* weight,
                                   const float* mean, const float* rstd, void* dx,
                                   float* dweight, float* dbias, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    const int code = dtype_code(dtype);
    return guarded([&] {
        static const char* fn = "gdn_layer_norm_backward";
        gdn_status s = check_norm(fn, rows, G, C);
        if (s != GDN_OK) return s;
        if (!valid_code(code)) return invalid(fn, "bad dtype");
        const gdn_dtype type = (gdn_dtype)code;
        const bool params = dweight || dbias;
        if (rows == 0 && !params) return GDN_OK;
        if (rows > 0) {
            s = check_ptrs(fn, {{"dy", dy}, {"x", x}, {"mean", mean}, {"rstd", rstd}, {"dx", dx}});
            if (s != GDN_OK) return s;
        }
        const std::pair<const char*, const void*> optional[] = {
            {"weight", weight}, {"dweight", dweight}, {"dbias", dbias}};
        for (auto& p : optional) {
            s = check_optional(fn, p.first, p.second);
            if (s != GDN_OK) return s;
        }
        const size_t need = params ? gdn::norm_backward_ws_floats(rows, G, C) * sizeof(float) : 0;
        s = check_workspace(fn, workspace, workspace_bytes, need);
        if (s != GDN_OK) return s;
        const size_t n = (size_t)rows * C * dtype_bytes(type), p = (size_t)G * C * 4, st = (size_t)rows * 4;
        const Range r_x = range("x", x, n), r_dy = range("dy", dy, n), r_dx = range("dx", dx, n);
        const Range r_w = range("weight", weight, weight ? p : 0);
        const Range r_m = range("mean", mean, st), r_r = range("rstd", rstd, st);
        const Range r_dw = range("dweight", dweight, dweight ? p : 0), r_db = range("dbias", dbias, dbias ? p : 0);
        const Range r_ws = range("workspace", workspace, need);
        if (dx != dy) {
            s = check_disjoint(fn, r_dx, {r_dy});
            if (s != GDN_OK) return s;
        }
        s = check_disjoint(fn, r_dx, {r_x, r_w, r_m, r_r, r_dw, r_db, r_ws});
        if (s != GDN_OK) return s;
        s = check_disjoint(fn, r_dw, {r_dy, r_x, r_w, r_m, r_r, r_db, r_ws});
        if (s != GDN_OK) return s;
        s = check_disjoint(fn, r_db, {r_dy, r_x, r_w, r_m, r_r, r_ws});
        if (s != GDN_OK) return s;
        s = check_disjoint(fn, r_ws, {r_dy, r_x, r_w, r_m, r_r});
        if (s != GDN_OK) return s;

        gdn::NormBackwardArgs a;
        a.rows = rows; a.G = G; a.C = C;
        a.dy = dy; a.x = x; a.dtype = to_dtype(type);
        a.weight = weight; a.mean = mean; a.rstd = rstd;
        a.dx = dx; a.dweight = dweight; a.dbias = dbias;
        a.ws = static_cast<float*>(workspace);
        hipError_t e = gdn::launch_layer_norm_backward(a, reinterpret_cast<hipStream_t>(stream));
        if (e != hipSuccess) return fail_hip("gdn_layer_norm_backward: kernel launch", e);
        return GDN_OK;
    });
}

}  // extern "C"
