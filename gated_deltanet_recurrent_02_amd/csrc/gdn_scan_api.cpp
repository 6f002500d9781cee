// C-ABI entry points declared in include/gdn_scan.h (the gated linear recurrence and its gradients): host-side
// validation, then kernel launches on the caller's stream. Nothing here synchronises or allocates device memory.

#include "gdn_scan.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "gdn_api_common.h"
#include "gdn_scan_launch.h"
#include "gdn_strided.h"

using namespace gdn::api;

static_assert(GDN_SCAN_CHECKPOINT == gdn::kScanChunk, "checkpoints");

namespace {

gdn_status check_sizes(const char* fn, int64_t B, int32_t T, int32_t C) {
    if (B < 0 || T < 0) return invalid(fn, "B and T must be >= 0");
    if (C < 1) return invalid(fn, "C must be >= 1");
    if (B >= (int64_t(1) << 31) || B * C >= (int64_t(1) << 31))
        return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": B * C must be < 2^31");
    if (T >= (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": T must be < 2^30");
    if ((size_t)B * C * (size_t)T >= kMaxElements) return invalid(fn, "size overflows");
    if (B * gdn::scan_chunks(T) * (((int64_t)C + 63) / 64) >= (int64_t(1) << 31))
        return fail(GDN_ERR_UNSUPPORTED, std::string(fn) + ": B * ceil(T / 64) * ceil(C / 64) must be < 2^31");
    return GDN_OK;
}

gdn_status rows(const char* fn, const char* name, const void* p, const int64_t* strides, int64_t B, int32_t T, int32_t C,
                size_t es, Strided* out) {
    return strided(fn, name, p, strides, 2, B, T, 1, C, es, out);
}

gdn::RowsView view(const Strided& t, size_t es) {
    return gdn::RowsView{reinterpret_cast<void*>(t.base), t.stride[0] / (int64_t)es, t.stride[1] / (int64_t)es};
}

gdn_status forward(const char* fn, bool prefill, int64_t B, int32_t T, int32_t C, const void* x, const int64_t* xs,
                   const void* a, const int64_t* as, const void* b, const int64_t* bs, int act, const float* rate,
                   const int32_t* lengths, void* state, int state_code, void* o, const int64_t* os, float* checkpoints,
                   void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status s = check_sizes(fn, B, T, C);
    if (s != GDN_OK) return s;
    if (!valid_code(act) || !valid_code(state_code)) return invalid(fn, "bad dtype");
    if (B == 0 || T == 0) return GDN_OK;
    const size_t es = act == GDN_F32 ? 4 : 2;
    Strided rx, ra, rb = absent("b"), ro;
    s = rows(fn, "x", x, xs, B, T, C, es, &rx);
    if (s != GDN_OK) return s;
    s = rows(fn, "a", a, as, B, T, C, es, &ra);
    if (s != GDN_OK) return s;
    if (b) {
        s = rows(fn, "b", b, bs, B, T, C, es, &rb);
        if (s != GDN_OK) return s;
    }
    s = rows(fn, "o", o, os, B, T, C, es, &ro);
    if (s != GDN_OK) return s;
    s = check_ptrs(fn, {{"state", state}});
    if (s != GDN_OK) return s;
    const std::pair<const char*, const void*> optional[] = {
        {"rate", rate}, {"lengths", lengths}, {"checkpoints", checkpoints}};
    for (auto& p : optional) {
        s = check_optional(fn, p.first, p.second);
        if (s != GDN_OK) return s;
    }
    const size_t need = prefill ? gdn::scan_prefill_ws_floats(B, T, C) * sizeof(float) : 0;
    s = check_workspace(fn, workspace, workspace_bytes, need);
    if (s != GDN_OK) return s;

    const Strided rr = run_of("rate", rate, (size_t)C * 4), rl = run_of("lengths", lengths, (size_t)B * 4);
    const Strided rs = run_of("state", state, (size_t)B * C * (state_code == GDN_F32 ? 4 : 2));
    const Strided rc = run_of("checkpoints", checkpoints, (size_t)B * gdn::scan_chunks(T) * C * 4);
    const Strided rw = run_of("workspace", need ? workspace : nullptr, need);
    const Strided* all[] = {&rx, &ra, &rb, &rr, &rl, &rs, &ro, &rc, &rw};
    const Strided* outs[] = {&ro, &rs, &rc, &rw};
    for (const Strided* out : outs) {
        s = check_output(fn, *out, all, sizeof(all) / sizeof(all[0]));
        if (s != GDN_OK) return s;
    }

    gdn::ScanArgs g{};
    g.B = B; g.T = T; g.C = C;
    g.act = to_dtype((gdn_dtype)act); g.state_dtype = to_dtype((gdn_dtype)state_code);
    g.x = view(rx, es); g.a = view(ra, es); g.o = view(ro, es);
    if (b) g.b = view(rb, es);
    g.rate = rate; g.lengths = lengths; g.state = state; g.checkpoints = checkpoints;
    g.ws = static_cast<float*>(workspace);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = prefill ? gdn::launch_scan_prefill(g, st) : gdn::launch_scan_decode(g, st);
    if (e != hipSuccess) return fail_hip((std::string(fn) + ": kernel launch").c_str(), e);
    return GDN_OK;
}

gdn_status workspace_size(const char* fn, int64_t B, int32_t T, int32_t C, bool backward, size_t* bytes) {
    if (!bytes) return invalid(fn, "bytes is NULL");
    *bytes = 0;
    gdn_status s = check_sizes(fn, B, T, C);
    if (s != GDN_OK) return s;
    *bytes = (backward ? gdn::scan_backward_ws_floats(B, T, C) : gdn::scan_prefill_ws_floats(B, T, C)) * sizeof(float);
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_gated_scan_decode_step(int64_t B, int32_t T, int32_t C, const void* x,
                                      const int64_t* x_strides, const void* a,
                                      const int64_t* a_strides, const void* b,
                                      const int64_t* b_strides, gdn_dtype act_dtype,
                                      const float* rate, const int32_t* lengths, void* state,
                                      gdn_dtype state_dtype, void* o, const int64_t* o_strides,
                                      void* stream) {
    const int act = dtype_code(act_dtype), st = dtype_code(state_dtype);
    return guarded([&] {
        return forward("gdn_gated_scan_decode_step", false, B, T, C, x, x_strides, a, a_strides, b, b_strides, act, rate,
                       lengths, state, st, o, o_strides, nullptr, nullptr, 0, stream);
    });
}

gdn_status gdn_gated_scan_prefill_workspace_size(int64_t B, int32_t T, int32_t C, size_t* bytes) {
    return guarded([&] { return workspace_size("gdn_gated_scan_prefill_workspace_size", B, T, C, false, bytes); });
}

gdn_status gdn_gated_scan_prefill(int64_t B, int32_t T, int32_t C, const void* x,
                                  const int64_t* x_strides, const void* a, const int64_t* a_strides,
                                  const void* b, const int64_t* b_strides, gdn_dtype act_dtype,
                                  const float* rate, const int32_t* lengths, void* state,
                                  gdn_dtype state_dtype, void* o, const int64_t* o_strides,
                                  float* checkpoints, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    const int act = dtype_code(act_dtype), st = dtype_code(state_dtype);
    return guarded([&] {
        return forward("gdn_gated_scan_prefill", true, B, T, C, x, x_strides, a, a_strides, b, b_strides, act, rate,
                       lengths, state, st, o, o_strides, checkpoints, workspace, workspace_bytes, stream);
    });
}

gdn_status gdn_gated_scan_backward_workspace_size(int64_t B, int32_t T, int32_t C, size_t* bytes) {
    return guarded([&] { return workspace_size("gdn_gated_scan_backward_workspace_size", B, T, C, true, bytes); });
}

gdn_status gdn_gated_scan_backward(
    int64_t B, int32_t T, int32_t C, const void* x, const int64_t* x_strides, const void* a,
    const int64_t* a_strides, const void* b, const int64_t* b_strides, gdn_dtype act_dtype,
    const float* rate, const int32_t* lengths, const void* state0, const float* checkpoints,
    const void* d_o, const int64_t* d_o_strides, const void* dstate, gdn_dtype state_dtype, void* dx,
    const int64_t* dx_strides, void* da, const int64_t* da_strides, void* db,
    const int64_t* db_strides, void* dstate0, float* drate, void* workspace, size_t workspace_bytes,
    void* stream) {
    const int act = dtype_code(act_dtype), state_code = dtype_code(state_dtype);
    return guarded([&] {
        static const char* fn = "gdn_gated_scan_backward";
        gdn_status s = check_sizes(fn, B, T, C);
        if (s != GDN_OK) return s;
        if (!valid_code(act) || !valid_code(state_code)) return invalid(fn, "bad dtype");
        // With no tokens the states' gradients remain: dstate0 = dstate, drate = 0.
        const bool empty = B == 0 || T == 0;
        if (empty && (B == 0 || !dstate0) && !drate) return GDN_OK;
        const size_t es = act == GDN_F32 ? 4 : 2, ss = state_code == GDN_F32 ? 4 : 2;
        struct Raw { const char* name; const void* p; const int64_t* strides; bool wanted; };
        const Raw raw[7] = {{"x", x, x_strides, true}, {"a", a, a_strides, true}, {"b", b, b_strides, b != nullptr},
                            {"d_o", d_o, d_o_strides, true}, {"dx", dx, dx_strides, true}, {"da", da, da_strides, true},
                            {"db", db, db_strides, b != nullptr}};
        if (!b && db) return invalid(fn, "db is given without b");
        Strided t[7];
        for (int i = 0; i < 7; ++i) {
            t[i] = absent(raw[i].name);
            if (empty || !raw[i].wanted) continue;
            s = rows(fn, raw[i].name, raw[i].p, raw[i].strides, B, T, C, es, &t[i]);
            if (s != GDN_OK) return s;
        }
        const std::pair<const char*, const void*> optional[] = {
            {"rate", rate}, {"lengths", lengths}, {"state0", state0}, {"checkpoints", checkpoints},
            {"dstate", dstate}, {"dstate0", dstate0}, {"drate", drate}};
        for (auto& p : optional) {
            s = check_optional(fn, p.first, p.second);
            if (s != GDN_OK) return s;
        }
        const size_t need = empty ? 0 : gdn::scan_backward_ws_floats(B, T, C) * sizeof(float);
        s = check_workspace(fn, workspace, workspace_bytes, need);
        if (s != GDN_OK) return s;
        const Strided rr = run_of("rate", rate, (size_t)C * 4), rl = run_of("lengths", lengths, (size_t)B * 4);
        const Strided r0 = run_of("state0", state0, (size_t)B * C * ss), r1 = run_of("dstate", dstate, (size_t)B * C * ss);
        const Strided rc = run_of("checkpoints", checkpoints, (size_t)B * gdn::scan_chunks(T) * C * 4);
        const Strided d0 = run_of("dstate0", dstate0, (size_t)B * C * ss), dr = run_of("drate", drate, (size_t)C * 4);
        const Strided rw = run_of("workspace", need ? workspace : nullptr, need);
        const Strided* all[] = {&t[0], &t[1], &t[2], &t[3], &rr, &rl, &r0, &r1, &rc, &t[4], &t[5], &t[6], &d0, &dr, &rw};
        const Strided* outs[] = {&t[4], &t[5], &t[6], &d0, &dr, &rw};
        for (const Strided* out : outs) {
            s = check_output(fn, *out, all, sizeof(all) / sizeof(all[0]));
            if (s != GDN_OK) return s;
        }

        gdn::ScanArgs g{};
        g.B = B; g.T = T; g.C = C;
        g.act = to_dtype((gdn_dtype)act); g.state_dtype = to_dtype((gdn_dtype)state_code);
        if (!empty) {
            g.x = view(t[0], es); g.a = view(t[1], es); g.d_o = view(t[3], es);
            g.dx = view(t[4], es); g.da = view(t[5], es);
            if (b) { g.b = view(t[2], es); g.db = view(t[6], es); }
        }
        g.rate = rate; g.lengths = lengths;
        g.state0 = state0; g.dstate = dstate; g.checkpoints = const_cast<float*>(checkpoints);
        g.dstate0 = dstate0; g.drate = drate;
        g.ws = static_cast<float*>(workspace);
        hipError_t e = gdn::launch_scan_backward(g, reinterpret_cast<hipStream_t>(stream));
        if (e != hipSuccess) return fail_hip("gdn_gated_scan_backward: kernel launch", e);
        return GDN_OK;
    });
}

}  // extern "C"
