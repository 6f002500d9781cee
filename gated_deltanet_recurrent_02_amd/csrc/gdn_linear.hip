// Linear attention with a decay for each head on gfx950 (CDNA4): the recurrent form and the
// gradients. Per sequence b and head h, with l = decay_h in [0, 1],
//     S_t = l S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
// and for the gradients, from do_t and the adjoint of the last state,
//     R_t = l R_{t+1} + scale do_t q_t^T,
//     dq_t = scale S_t^T do_t,   dk_t = R_t^T v_t,   dv_t = R_t k_t,   dS_0 = l R_0,
//     dl = sum_t <R_t, S_{t-1}>.
//
// All of these are one operation, a sweep: a state N (rows indexed by z's dimension, columns by
// y's) takes N <- l N + z_t y_t^T and gives out_t = N x_t, forward or backward in time:
//     o : x = q,  y = k,  z = v,  forward         dv: x = k, y = q,  z = scale do, backward
//     dq: x = do, y = v,  z = k,  forward         dk: x = v, y = do, z = scale q,  backward
// dq's state is S transposed and dk's is R transposed, so a sweep may read its first state
// transposed. A backward sweep numbers tokens from its sequence's last one; its first state is the
// adjoint of the last state, which enters that token undecayed, so the decay comes after a token
// instead of before it, and the state left at the end is l R_0 = dS_0.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_linear_common.h"
#include "gdn_linear_launch.h"

namespace gdn {
namespace {

// Lanes per state row and rows per wave of the recurrent kernel: a wave's load instruction covers
// whole 128-byte lines of the state. One token: 8 rows a wave, the state's stream decides (B = 256, H = 48,
// D = 128, fp32 state: 257 us, 6.3 TB/s, with 16 rows 280, with 32 283; bf16 state 129, 129 and 133). Several
// tokens: 16 rows, since every token's k and q are widened once a wave (bf16 state, B = 96, T = 4, ragged: 62 us,
// with 8 rows 74, with 32 65; fp32 state 114, 117 and 112).
template <int D, typename ST, bool MULTI>
struct RowGeo {
    static constexpr int VW = 16 / (int)sizeof(ST);           // elements per 16-byte access
    static constexpr int LPR = D / VW >= 16 ? (sizeof(ST) == 4 ? 16 : 8) : (D / VW < 4 ? 4 : D / VW);
    static constexpr int E = D / LPR;                         // state columns per lane
    static constexpr int CW = E < VW ? E : VW;                // columns per access
    static constexpr int RPP = 64 / LPR;                      // rows per pass
    static constexpr int RPW = RPP > (MULTI ? 16 : 8) ? RPP : (MULTI ? 16 : 8);  // rows per wave
    static constexpr int P = RPW / RPP;                       // passes
    static constexpr int WPH = D / RPW;                       // waves (workgroups) per head
    static_assert(D % RPW == 0 && E % CW == 0, "geometry");
    static __device__ __forceinline__ int col(int l, int c) { return (c * LPR + l) * CW; }
};

// The recurrent form: one wave per RPW state rows, token by token on the state in registers; no
// two waves share anything but read-only inputs. REV and TR are the sweep's reverse and transposed.
template <int D, typename AT, typename ST, typename OT, bool REV, bool TR, bool MULTI>
__global__ __launch_bounds__(64) void gdn_linear_recurrent_kernel(Sweep a) {
    using G = RowGeo<D, ST, MULTI>;
    constexpr int E = G::E, CW = G::CW, P = G::P;
    const int lane = threadIdx.x, g = lane / G::LPR, l = lane % G::LPR;
    const uint32_t bid = blockIdx.x;
    const int w = (int)(bid % G::WPH);
    const uint32_t head = bid / G::WPH;
    const int64_t bh = head, b = head / (uint32_t)a.H;
    const int h = (int)(head % (uint32_t)a.H);
    const int T = a.T;
    const int n = tokens_of(a.lengths, b, T);
    const float lam = a.decay[h];
    const int row0 = w * G::RPW + g;

    OT* out = (OT*)a.out + ((size_t)b * T * a.H + h) * D;
    const size_t ostride = (size_t)a.H * D;
    // outputs past the sequence's end
    if (l == 0) {
        for (int t = n; t < T; ++t)
#pragma unroll
            for (int p = 0; p < P; ++p) out[t * ostride + row0 + p * G::RPP] = from_f32<OT>(0.0f);
    }
    if (n == 0 && (a.last == nullptr || a.last == a.first)) return;

    float S[P][E];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < E; ++e) S[p][e] = 0.0f;
    if (a.first) {
        const ST* s = (const ST*)a.first + (size_t)bh * D * D;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int c = 0; c < E / CW; ++c) {
                const int i = row0 + p * G::RPP, j = G::col(l, c);
                if constexpr (TR) {
#pragma unroll
                    for (int e = 0; e < CW; ++e) S[p][c * CW + e] = to_f32<ST>(s[(size_t)(j + e) * D + i]);
                } else {
                    Run<ST, CW> r;
                    r.template load<true>(s + (size_t)i * D + j);
#pragma unroll
                    for (int e = 0; e < CW; ++e) S[p][c * CW + e] = r.get(e);
                }
            }
    }

    const int Hx = a.H / a.gx, Hy = a.H / a.gy, Hz = a.H / a.gz;
    const AT* x = (const AT*)a.x + ((size_t)b * T * Hx + h / a.gx) * D;
    const AT* y = (const AT*)a.y + ((size_t)b * T * Hy + h / a.gy) * D;
    const AT* z = (const AT*)a.z + ((size_t)b * T * Hz + h / a.gz) * D;
    for (int i = 0; i < n; ++i) {
        const size_t t = REV ? n - 1 - i : i;
        float xv[E], yv[E];
#pragma unroll
        for (int c = 0; c < E / CW; ++c) {
            Run<AT, CW> rx, ry;
            rx.load(x + t * Hx * D + G::col(l, c));
            ry.load(y + t * Hy * D + G::col(l, c));
#pragma unroll
            for (int e = 0; e < CW; ++e) { xv[c * CW + e] = rx.get(e); yv[c * CW + e] = ry.get(e); }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float zi = a.zscale * to_f32<AT>(z[t * Hz * D + row0 + p * G::RPP]);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                S[p][e] = fmaf(zi, yv[e], REV ? S[p][e] : lam * S[p][e]);
                sum = fmaf(S[p][e], xv[e], sum);
                if constexpr (REV) S[p][e] *= lam;
            }
            sum = lane_sum<G::LPR>(sum);
            if (l == 0) out[t * ostride + row0 + p * G::RPP] = from_f32<OT>(a.oscale * sum);
        }
    }

    if (a.last) {
        ST* s = (ST*)a.last + (size_t)bh * D * D;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int c = 0; c < E / CW; ++c) {
                Run<ST, CW> r;
                r.set(&S[p][c * CW]);
                r.template store<true>(s + (size_t)(row0 + p * G::RPP) * D + G::col(l, c));
            }
    }
}

// The decay's gradient, token by token: with M_t = dS_t / dl = l M_{t-1} + S_{t-1} the loss's
// derivative is sum_t scale do_t^T M_t q_t + <dS_T, M_T>; every row of S and M adds its own part.
// One partial sum per wave, written to part[wave of the head][b][h].
template <int D, typename AT, typename ST>
__global__ __launch_bounds__(64) void gdn_linear_tangent_kernel(
    int64_t B, int T, int H, int group, const AT* __restrict__ q, const AT* __restrict__ k,
    const AT* __restrict__ v, const AT* __restrict__ d_o, const float* __restrict__ decay,
    const int32_t* __restrict__ lengths, const ST* __restrict__ state0,
    const ST* __restrict__ dstate, float scale, float* __restrict__ part) {
    using G = RowGeo<D, ST, false>;
    constexpr int E = G::E, CW = G::CW, P = G::P;
    const int lane = threadIdx.x, g = lane / G::LPR, l = lane % G::LPR;
    const uint32_t bid = blockIdx.x;
    const int w = (int)(bid % G::WPH);
    const uint32_t head = bid / G::WPH;
    const int64_t bh = head, b = head / (uint32_t)H;
    const int h = (int)(head % (uint32_t)H);
    const int n = tokens_of(lengths, b, T);
    const float lam = decay[h];
    const int row0 = w * G::RPW + g;
    const int Hk = H / group;

    float S[P][E], M[P][E];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < E; ++e) S[p][e] = M[p][e] = 0.0f;
    if (state0) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int c = 0; c < E / CW; ++c) {
                Run<ST, CW> r;
                r.load(state0 + ((size_t)bh * D + row0 + p * G::RPP) * D + G::col(l, c));
#pragma unroll
                for (int e = 0; e < CW; ++e) S[p][c * CW + e] = r.get(e);
            }
    }
    double total = 0.0;
    for (int t = 0; t < n; ++t) {
        const size_t qk = ((size_t)(b * T + t) * Hk + h / group) * D;
        const size_t vo = ((size_t)(b * T + t) * H + h) * D;
        float qv[E], kv[E];
#pragma unroll
        for (int c = 0; c < E / CW; ++c) {
            Run<AT, CW> rq, rk;
            rq.load(q + qk + G::col(l, c));
            rk.load(k + qk + G::col(l, c));
#pragma unroll
            for (int e = 0; e < CW; ++e) { qv[c * CW + e] = rq.get(e); kv[c * CW + e] = rk.get(e); }
        }
        float add = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float vi = to_f32<AT>(v[vo + row0 + p * G::RPP]);
            const float di = to_f32<AT>(d_o[vo + row0 + p * G::RPP]);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                M[p][e] = fmaf(lam, M[p][e], S[p][e]);
                S[p][e] = fmaf(vi, kv[e], lam * S[p][e]);
                sum = fmaf(M[p][e], qv[e], sum);
            }
            add = fmaf(di, sum, add);
        }
        total += (double)(scale * add);
    }
    if (dstate && n > 0) {  // without tokens M is 0, whatever dstate holds
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int c = 0; c < E / CW; ++c) {
                Run<ST, CW> r;
                r.load(dstate + ((size_t)bh * D + row0 + p * G::RPP) * D + G::col(l, c));
#pragma unroll
                for (int e = 0; e < CW; ++e) total += (double)(r.get(e) * M[p][c * CW + e]);
            }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m);
    if (lane == 0) part[(size_t)w * B * H + bh] = (float)total;
}

// ddecay[h] = the sum of n partial sums part[i][h], i < n, in a fixed order; in 64 bits, since the
// sums of many sequences may cancel.
__global__ __launch_bounds__(64) void gdn_linear_ddecay_kernel(int64_t n, int H, const float* __restrict__ part,
                                                               float* __restrict__ ddecay) {
    const int h = blockIdx.x;
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 64) sum += (double)part[(size_t)i * H + h];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if (threadIdx.x == 0) ddecay[h] = (float)sum;
}

// dst[row] = the sum over a group's heads of src [rows][group][D] (fp32 gradients of the heads that
// share a q/k head), rounded once; dq and dk in one launch.
template <typename AT>
__global__ __launch_bounds__(256) void gdn_linear_group_sum_kernel(int64_t n4, int D4, int group,
                                                                   const f32x4* __restrict__ src0,
                                                                   const f32x4* __restrict__ src1,
                                                                   AT* __restrict__ dst0, AT* __restrict__ dst1) {
    const f32x4* src = blockIdx.y ? src1 : src0;
    AT* dst = blockIdx.y ? dst1 : dst0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / D4;
        const int c = (int)(i % D4);
        f32x4 s = src[row * group * D4 + c];
        for (int j = 1; j < group; ++j) s += src[(row * group + j) * D4 + c];
        const float f[4] = {s.x, s.y, s.z, s.w};
        Run<AT, 4> r;
        r.set(f);
        r.store(dst + i * 4);
    }
}

// ------------------------------------------------------------------------ dispatch

template <typename F>
hipError_t launch(F kernel, int64_t blocks, int threads, hipStream_t s, void** args) {
    return hipLaunchKernel((const void*)kernel, dim3((unsigned)blocks), dim3((unsigned)threads), args, 0, s);
}

template <int D, typename AT, typename ST, typename OT, bool REV, bool TR>
hipError_t launch_recurrent(Sweep w, int64_t B, hipStream_t s) {
    void* args[] = {&w};
    static_assert(64 * RowGeo<D, ST, false>::WPH <= kThreadsPerHeadPerDim * D, "threads per head");
    if constexpr (!REV && !TR) {
        if (w.T > 1)
            return launch(gdn_linear_recurrent_kernel<D, AT, ST, OT, REV, TR, true>, B * w.H * RowGeo<D, ST, true>::WPH, 64, s, args);
    }
    return launch(gdn_linear_recurrent_kernel<D, AT, ST, OT, REV, TR, false>, B * w.H * RowGeo<D, ST, false>::WPH, 64, s, args);
}

Sweep forward_sweep(const LinearArgs& a) {
    const int g = a.H / a.Hk;
    return Sweep{a.T, a.H, g, g, 1, a.q, a.k, a.v, a.decay, a.lengths, a.state, a.state, a.o, 1.0f, a.scale,
                 false, false, false, a.state_dtype};
}

template <int D, typename AT, typename ST>
hipError_t decode_t(const LinearArgs& a, hipStream_t s) {
    return launch_recurrent<D, AT, ST, AT, false, false>(forward_sweep(a), a.B, s);
}

// The three sweeps of the gradients: dq, dk, dv. Where heads share q and k, dq and dk are every
// head's own, in fp32.
struct BackwardSweeps { Sweep s[3]; };

BackwardSweeps backward_sweeps(const LinearBackwardArgs& a, void* dq, void* dk) {
    const int g = a.H / a.Hk;
    const bool f32 = g > 1;
    return BackwardSweeps{{
        Sweep{a.T, a.H, 1, 1, g, a.d_o, a.v, a.k, a.decay, a.lengths, a.state0, nullptr, dq, 1.0f, a.scale,
              false, true, f32, a.state_dtype},
        Sweep{a.T, a.H, 1, 1, g, a.v, a.d_o, a.q, a.decay, a.lengths, a.dstate, nullptr, dk, a.scale, 1.0f,
              true, true, f32, a.state_dtype},
        Sweep{a.T, a.H, g, g, 1, a.k, a.q, a.d_o, a.decay, a.lengths, a.dstate, a.dstate0, a.dv, a.scale, 1.0f,
              true, false, false, a.state_dtype}}};
}

template <typename AT>
hipError_t group_sum(const float* pq, const float* pk, void* dq, void* dk, int64_t rows, int D, int group, hipStream_t s) {
    int64_t n4 = rows * (D / 4);
    int D4 = D / 4;
    AT *q = (AT*)dq, *k = (AT*)dk;
    void* args[] = {&n4, &D4, &group, &pq, &pk, &q, &k};
    const int64_t blocks = (n4 + 255) / 256, most = 1 << 20;  // a dispatch covers fewer than 2^32 work-items
    return hipLaunchKernel((const void*)gdn_linear_group_sum_kernel<AT>,
                           dim3((unsigned)(blocks < most ? blocks : most), 2), dim3(256), args, 0, s);
}

// The sweeps of a short run, token by token.
template <int D, typename AT, typename ST, typename OT>
hipError_t backward_recurrent(const BackwardSweeps& w, int64_t B, hipStream_t s) {
    hipError_t e = launch_recurrent<D, AT, ST, OT, false, true>(w.s[0], B, s);
    if (e != hipSuccess) return e;
    e = launch_recurrent<D, AT, ST, OT, true, true>(w.s[1], B, s);
    if (e != hipSuccess) return e;
    return launch_recurrent<D, AT, ST, AT, true, false>(w.s[2], B, s);
}

template <int D, typename AT, typename ST>
hipError_t backward_t(const LinearBackwardArgs& a, hipStream_t s) {
    const int g = a.H / a.Hk;
    const size_t partial = g > 1 ? (size_t)a.B * a.T * a.H * D : 0;
    float* pq = a.ws;
    float* pk = a.ws + partial;
    float* rest = a.ws + 2 * partial;
    hipError_t e;
    if (a.B > 0) {
        const BackwardSweeps w = backward_sweeps(a, g > 1 ? pq : a.dq, g > 1 ? pk : a.dk);
        if (linear_chunked(a.T, a.H, D)) e = launch_linear_chunk(w.s, 3, a.B, D, a.act, rest, s);
        else if (g > 1) e = backward_recurrent<D, AT, ST, float>(w, a.B, s);
        else e = backward_recurrent<D, AT, ST, AT>(w, a.B, s);
        if (e != hipSuccess) return e;
        if (g > 1 && a.T > 0) {
            e = group_sum<AT>(pq, pk, a.dq, a.dk, a.B * a.T * a.Hk, D, g, s);
            if (e != hipSuccess) return e;
        }
    }
    if (a.ddecay) {  // rest is free again
        float* part = rest;
        int64_t parts = RowGeo<D, ST, false>::WPH;
        if (a.B > 0 && linear_chunked(a.T, a.H, D)) {
            e = launch_linear_tangent(a, rest, &parts, s);
            if (e != hipSuccess) return e;
            part = rest + linear_tangent_state_floats(a.B, a.T, a.H, D);
        } else if (a.B > 0) {
            int64_t B = a.B;
            int T = a.T, H = a.H, group = g;
            const AT *q = (const AT*)a.q, *k = (const AT*)a.k, *v = (const AT*)a.v, *d = (const AT*)a.d_o;
            const ST *s0 = (const ST*)a.state0, *ds = (const ST*)a.dstate;
            const float* decay = a.decay;
            const int32_t* lengths = a.lengths;
            float scale = a.scale;
            void* args[] = {&B, &T, &H, &group, &q, &k, &v, &d, &decay, &lengths, &s0, &ds, &scale, &part};
            e = launch(gdn_linear_tangent_kernel<D, AT, ST>, a.B * a.H * RowGeo<D, ST, false>::WPH, 64, s, args);
            if (e != hipSuccess) return e;
        }
        int64_t n = a.B * parts;
        int H = a.H;
        float* out = a.ddecay;
        void* args[] = {&n, &H, &part, &out};
        e = launch(gdn_linear_ddecay_kernel, a.H, 64, s, args);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// f.template run<D, AT, ST>() for the call's head dim and types.
template <int D, typename AT, typename F>
hipError_t by_state(DType st, F&& f) {
    switch (st) {
        case DType::F32: return f.template run<D, AT, float>();
        case DType::BF16: return f.template run<D, AT, uint16_t>();
        default: return f.template run<D, AT, _Float16>();
    }
}
template <int D, typename F>
hipError_t by_act(DType act, DType st, F&& f) {
    switch (act) {
        case DType::F32: return by_state<D, float>(st, f);
        case DType::BF16: return by_state<D, uint16_t>(st, f);
        default: return by_state<D, _Float16>(st, f);
    }
}
template <typename F>
hipError_t by_dim(int D, DType act, DType st, F&& f) {
    switch (D) {
        case 16: return by_act<16>(act, st, f);
        case 32: return by_act<32>(act, st, f);
        case 64: return by_act<64>(act, st, f);
        default: return by_act<128>(act, st, f);
    }
}

struct DecodeRun {
    const LinearArgs& a;
    hipStream_t s;
    template <int D, typename AT, typename ST> hipError_t run() { return decode_t<D, AT, ST>(a, s); }
};
struct BackwardRun {
    const LinearBackwardArgs& a;
    hipStream_t s;
    template <int D, typename AT, typename ST> hipError_t run() { return backward_t<D, AT, ST>(a, s); }
};

}  // namespace

hipError_t launch_linear_decode(const LinearArgs& a, hipStream_t s) {
    return by_dim(a.D, a.act, a.state_dtype, DecodeRun{a, s});
}

hipError_t launch_linear_prefill(const LinearArgs& a, hipStream_t s) {
    if (!linear_chunked(a.T, a.H, a.D)) return launch_linear_decode(a, s);
    const Sweep w = forward_sweep(a);
    return launch_linear_chunk(&w, 1, a.B, a.D, a.act, a.ws, s);
}

hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t s) {
    return by_dim(a.D, a.act, a.state_dtype, BackwardRun{a, s});
}

}  // namespace gdn
