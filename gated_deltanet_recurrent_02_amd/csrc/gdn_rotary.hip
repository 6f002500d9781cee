// The rotation of queries and keys by their position, and their norm in every head, with gradients.
//
// A row is a head of one token. A group of G lanes (a power of two up to a wave) holds a row in registers: each
// lane has units of two vectors of V values, the two partners of V pairs (half layout: vectors R/2 apart;
// interleaved: neighbouring vectors) or two vectors of the part that is not turned. So the pairs, and all of
// a row but the sum of its squares, stay within a lane, and the lane's V cosines and sines serve every head
// of its token: angles are formed once for up to UN heads.
// All of it is bound by memory.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_linear_common.h"
#include "gdn_rotary_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int64_t kMaxBlocks = 1 << 20;  // of a dimension of the grid; more tokens are taken in a loop

// What a kernel needs besides the tensors.
struct RotaryPlan {
    RotaryArgs a;
    int tokens;        // B T
    int units, turned; // of a row; of its pairs
    int lg;            // log2 of a group's lanes
    int lhs;           // log2 of the heads that a wave has side by side; the rest of its groups take other tokens
};

// Where a lane's two vectors of unit u start. The second may be missing past the turned part.
template <int V>
__device__ __forceinline__ void unit_at(const RotaryArgs& a, int units, int turned, int u, int& e0, int& e1, bool& has0,
                                        bool& has1) {
    has0 = u < units;
    if (u < turned) {
        e0 = a.interleaved ? 2 * u * V : u * V;
        e1 = a.interleaved ? e0 + V : e0 + a.R / 2;
    } else {
        e0 = a.R + 2 * (u - turned) * V;
        e1 = e0 + V;
    }
    has1 = has0 && e1 < a.D;
}

// Cosines and sines of the V pairs from pair i on at position p, times the amplitude. The angle in turns,
// reduced to [-1/2, 1/2] in 64 bits, is then exact to 2^-25 of a turn in 32.
template <int V>
__device__ __forceinline__ void angles(const RotaryArgs& a, int i, int p, float* c, float* s) {
    const double turns_per_radian = 0.15915494309189533577;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        double t = (double)p * a.freqs[i + e] * turns_per_radian;
        t -= __builtin_rint(t);
        float sn, cs;
        sincospif((float)(2.0 * t), &sn, &cs);
        c[e] = cs * a.amplitude;
        s[e] = a.transposed ? -sn * a.amplitude : sn * a.amplitude;
    }
}

// Turns the pairs of two vectors. Pairs lie across the vectors, or (interleaved, V > 1) within each of them.
template <int V>
__device__ __forceinline__ void turn(bool within, const float* c, const float* s, float* x, float* y) {
    if (V > 1 && within) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float x0 = x[e], x1 = x[e + 1], y0 = y[e], y1 = y[e + 1];
            x[e] = x0 * c[e / 2] - x1 * s[e / 2];
            x[e + 1] = x0 * s[e / 2] + x1 * c[e / 2];
            y[e] = y0 * c[(V + e) / 2] - y1 * s[(V + e) / 2];
            y[e + 1] = y0 * s[(V + e) / 2] + y1 * c[(V + e) / 2];
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float x0 = x[e], y0 = y[e];
            x[e] = x0 * c[e] - y0 * s[e];
            y[e] = x0 * s[e] + y0 * c[e];
        }
    }
}

// Sums over aligned groups of 2^lg lanes, N at once; every lane of a group gets the same value.
template <int N>
__device__ __forceinline__ void group_sum(float* x, int lg) {
    if (lg >= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += dpp_mov<0xB1>(x[i]);
    }
    if (lg >= 2) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += dpp_mov<0x4E>(x[i]);
    }
    if (lg >= 3) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += dpp_mov<0x141>(x[i]);
    }
    if (lg >= 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += dpp_mov<0x140>(x[i]);
    }
    if (lg >= 5) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor(x[i], 16);
    }
    if (lg >= 6) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor(x[i], 32);
    }
}

template <typename T>
__device__ __forceinline__ const T* row_of(const HeadsView& v, int b, int t, int h) {
    return (const T*)v.p + (int64_t)b * v.sb + (int64_t)t * v.st + (int64_t)h * v.sh;
}

// The forward passes: rope (either direction), and with NORM the norm before it. Every group takes its
// heads h0, h0 + HS, ... (UN of them) of one token at a time.
template <typename T, int V, int KU, int UN, bool NORM>
__global__ __launch_bounds__(kThreads) void gdn_rotary_kernel(RotaryPlan p) {
    const RotaryArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & ((1 << p.lg) - 1), group = lane >> p.lg;
    const int HS = 1 << p.lhs, lts = 6 - p.lg - p.lhs;
    const int H = a.Hq + a.Hk, h0 = blockIdx.y * HS * UN + (group & (HS - 1));
    int e0[KU], e1[KU];
    bool has0[KU], has1[KU];
#pragma unroll
    for (int k = 0; k < KU; ++k) unit_at<V>(a, p.units, p.turned, li + (k << p.lg), e0[k], e1[k], has0[k], has1[k]);

    for (int64_t n = (((int64_t)blockIdx.x * kWaves + wave) << lts) + (group >> p.lhs); n < p.tokens;
         n += ((int64_t)gridDim.x * kWaves) << lts) {
        const int b = (int)n / a.T, t = (int)n - b * a.T;
        const bool here = t < tokens_of(a.lengths, b, a.T);
        Run<T, V> r0[UN][KU], r1[UN][KU];
        T* out[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int h = h0 + i * HS;
            const bool q = h < a.Hq;
            const RotarySet& set = q ? a.q : a.k;
            const int hh = q ? h : h - a.Hq;
            out[i] = h < H ? const_cast<T*>(row_of<T>(set.y, b, t, hh)) : nullptr;
            const T* in = row_of<T>(set.x, b, t, hh);
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                if (here && h < H && has0[k]) r0[i][k].load(in + e0[k]); else r0[i][k].zero();
                if (here && h < H && has1[k]) r1[i][k].load(in + e1[k]); else r1[i][k].zero();
            }
        }
        if (here) {
            const int pos = a.positions ? a.positions[n] : t;
            float ss[UN];
            if constexpr (NORM) {
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    ss[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < KU; ++k)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float x = r0[i][k].get(e), y = r1[i][k].get(e);
                            ss[i] = fmaf(x, x, ss[i]);
                            ss[i] = fmaf(y, y, ss[i]);
                        }
                }
                group_sum<UN>(ss, p.lg);
#pragma unroll
                for (int i = 0; i < UN; ++i) ss[i] = 1.0f / sqrtf(ss[i] / (float)a.D + a.eps);
            }
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                const int u = li + (k << p.lg);
                float c[V], s[V];
                if (u < p.turned) angles<V>(a, u * V, pos, c, s);
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const int h = h0 + i * HS;
                    float x[V], y[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) { x[e] = r0[i][k].get(e); y[e] = r1[i][k].get(e); }
                    if constexpr (NORM) {
                        const bool q = h < a.Hq;
                        const float* w = q ? a.q.w : a.k.w;
                        if (w && a.per_head) w += (int64_t)(q ? h : h - a.Hq) * a.D;
                        Run<float, V> w0, w1;
                        const bool on = w && h < H;
                        if (on && has0[k]) w0.load(w + e0[k]);
                        if (on && has1[k]) w1.load(w + e1[k]);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            x[e] *= ss[i];
                            y[e] *= ss[i];
                            if (on && has0[k]) x[e] *= w0.get(e);
                            if (on && has1[k]) y[e] *= w1.get(e);
                        }
                    }
                    if (u < p.turned) turn<V>(a.interleaved, c, s, x, y);
                    r0[i][k].set(x);
                    r1[i][k].set(y);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (out[i]) {
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    if (has0[k]) r0[i][k].store(out[i] + e0[k]);
                    if (has1[k]) r1[i][k].store(out[i] + e1[k]);
                }
            }
    }
}

// The norm's backward: dx of every row, and each workgroup's sums of g n over its tokens for every head
// (part [slabs][H][D], where wanted). A group keeps UN heads over all its tokens, so their sums stay in registers.
template <typename T, int V, int KU, int UN>
__global__ __launch_bounds__(kThreads) void gdn_rotary_norm_backward_kernel(RotaryPlan p, float* part) {
    const RotaryArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & ((1 << p.lg) - 1), group = lane >> p.lg;
    const int HS = 1 << p.lhs, lts = 6 - p.lg - p.lhs;
    const int H = a.Hq + a.Hk, h0 = blockIdx.y * HS * UN + (group & (HS - 1));
    int e0[KU], e1[KU];
    bool has0[KU], has1[KU];
#pragma unroll
    for (int k = 0; k < KU; ++k) unit_at<V>(a, p.units, p.turned, li + (k << p.lg), e0[k], e1[k], has0[k], has1[k]);
    float acc[UN][KU][2 * V];
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) acc[i][k][e] = 0.0f;

    for (int64_t n = (((int64_t)blockIdx.x * kWaves + wave) << lts) + (group >> p.lhs); n < p.tokens;
         n += ((int64_t)gridDim.x * kWaves) << lts) {
        const int b = (int)n / a.T, t = (int)n - b * a.T;
        const bool here = t < tokens_of(a.lengths, b, a.T);
        Run<T, V> x0[UN][KU], x1[UN][KU], g0[UN][KU], g1[UN][KU];
        T* out[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int h = h0 + i * HS;
            const bool q = h < a.Hq;
            const RotarySet& set = q ? a.q : a.k;
            const int hh = q ? h : h - a.Hq;
            out[i] = h < H ? const_cast<T*>(row_of<T>(set.y, b, t, hh)) : nullptr;
            const T* in = row_of<T>(set.x, b, t, hh);
            const T* dy = row_of<T>(set.dy, b, t, hh);
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                const bool on0 = here && h < H && has0[k], on1 = here && h < H && has1[k];
                if (on0) x0[i][k].load(in + e0[k]); else x0[i][k].zero();
                if (on1) x1[i][k].load(in + e1[k]); else x1[i][k].zero();
                if (on0) g0[i][k].load(dy + e0[k]); else g0[i][k].zero();
                if (on1) g1[i][k].load(dy + e1[k]); else g1[i][k].zero();
            }
        }
        if (here) {
            const int pos = a.positions ? a.positions[n] : t;
            float c[KU][V], s[KU][V];
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                const int u = li + (k << p.lg);
                if (u < p.turned) angles<V>(a, u * V, pos, c[k], s[k]);
            }
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int h = h0 + i * HS;
                const bool q = h < a.Hq;
                const float* w = q ? a.q.w : a.k.w;
                if (w && a.per_head) w += (int64_t)(q ? h : h - a.Hq) * a.D;
                float sums[2] = {0.0f, 0.0f};  // of x^2, and of g w x
                float gw0[KU][V], gw1[KU][V], d0[KU][V], d1[KU][V];
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    const int u = li + (k << p.lg);
#pragma unroll
                    for (int e = 0; e < V; ++e) { d0[k][e] = g0[i][k].get(e); d1[k][e] = g1[i][k].get(e); }
                    if (u < p.turned) turn<V>(a.interleaved, c[k], s[k], d0[k], d1[k]);
                    Run<float, V> w0, w1;
                    const bool on = w && h < H;
                    if (on && has0[k]) w0.load(w + e0[k]);
                    if (on && has1[k]) w1.load(w + e1[k]);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float x = x0[i][k].get(e), y = x1[i][k].get(e);
                        gw0[k][e] = on && has0[k] ? d0[k][e] * w0.get(e) : d0[k][e];
                        gw1[k][e] = on && has1[k] ? d1[k][e] * w1.get(e) : d1[k][e];
                        sums[0] = fmaf(x, x, sums[0]);
                        sums[0] = fmaf(y, y, sums[0]);
                        sums[1] = fmaf(gw0[k][e], x, sums[1]);
                        sums[1] = fmaf(gw1[k][e], y, sums[1]);
                    }
                }
                group_sum<2>(sums, p.lg);
                const float r = 1.0f / sqrtf(sums[0] / (float)a.D + a.eps);
                const float m = sums[1] * r / (float)a.D;  // mean of g w n
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    float o0[V], o1[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float n0 = x0[i][k].get(e) * r, n1 = x1[i][k].get(e) * r;
                        acc[i][k][e] = fmaf(d0[k][e], n0, acc[i][k][e]);
                        acc[i][k][V + e] = fmaf(d1[k][e], n1, acc[i][k][V + e]);
                        o0[e] = r * (gw0[k][e] - n0 * m);
                        o1[e] = r * (gw1[k][e] - n1 * m);
                    }
                    g0[i][k].set(o0);
                    g1[i][k].set(o1);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (out[i]) {
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    if (has0[k]) g0[i][k].store(out[i] + e0[k]);
                    if (has1[k]) g1[i][k].store(out[i] + e1[k]);
                }
            }
    }
    if (!part) return;

    // The workgroup's sums of every head: over the groups that share it in a wave, then over the waves, head
    // by head, so that LDS holds one value per lane at a time.
    __shared__ float sum[kWaves][64][2 * V + 1];
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) sum[wave][lane][e] = acc[i][k][e];
            __syncthreads();
            const int h = h0 + i * HS;
            // the lanes of the wave's first token, one head each, take the others' values
            if ((group >> p.lhs) == 0 && h < H) {
                for (int e = wave; e < 2 * V; e += kWaves) {
                    float v = 0.0f;
                    for (int j = 0; j < kWaves; ++j)
                        for (int g = 0; g < (1 << lts); ++g) v += sum[j][lane + (g << (p.lg + p.lhs))][e];
                    const bool second = e >= V;
                    if (second ? has1[k] : has0[k])
                        part[((int64_t)blockIdx.x * H + h) * a.D + (second ? e1[k] + e - V : e0[k] + e)] = v;
                }
            }
        }
}

// Sums over the first axis of part [n][columns], a lane per column and 1/4 of the rows: out[column]. Where
// `second` is given, the columns from `split` on go there.
__global__ __launch_bounds__(256) void gdn_rotary_sum_kernel(const float* part, int n, int64_t columns, float* out,
                                                             float* second, int64_t split) {
    __shared__ float sum[4][64];
    const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < columns; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float v = 0.0f;
        if (c < columns) {
#pragma unroll 8
            for (int i = row; i < n; i += 4) v += part[(int64_t)i * columns + c];
        }
        sum[row][lane] = v;
        __syncthreads();
        if (row == 0 && c < columns) {
            v = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
            if (c < split) { if (out) out[c] = v; } else if (second) second[c - split] = v;
        }
        __syncthreads();
    }
}

// --------------------------------------------------------------------------------------- launches

bool fits(const HeadsView& v, int H, const RotaryArgs& a, size_t bytes) {
    const size_t es = a.dtype == DType::F32 ? 4 : 2;
    auto whole = [&](int64_t s, int64_t n) { return n <= 1 || (size_t)s * es % bytes == 0; };
    return (uintptr_t)v.p % bytes == 0 && whole(v.sb, a.B) && whole(v.st, a.T) && whole(v.sh, H);
}

// The widest vectors, in values, that every row of the call starts and splits at.
int vector_of(const RotaryArgs& a, bool backward) {
    const int es = a.dtype == DType::F32 ? 4 : 2;
    for (int v = 16 / es; v > 1; v /= 2) {
        const size_t bytes = (size_t)v * es;
        if (a.R % (2 * v) != 0 || (a.D - a.R) % v != 0) continue;
        if (!fits(a.q.x, a.Hq, a, bytes) || !fits(a.q.y, a.Hq, a, bytes)) continue;
        if (backward && !fits(a.q.dy, a.Hq, a, bytes)) continue;
        if (a.Hk) {
            if (!fits(a.k.x, a.Hk, a, bytes) || !fits(a.k.y, a.Hk, a, bytes)) continue;
            if (backward && !fits(a.k.dy, a.Hk, a, bytes)) continue;
        }
        return v;
    }
    return 1;
}

int log2_up(int n) {
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}

RotaryPlan plan(const RotaryArgs& a, int v) {
    RotaryPlan p;
    p.a = a;
    p.tokens = (int)(a.B * a.T);
    p.turned = a.R / (2 * v);
    p.units = p.turned + ((a.D - a.R) / v + 1) / 2;
    p.lg = log2_up(p.units < 64 ? p.units : 64);
    const int lh = log2_up(a.Hq + a.Hk);
    p.lhs = lh < 6 - p.lg ? lh : 6 - p.lg;
    return p;
}

// Workgroups along the tokens and the heads.
dim3 grid_of(const RotaryPlan& p, int un) {
    const int64_t per = (int64_t)kWaves << (6 - p.lg - p.lhs);
    const int64_t x = (p.tokens + per - 1) / per, heads = (int64_t)un << p.lhs;
    const int64_t y = (p.a.Hq + p.a.Hk + heads - 1) / heads;
    return dim3((unsigned)(x < kMaxBlocks ? x : kMaxBlocks), (unsigned)y);
}

hipError_t launch(const void* kernel, dim3 grid, hipStream_t s, void** args) {
    return hipLaunchKernel(kernel, grid, dim3(kThreads), args, 0, s);
}

template <typename T, int V, int KU, bool NORM>
hipError_t forward(const RotaryArgs& a, hipStream_t s) {
    RotaryPlan p = plan(a, V);
    void* args[] = {&p};
    if constexpr (KU == 1) {
        const dim3 g = grid_of(p, 4);
        if ((int64_t)g.x * g.y >= 1024) return launch((const void*)gdn_rotary_kernel<T, V, KU, 4, NORM>, g, s, args);
    }
    return launch((const void*)gdn_rotary_kernel<T, V, KU, 1, NORM>, grid_of(p, 1), s, args);
}

template <typename T, int V, int KU>
hipError_t backward(const RotaryArgs& a, hipStream_t s) {
    RotaryPlan p = plan(a, V);
    constexpr int UN = KU == 1 ? 2 : 1;
    const bool params = a.q.dw || a.k.dw;
    const int H = a.Hq + a.Hk;
    dim3 g = grid_of(p, UN);
    const int64_t slabs = rotary_slabs(p.tokens, H);
    if (params && g.x > slabs) g.x = (unsigned)slabs;
    float* part = params ? a.ws : nullptr;
    void* args[] = {&p, &part};
    hipError_t e = launch((const void*)gdn_rotary_norm_backward_kernel<T, V, KU, UN>, g, s, args);
    if (e != hipSuccess || !params) return e;
    // over the slabs; then, where the heads share a weight, over the heads
    int n = (int)g.x;
    int64_t columns = (int64_t)H * a.D, split = (int64_t)a.Hq * a.D;
    float *out = a.q.dw, *second = a.k.dw;
    float* heads = a.ws + (size_t)slabs * H * a.D;
    if (!a.per_head) { out = heads; second = heads + split; }
    const int64_t blocks = (columns + 63) / 64;
    {
        const float* in = part;
        void* args2[] = {&in, &n, &columns, &out, &second, &split};
        e = launch((const void*)gdn_rotary_sum_kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), s, args2);
    }
    if (e != hipSuccess || a.per_head) return e;
    columns = a.D;
    split = a.D;
    float* none = nullptr;
    for (int i = 0; i < 2; ++i) {
        float* dw = i ? a.k.dw : a.q.dw;
        if (!dw) continue;
        const float* in = i ? second : out;
        n = i ? a.Hk : a.Hq;
        void* args2[] = {&in, &n, &columns, &dw, &none, &split};
        e = launch((const void*)gdn_rotary_sum_kernel, dim3((unsigned)((a.D + 63) / 64)), s, args2);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// f.template run<T, V, KU>() for the call's type and vector width. KU units per lane hold the longest row
// of 512 values: 256 units of single values, 128 of two, 64 of four or more.
template <typename T, typename F>
hipError_t by_width(const RotaryArgs& a, int v, F f) {
    const int units = plan(a, v).units;
    if constexpr (sizeof(T) == 2) {
        if (v == 8) return f.template run<T, 8, 1>();
    }
    if (v == 4) return f.template run<T, 4, 1>();
    if (v == 2) return units <= 64 ? f.template run<T, 2, 1>() : f.template run<T, 2, 2>();
    return units <= 64 ? f.template run<T, 1, 1>() : f.template run<T, 1, 4>();
}

template <typename F>
hipError_t by_type(const RotaryArgs& a, int v, F f) {
    switch (a.dtype) {
        case DType::F32: return by_width<float>(a, v, f);
        case DType::BF16: return by_width<uint16_t>(a, v, f);
        default: return by_width<_Float16>(a, v, f);
    }
}

template <bool NORM>
struct ForwardRun {
    const RotaryArgs& a;
    hipStream_t s;
    template <typename T, int V, int KU>
    hipError_t run() { return forward<T, V, KU, NORM>(a, s); }
};

struct BackwardRun {
    const RotaryArgs& a;
    hipStream_t s;
    template <typename T, int V, int KU>
    hipError_t run() { return backward<T, V, KU>(a, s); }
};

}  // namespace

hipError_t launch_rope(const RotaryArgs& a, hipStream_t s) {
    return by_type(a, vector_of(a, false), ForwardRun<false>{a, s});
}

hipError_t launch_qk_norm_rope(const RotaryArgs& a, hipStream_t s) {
    return by_type(a, vector_of(a, false), ForwardRun<true>{a, s});
}

hipError_t launch_qk_norm_rope_backward(const RotaryArgs& a, hipStream_t s) {
    if (a.B == 0 || a.T == 0) {  // no rows: the sums are 0
        int n = 0;
        const float* in = nullptr;
        float* none = nullptr;
        for (int i = 0; i < 2; ++i) {
            float* dw = i ? a.k.dw : a.q.dw;
            if (!dw) continue;
            int64_t columns = (int64_t)(a.per_head ? (i ? a.Hk : a.Hq) : 1) * a.D, split = columns;
            const int64_t blocks = (columns + 63) / 64;
            void* args[] = {&in, &n, &columns, &dw, &none, &split};
            hipError_t e = launch((const void*)gdn_rotary_sum_kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), s, args);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    return by_type(a, vector_of(a, true), BackwardRun{a, s});
}

}  // namespace gdn
