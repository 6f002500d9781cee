// The rotation of queries and keys by their position, and their norm in every head, with gradients.
//
// A row is a head of one token. A group of G lanes (a power of two up to a wave) holds a row in registers: each
// lane has units of two vectors of V values, the two partners of V pairs (half layout: vectors R/2 apart;
// interleaved: neighbouring vectors) or two vectors of the part that is not turned. So the pairs, and all of
// a row but the sum of its squares, stay within a lane, and the lane's V cosines and sines serve every head
// of its token: angles are formed once for up to UN heads. A workgroup has heads of q or of k alone, so that pointers and
// strides are scalars. Loads are streamed, since each value is read once (with one head a group, the norm took 150 us without
// and 138 with).
// All of it is bound by memory. 16384 tokens of 48 + 16 heads of 128 bf16 values (537 MB): the rotation 101 us (5.3 TB/s), norm
// and rotation 104, the norm's gradients (805 MB) 171 to 178 and 5 for the join of the weights' sums.
// Rows whose R or D - R are no multiples of a vector, or whose strides or starts are none, take narrower vectors throughout, down to
// single values: 16384 tokens of 32 + 8 heads of 50 bf16 values 71 us (1.8 TB/s), of 75 129 (1.5), of 64 36 (4.7).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_linear_common.h"
#include "gdn_rotary_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int64_t kMaxBlocks = 1 << 20;  // of a dimension of the grid; more tokens are taken in a loop

// What a kernel needs besides the tensors. A workgroup has heads of q alone, or of k alone.
struct RotaryPlan {
    RotaryArgs a;
    int tokens;           // B T
    int units, turned;    // of a row; of its pairs
    int lg;               // log2 of a group's lanes
    int lhs[2];           // log2 of the heads that a wave has side by side, for q and k; its other groups take other tokens
    int heads[2];         // of a workgroup, in all
    int blocks[2];        // workgroups along the heads of q and of k
};

// The part of a workgroup and a group of lanes in it.
struct Place {
    const RotarySet& set;
    int which;                 // 0: q, 1: k
    int H, HS, lts;            // heads of the set, heads side by side, log2 of the tokens side by side
    int block;                 // among the set's workgroups along the heads
    int li, group, h0;         // lane in its group, group in its wave, first head
    __device__ __forceinline__ Place(const RotaryPlan& p)
        : set((int)blockIdx.y < p.blocks[0] ? p.a.q : p.a.k), which((int)blockIdx.y < p.blocks[0] ? 0 : 1) {
        const int lane = threadIdx.x & 63, lhs = p.lhs[which];
        H = which ? p.a.Hk : p.a.Hq;
        HS = 1 << lhs;
        lts = 6 - p.lg - lhs;
        block = (int)blockIdx.y - (which ? p.blocks[0] : 0);
        li = lane & ((1 << p.lg) - 1);
        group = lane >> p.lg;
        h0 = block * p.heads[which] + (group & (HS - 1));
    }
    // The token of the wave's group, and the distance to its next one.
    __device__ __forceinline__ int64_t first(const RotaryPlan& p) const {
        return (((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) << lts) + (group >> p.lhs[which]);
    }
    __device__ __forceinline__ int64_t step() const { return ((int64_t)gridDim.x * kWaves) << lts; }
};

// 1 / sqrt(m), within two steps; the instruction takes no subnormal numbers.
__device__ __forceinline__ float inverse_root(float m) {
    if (__builtin_expect(m < 1e-30f, 0)) return 1.0f / sqrtf(m);
    return __builtin_amdgcn_rsqf(m);
}

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

// Cosines and sines of the V pairs from pair i on at position p, times the amplitude. The angle is reduced in 64 bits,
// to quarter turns q and the rest f in [-1/2, 1/2] of one, where the Taylor series of sine and cosine need five terms
// for 2^-25.
template <int V>
__device__ __forceinline__ void angles(const RotaryArgs& a, int i, int p, float* c, float* s) {
    const double turns_per_radian = 0.15915494309189533577;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        double t = (double)p * a.freqs[i + e] * turns_per_radian;
        t = 4.0 * (t - __builtin_rint(t));
        const double q = __builtin_rint(t);
        const float f = (float)(t - q), f2 = f * f;
        const int n = (int)q;
        const float sn = f * fmaf(f2, fmaf(f2, fmaf(f2, fmaf(f2, 1.60441184787e-4f, -4.68175413531e-3f), 7.96926262461e-2f),
                                           -6.45964097506e-1f), 1.57079632679f);
        const float cs = fmaf(f2, fmaf(f2, fmaf(f2, fmaf(f2, 9.19260274839e-4f, -2.08634807633e-2f), 2.53669507901e-1f),
                                       -1.23370055014f), 1.0f);
        const float u = n & 1 ? sn : cs, v = n & 1 ? cs : sn;  // of the quarter turns only their parity is left
        const float cr = (n + 1) & 2 ? -u : u, sr = n & 2 ? -v : v;
        c[e] = cr * a.amplitude;
        s[e] = a.transposed ? -sr * a.amplitude : sr * a.amplitude;
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
__device__ __forceinline__ T* token_of(const HeadsView& v, int b, int t) {
    return (T*)v.p + (int64_t)b * v.sb + (int64_t)t * v.st;
}

// The forward passes: rope (either direction), and with NORM the norm before it. A group takes UN heads, h0 and
// h0 + HS, of a token at a time: two where there are workgroups enough (norm and rotation by calls, two heads 112 us; four
// take 234 registers and 127, eight 151; two after two of the same token, with the angles kept, 117).
template <typename T, int V, int KU, int UN, bool NORM>
__global__ __launch_bounds__(kThreads) void gdn_rotary_kernel(RotaryPlan p) {
    const RotaryArgs& a = p.a;
    const Place at(p);
    int e0[KU], e1[KU];
    bool has0[KU], has1[KU];
#pragma unroll
    for (int k = 0; k < KU; ++k) unit_at<V>(a, p.units, p.turned, at.li + (k << p.lg), e0[k], e1[k], has0[k], has1[k]);
    const float per_value = 1.0f / (float)a.D;
    Run<float, V> w0[KU], w1[KU];
    const bool weights = NORM && at.set.w, shared = weights && !a.per_head;
#pragma unroll
    for (int k = 0; k < KU; ++k) {
        if (shared && has0[k]) w0[k].load(at.set.w + e0[k]); else w0[k].zero();
        if (shared && has1[k]) w1[k].load(at.set.w + e1[k]); else w1[k].zero();
    }

    for (int64_t n = at.first(p); n < p.tokens; n += at.step()) {
        const int b = (int)n / a.T, t = (int)n - b * a.T;
        const bool here = t < tokens_of(a.lengths, b, a.T);
        const T* in = token_of<const T>(at.set.x, b, t) + (int64_t)at.h0 * at.set.x.sh;
        T* out = token_of<T>(at.set.y, b, t) + (int64_t)at.h0 * at.set.y.sh;
        Run<T, V> r0[UN][KU], r1[UN][KU];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const bool on = here && at.h0 + i * at.HS < at.H;
            const T* row = in + (int64_t)(i * at.HS) * at.set.x.sh;
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                if (on && has0[k]) r0[i][k].template load<true>(row + e0[k]); else r0[i][k].zero();
                if (on && has1[k]) r1[i][k].template load<true>(row + e1[k]); else r1[i][k].zero();
            }
        }
        if (here) {
            const int pos = a.positions ? a.positions[n] : t;
            float c[KU][V], s[KU][V];
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                const int u = at.li + (k << p.lg);
                if (u < p.turned) angles<V>(a, u * V, pos, c[k], s[k]);
            }
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
                for (int i = 0; i < UN; ++i) ss[i] = inverse_root(fmaf(ss[i], per_value, a.eps));
            }
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                const int u = at.li + (k << p.lg);
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    float x[V], y[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) { x[e] = r0[i][k].get(e); y[e] = r1[i][k].get(e); }
                    if constexpr (NORM) {
                        if (weights && a.per_head) {
                            const bool on = at.h0 + i * at.HS < at.H;
                            const float* w = at.set.w + (int64_t)(at.h0 + i * at.HS) * a.D;
                            if (on && has0[k]) w0[k].load(w + e0[k]);
                            if (on && has1[k]) w1[k].load(w + e1[k]);
                        }
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            x[e] *= ss[i];
                            y[e] *= ss[i];
                            if (weights) {
                                x[e] *= w0[k].get(e);
                                y[e] *= w1[k].get(e);
                            }
                        }
                    }
                    if (u < p.turned) turn<V>(a.interleaved, c[k], s[k], x, y);
                    r0[i][k].set(x);
                    r1[i][k].set(y);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (at.h0 + i * at.HS < at.H) {
                T* row = out + (int64_t)(i * at.HS) * at.set.y.sh;
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    if (has0[k]) r0[i][k].store(row + e0[k]);
                    if (has1[k]) r1[i][k].store(row + e1[k]);
                }
            }
    }
}

// The norm's backward: dx of every row, and each workgroup's sums of g n over its tokens (part, where wanted). A group
// keeps UN heads over all its tokens, so their sums stay in registers, in 32 bits as the terms are: n terms one
// after the other (the tokens of a lane, then the slabs, 4 or 16 rows of them at a time) are off by at most n 2^-24 of their magnitude;
// 1503 tokens of 10 heads come out within 1.6e-7 with everything else, in 64 bits 0.7e-7.
template <typename T, int V, int KU, int UN>
__global__ __launch_bounds__(kThreads) void gdn_rotary_norm_backward_kernel(RotaryPlan p, float* part) {
    const RotaryArgs& a = p.a;
    const Place at(p);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int e0[KU], e1[KU];
    bool has0[KU], has1[KU];
#pragma unroll
    for (int k = 0; k < KU; ++k) unit_at<V>(a, p.units, p.turned, at.li + (k << p.lg), e0[k], e1[k], has0[k], has1[k]);
    const float per_value = 1.0f / (float)a.D;
    float acc[UN][KU][2 * V];
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) acc[i][k][e] = 0.0f;

    for (int64_t n = at.first(p); n < p.tokens; n += at.step()) {
        const int b = (int)n / a.T, t = (int)n - b * a.T;
        const bool here = t < tokens_of(a.lengths, b, a.T);
        const T* in = token_of<const T>(at.set.x, b, t) + (int64_t)at.h0 * at.set.x.sh;
        const T* dy = token_of<const T>(at.set.dy, b, t) + (int64_t)at.h0 * at.set.dy.sh;
        T* out = token_of<T>(at.set.y, b, t) + (int64_t)at.h0 * at.set.y.sh;
        Run<T, V> x0[UN][KU], x1[UN][KU], g0[UN][KU], g1[UN][KU];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const bool on = here && at.h0 + i * at.HS < at.H;
            const T* rx = in + (int64_t)(i * at.HS) * at.set.x.sh;
            const T* rg = dy + (int64_t)(i * at.HS) * at.set.dy.sh;
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                if (on && has0[k]) x0[i][k].template load<true>(rx + e0[k]); else x0[i][k].zero();
                if (on && has1[k]) x1[i][k].template load<true>(rx + e1[k]); else x1[i][k].zero();
                if (on && has0[k]) g0[i][k].template load<true>(rg + e0[k]); else g0[i][k].zero();
                if (on && has1[k]) g1[i][k].template load<true>(rg + e1[k]); else g1[i][k].zero();
            }
        }
        if (here) {
            const int pos = a.positions ? a.positions[n] : t;
            float c[KU][V], s[KU][V];
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                const int u = at.li + (k << p.lg);
                if (u < p.turned) angles<V>(a, u * V, pos, c[k], s[k]);
            }
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // one head at a time: interleaved they take registers for two
                const int h = at.h0 + i * at.HS;
                const bool weights = at.set.w && h < at.H;
                const float* w = weights && a.per_head ? at.set.w + (int64_t)h * a.D : at.set.w;
                float sums[2] = {0.0f, 0.0f};  // of x^2, and of g w x
                float gw0[KU][V], gw1[KU][V], d0[KU][V], d1[KU][V];
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    const int u = at.li + (k << p.lg);
#pragma unroll
                    for (int e = 0; e < V; ++e) { d0[k][e] = g0[i][k].get(e); d1[k][e] = g1[i][k].get(e); }
                    if (u < p.turned) turn<V>(a.interleaved, c[k], s[k], d0[k], d1[k]);
                    Run<float, V> w0, w1;
                    w0.zero();
                    w1.zero();
                    if (weights && has0[k]) w0.load(w + e0[k]);
                    if (weights && has1[k]) w1.load(w + e1[k]);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float x = x0[i][k].get(e), y = x1[i][k].get(e);
                        gw0[k][e] = at.set.w ? d0[k][e] * w0.get(e) : d0[k][e];
                        gw1[k][e] = at.set.w ? d1[k][e] * w1.get(e) : d1[k][e];
                        sums[0] = fmaf(x, x, sums[0]);
                        sums[0] = fmaf(y, y, sums[0]);
                        sums[1] = fmaf(gw0[k][e], x, sums[1]);
                        sums[1] = fmaf(gw1[k][e], y, sums[1]);
                    }
                }
                group_sum<2>(sums, p.lg);
                const float r = inverse_root(fmaf(sums[0], per_value, a.eps));
                const float m = sums[1] * r * per_value;  // mean of g w n
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    float o0[V], o1[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float n0 = x0[i][k].get(e) * r, n1 = x1[i][k].get(e) * r;
                        acc[i][k][e] = fmaf(d0[k][e], n0, acc[i][k][e]);
                        acc[i][k][V + e] = fmaf(d1[k][e], n1, acc[i][k][V + e]);
                        o0[e] = r * fmaf(-n0, m, gw0[k][e]);
                        o1[e] = r * fmaf(-n1, m, gw1[k][e]);
                    }
                    g0[i][k].set(o0);
                    g1[i][k].set(o1);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (at.h0 + i * at.HS < at.H) {
                T* row = out + (int64_t)(i * at.HS) * at.set.y.sh;
#pragma unroll
                for (int k = 0; k < KU; ++k) {
                    if (has0[k]) g0[i][k].store(row + e0[k]);
                    if (has1[k]) g1[i][k].store(row + e1[k]);
                }
            }
    }
    if (!part) return;

    // The workgroup's sums: over the groups that share a head in a wave, then over the waves; and, where the heads share
    // a weight, over the heads. One head of each group at a time, so that LDS stays small.
    __shared__ float sum[kWaves][64][2 * V + 1];
    constexpr int E = (2 * V + kWaves - 1) / kWaves;   // elements of a unit that a wave adds up
    const int groups = 64 >> p.lg;                     // group g: head g % HS
    const int H = a.Hq + a.Hk, before = at.which ? a.Hq : 0;
    float all[KU][E];
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j) all[k][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) sum[wave][lane][e] = acc[i][k][e];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int e = wave + j * kWaves, h = at.h0 + i * at.HS;
                const bool second = e >= V;
                if (e >= 2 * V) continue;
                if (a.per_head) {
                    if (at.group >= at.HS || h >= at.H) continue;  // the groups of the wave's first token, one head each
                    float v = 0.0f;
                    for (int w = 0; w < kWaves; ++w)
                        for (int g = at.group; g < groups; g += at.HS) v += sum[w][at.li + (g << p.lg)][e];
                    if (second ? has1[k] : has0[k])
                        part[((int64_t)blockIdx.x * H + before + h) * a.D + (second ? e1[k] + e - V : e0[k] + e)] = v;
                } else if (at.group == 0) {  // (heads past H have added nothing)
                    for (int g = 0; g < groups; ++g)
                        for (int w = 0; w < kWaves; ++w) all[k][j] += sum[w][at.li + (g << p.lg)][e];
                }
            }
        }
    if (a.per_head || at.group != 0) return;
    float* to = part + ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * a.D;  // a row a workgroup
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int e = wave + j * kWaves;
            if (e >= 2 * V) continue;
            const bool second = e >= V;
            if (second ? has1[k] : has0[k]) to[second ? e1[k] + e - V : e0[k] + e] = all[k][j];
        }
}

// Weights shared by the heads: out[set] is the sum of the rows first[set] .. first[set] + count[set] of every slab of
// part [slabs][rows][D], a lane per column and 1/16 of the rows.
struct JoinPlan {
    const float* part;
    int slabs, rows, D, first[2], count[2];
    float* out[2];
};
__global__ __launch_bounds__(1024) void gdn_rotary_join_kernel(JoinPlan p) {
    __shared__ float sum[16][64];
    const int lane = threadIdx.x & 63, row = threadIdx.x >> 6, set = blockIdx.y, c = blockIdx.x * 64 + lane;
    const int count = p.count[set], n = p.slabs * count;
    float v = 0.0f;
    if (c < p.D) {
#pragma unroll 4
        for (int i = row; i < n; i += 16) {
            const int slab = i / count;
            v += p.part[((int64_t)slab * p.rows + p.first[set] + i - slab * count) * p.D + c];
        }
    }
    sum[row][lane] = v;
    __syncthreads();
    if (row == 0 && c < p.D && p.out[set]) {
        for (int i = 1; i < 16; ++i) v += sum[i][lane];
        p.out[set][c] = v;
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

// `un` heads for a group at once.
RotaryPlan plan(const RotaryArgs& a, int v, int un) {
    RotaryPlan p;
    p.a = a;
    p.tokens = (int)(a.B * a.T);
    p.turned = a.R / (2 * v);
    p.units = p.turned + ((a.D - a.R) / v + 1) / 2;
    p.lg = log2_up(p.units < 64 ? p.units : 64);
    for (int i = 0; i < 2; ++i) {
        const int H = i ? a.Hk : a.Hq, lh = log2_up(H);
        p.lhs[i] = lh < 6 - p.lg ? lh : 6 - p.lg;
        p.heads[i] = un << p.lhs[i];
        p.blocks[i] = (H + p.heads[i] - 1) / p.heads[i];
    }
    return p;
}

// Workgroups along the tokens (as many as the set with the fewest tokens side by side needs) and the heads.
dim3 grid_of(const RotaryPlan& p) {
    int64_t x = 0;
    for (int i = 0; i < 2; ++i) {
        const int64_t per = (int64_t)kWaves << (6 - p.lg - p.lhs[i]), need = (p.tokens + per - 1) / per;
        if (p.blocks[i] && need > x) x = need;
    }
    return dim3((unsigned)(x < kMaxBlocks ? x : kMaxBlocks), (unsigned)(p.blocks[0] + p.blocks[1]));
}

hipError_t launch(const void* kernel, dim3 grid, hipStream_t s, void** args) {
    return hipLaunchKernel(kernel, grid, dim3(kThreads), args, 0, s);
}

template <typename T, int V, int KU, bool NORM>
hipError_t forward(const RotaryArgs& a, hipStream_t s) {
    RotaryPlan p;
    void* args[] = {&p};
    if constexpr (KU == 1) {
        // Two heads a group from 2048 workgroups on. Norm and rotation, bf16, D = 128, one head and two: 48 + 16 heads, 512 workgroups
        // of two heads 4.7 and 4.9 us, 1024 6.8 and 6.0, 2048 11.4 and 9.3, 32768 132 and 100. With 8 + 2 heads two are slower
        // (1024 workgroups 5.5 and 6.2, 4096 14.4 and 16.5): the groups that hold k are half empty.
        p = plan(a, V, 2);
        const dim3 g = grid_of(p);
        if ((int64_t)g.x * g.y >= 2048) return launch((const void*)gdn_rotary_kernel<T, V, KU, 2, NORM>, g, s, args);
    }
    p = plan(a, V, 1);
    return launch((const void*)gdn_rotary_kernel<T, V, KU, 1, NORM>, grid_of(p), s, args);
}

template <typename T, int V, int KU>
hipError_t backward(const RotaryArgs& a, hipStream_t s) {
    // Two heads of eight values a vector fill the registers (bf16: 187 us, with one 181); of four they do not (fp32, half the
    // tokens: 164 us, with one 194).
    constexpr int UN = KU == 1 && V < 8 ? 2 : 1;
    RotaryPlan p = plan(a, V, UN);
    const bool params = a.q.dw || a.k.dw;
    const int H = a.Hq + a.Hk;
    dim3 g = grid_of(p);
    const int64_t slabs = rotary_slabs(p.tokens, H);
    // Every workgroup ends with its sums, so it takes two rounds of tokens where that leaves enough of them (1024 tokens of
    // 32 + 8 heads of 128: 32.9 us with one round each, 24.7 with two, 23.8 with four; 64 tokens 10.2, 11.7 and 15.0).
    if (params && (int64_t)g.x * g.y >= 512) g.x = (g.x + 1) / 2;
    if (params && g.x > slabs) g.x = (unsigned)slabs;
    float* part = params ? a.ws : nullptr;
    void* args[] = {&p, &part};
    hipError_t e = launch((const void*)gdn_rotary_norm_backward_kernel<T, V, KU, UN>, g, s, args);
    if (e != hipSuccess || !params) return e;
    int n = (int)g.x;
    if (a.per_head) {
        int64_t columns = (int64_t)H * a.D, split = (int64_t)a.Hq * a.D;
        float *out = a.q.dw, *second = a.k.dw;
        const float* in = part;
        const int64_t blocks = (columns + 63) / 64;
        void* args2[] = {&in, &n, &columns, &out, &second, &split};
        return launch((const void*)gdn_rotary_sum_kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), s, args2);
    }
    JoinPlan j;
    j.part = part;
    j.slabs = n;
    j.rows = (int)g.y;
    j.D = a.D;
    j.first[0] = 0;
    j.count[0] = p.blocks[0];
    j.first[1] = p.blocks[0];
    j.count[1] = p.blocks[1];
    j.out[0] = a.q.dw;
    j.out[1] = a.k.dw;
    void* args2[] = {&j};
    return hipLaunchKernel((const void*)gdn_rotary_join_kernel, dim3((unsigned)((a.D + 63) / 64), a.Hk ? 2 : 1), dim3(1024), args2, 0, s);
}

// f.template run<T, V, KU>() for the call's type and vector width. KU units per lane hold the longest row
// of 512 values: 256 units of single values, 128 of two, 64 of four or more.
template <typename T, typename F>
hipError_t by_width(const RotaryArgs& a, int v, F f) {
    const int units = plan(a, v, 1).units;
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
