// The gated linear recurrence h <- alpha h + beta x of every channel, over a few tokens, over prompts, and its
// gradients.
//
// A token is the map h -> alpha h + u of its channel, and maps compose: (P, H) after (p, u) is (P p, P u + H). A
// tile of 64 tokens is split over the waves of a workgroup along the tokens; each lane composes its tokens' maps
// in registers, the waves' maps meet in LDS, and a state at the tile's start then gives every token's.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_linear_common.h"
#include "gdn_scan_launch.h"

namespace gdn {
namespace {

constexpr int64_t kMaxBlocks = 1 << 20;  // of a launch; more work is taken in a loop

// -------------------------------------------------------------------------------------------- gates

// e^-x for x >= 0 within about two steps: the product with log2 e carries its rounding error along.
__device__ __forceinline__ float exp_neg(float x) {
    const float l2e = 1.44269502162933349609375f, l2e_low = 1.925963033500011e-8f, ln2 = 0.693147182464599609375f;
    const float p = -x * l2e;
    const float low = fmaf(-x, l2e_low, fmaf(-x, l2e, -p));
    const float w = __builtin_amdgcn_exp2f(p);
    return w == 0.0f ? w : fmaf(w, low * ln2, w);
}

// A sigmoid and its complement.
struct Sigmoid {
    float up, down;  // sigmoid(a), sigmoid(-a)
    float w;         // e^-|a|
    __device__ __forceinline__ explicit Sigmoid(float a) {
        w = exp_neg(fabsf(a));
        const float r = __builtin_amdgcn_rcpf(1.0f + w), s = w * r;
        up = a >= 0.0f ? r : s;
        down = a >= 0.0f ? s : r;
    }
};

// softplus(a), given w = e^-|a|: ln(1 + w) with what 1 + w rounds away added back.
__device__ __forceinline__ float softplus(float a, float w) {
    const float u = 1.0f + w, lost = w - (u - 1.0f);
    return fmaf(__builtin_amdgcn_logf(u), 0.693147182464599609375f, lost) + (a > 0.0f ? a : 0.0f);
}

// A token's decay. Next to 1 the difference 1 - alpha carries what alpha's rounding would lose, step after
// step, over a long memory; far below 1, alpha does. m holds one of them: -(1 - alpha) with the sign set where
// alpha lies in [1/2, 1], alpha otherwise.
struct Decay {
    float m;
    float lost;  // 1 - alpha
    __device__ __forceinline__ Decay(float alpha, float lost_) : lost(lost_) {
        m = alpha >= 0.5f && lost >= 0.0f ? __uint_as_float(__float_as_uint(lost) | 0x80000000u) : alpha;
    }
};
__device__ __forceinline__ float keep_of(float m) { return (int)__float_as_uint(m) < 0 ? 1.0f : 0.0f; }
// alpha v
__device__ __forceinline__ float decayed(float m, float v) { return fmaf(keep_of(m), v, m * v); }

template <bool RATE>
__device__ __forceinline__ Decay decay_of(float a, const Sigmoid& s, float rate, float* soft) {
    if constexpr (!RATE) {
        return Decay(s.down, s.up);  // exp(-softplus(a)) = sigmoid(-a)
    } else {
        *soft = softplus(a, s.w);
        const float e = rate * *soft;
        const float alpha = __builtin_amdgcn_exp2f(e * -1.44269502162933349609375f);
        // 1 - exp(-e) as its series up to e^5 / 120 for |e| < 1/8 (the next term is below 2^-24 of it)
        const float series = e * fmaf(e, fmaf(e, fmaf(e, fmaf(e, 1.0f / 120, -1.0f / 24), 1.0f / 6), -0.5f), 1.0f);
        return Decay(alpha, fabsf(e) < 0.125f ? series : 1.0f - alpha);
    }
}

// -------------------------------------------------------------------------------------------- memory

__device__ __forceinline__ float state_at(const void* p, DType t, int64_t i) {
    if (t == DType::F32) return ((const float*)p)[i];
    if (t == DType::BF16) return to_f32<uint16_t>(((const uint16_t*)p)[i]);
    return (float)((const _Float16*)p)[i];
}
__device__ __forceinline__ void set_state(void* p, DType t, int64_t i, float x) {
    if (t == DType::F32) ((float*)p)[i] = x;
    else if (t == DType::BF16) ((uint16_t*)p)[i] = from_f32<uint16_t>(x);
    else ((_Float16*)p)[i] = (_Float16)x;
}

// S rows of a segment, V channels a lane; the rows from n on are zeros and are not read.
template <typename T, int V, int S>
struct Rows {
    Run<T, V> r[S];
    __device__ __forceinline__ void load(const RowsView& v, int64_t b, int64_t t0, int64_t c, int n) {
        const T* p = (const T*)v.p + b * v.sb + t0 * v.st + c;
        if (n == S) {
#pragma unroll
            for (int s = 0; s < S; ++s) r[s].load(p + s * v.st);
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (s < n) r[s].load(p + s * v.st); else r[s].zero();
        }
    }
    // Stores the rows before `rows`; those from n on as zeros.
    __device__ __forceinline__ void store(const RowsView& v, int64_t b, int64_t t0, int64_t c, int n, int rows) {
        T* p = (T*)v.p + b * v.sb + t0 * v.st + c;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s >= n) r[s].zero();
            if (s < rows) r[s].store(p + s * v.st);
        }
    }
};

// -------------------------------------------------------------------------------------------- few tokens

// A lane takes V channels of a sequence through its tokens.
template <typename T, int V, bool COUPLED, bool RATE>
__global__ __launch_bounds__(256) void gdn_scan_decode_kernel(ScanArgs a) {
    const int64_t per = a.C / V, total = a.B * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t b = i / per, c = (i - b * per) * V;
        const int n = tokens_of(a.lengths, b, a.T);
        float h[V], rate[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = n > 0 ? state_at(a.state, a.state_dtype, b * a.C + c + v) : 0.0f;
            rate[v] = RATE ? a.rate[c + v] : 1.0f;
        }
        const T* px = (const T*)a.x.p + b * a.x.sb + c;
        const T* pa = (const T*)a.a.p + b * a.a.sb + c;
        const T* pb = (const T*)a.b.p + b * a.b.sb + c;
        T* po = (T*)a.o.p + b * a.o.sb + c;
        for (int t = 0; t < a.T; ++t) {
            Run<T, V> out;
            out.zero();
            if (t < n) {
                Run<T, V> x, ga, gb;
                x.load(px + t * a.x.st);
                ga.load(pa + t * a.a.st);
                if (!COUPLED) gb.load(pb + t * a.b.st);
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float soft;
                    const float av = ga.get(v);
                    const Decay d = decay_of<RATE>(av, Sigmoid(av), rate[v], &soft);
                    const float beta = COUPLED ? d.lost : Sigmoid(gb.get(v)).up;
                    h[v] = fmaf(keep_of(d.m), h[v], fmaf(d.m, h[v], beta * x.get(v)));
                    o[v] = h[v];
                }
                out.set(o);
            }
            out.store(po + t * a.o.st);
        }
        if (n > 0)
#pragma unroll
            for (int v = 0; v < V; ++v) set_state(a.state, a.state_dtype, b * a.C + c + v, h[v]);
    }
}

// -------------------------------------------------------------------------------------------- prompts

// The tile of a workgroup: sequence, chunk of 64 tokens and 64 V channels.
struct Tile {
    int64_t b, j, c;
    int n, rows;   // tokens of the wave's segment within the sequence, and within T
    int64_t t0;
    template <int V, int S>
    __device__ __forceinline__ static Tile at(const ScanArgs& a, int64_t id, int64_t chunks) {
        const int64_t width = (a.C + 64 * V - 1) / (64 * V);
        Tile t;
        const int64_t ct = id % width, r = id / width;
        t.b = r % a.B;
        t.j = r / a.B;
        t.c = ct * 64 * V + (threadIdx.x & 63) * V;
        t.t0 = t.j * kScanChunk + (threadIdx.x >> 6) * S;
        const int64_t len = tokens_of(a.lengths, t.b, a.T);
        t.n = (int)(len < t.t0 ? 0 : (len - t.t0 < S ? len - t.t0 : S));
        t.rows = (int)(a.T < t.t0 ? 0 : (a.T - t.t0 < S ? a.T - t.t0 : S));
        return t;
    }
};

// Forward. ENDS: the maps of whole tiles only, decays to part[0] and ends to part[1] of [B][chunks][C]; otherwise o
// from the tiles' starts (nullptr: one tile, from and to the state).
template <typename T, int V, bool COUPLED, bool RATE, bool ENDS>
__global__ __launch_bounds__(256) void gdn_scan_forward_kernel(ScanArgs a, float* part, const float* starts) {
    constexpr int S = 16, W = kScanChunk / S;
    __shared__ float maps[W][2 * V][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t chunks = (a.T + (int64_t)kScanChunk - 1) / kScanChunk, tiles = a.B * chunks * ((a.C + 64 * V - 1) / (64 * V));
    for (int64_t id = blockIdx.x; id < tiles; id += gridDim.x) {
        const Tile t = Tile::at<V, S>(a, id, chunks);
        const bool on = t.c < a.C;
        const int64_t c = on ? t.c : 0;
        float P[V], H[V], rate[V], ps[S][V], hs[S][V];
        Rows<T, V, S> x, ga, gb;
        ga.load(a.a, t.b, t.t0, c, t.n);
        x.load(a.x, t.b, t.t0, c, t.n);
        if (!COUPLED) gb.load(a.b, t.b, t.t0, c, t.n);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.0f;
            H[v] = 0.0f;
            rate[v] = RATE ? a.rate[c + v] : 1.0f;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (s < t.n) {
                    float soft;
                    const float av = ga.r[s].get(v);
                    const Decay d = decay_of<RATE>(av, Sigmoid(av), rate[v], &soft);
                    const float beta = COUPLED ? d.lost : Sigmoid(gb.r[s].get(v)).up;
                    const float keep = keep_of(d.m);
                    P[v] = fmaf(keep, P[v], d.m * P[v]);
                    H[v] = fmaf(keep, H[v], fmaf(d.m, H[v], beta * x.r[s].get(v)));
                }
                ps[s][v] = P[v];
                hs[s][v] = H[v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            maps[wave][2 * v][lane] = P[v];
            maps[wave][2 * v + 1][lane] = H[v];
        }
        __syncthreads();
        if constexpr (ENDS) {
            if (wave == 0 && on) {
                const int64_t i = (t.b * chunks + t.j) * a.C + c, half = a.B * chunks * a.C;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    for (int w = 1; w < W; ++w) {
                        const float p = maps[w][2 * v][lane];
                        P[v] *= p;
                        H[v] = fmaf(p, H[v], maps[w][2 * v + 1][lane]);
                    }
                    part[i + v] = P[v];
                    part[half + i + v] = H[v];
                }
            }
        } else {
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = starts ? starts[(t.b * chunks + t.j) * a.C + c + v] : state_at(a.state, a.state_dtype, t.b * a.C + c + v);
                for (int w = 0; w < wave; ++w) h[v] = fmaf(maps[w][2 * v][lane], h[v], maps[w][2 * v + 1][lane]);
            }
            if (!starts && a.checkpoints && wave == 0 && on)
#pragma unroll
                for (int v = 0; v < V; ++v) a.checkpoints[t.b * a.C + c + v] = h[v];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = fmaf(ps[s][v], h[v], hs[s][v]);
                x.r[s].set(o);
            }
            if (on) x.store(a.o, t.b, t.t0, c, t.n, t.rows);
            if (!starts) {
                __syncthreads();  // every wave has read the state
                if (wave == W - 1 && on && tokens_of(a.lengths, t.b, a.T) > 0)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        set_state(a.state, a.state_dtype, t.b * a.C + c + v, fmaf(P[v], h[v], H[v]));
            }
        }
        __syncthreads();
    }
}

// Carries a value of every sequence and channel over the chunks' maps, forwards or (REV) backwards: starts takes it
// before each chunk, and `last` after all of them. `first`: nullptr for 0; it may be `last`.
template <bool REV>
__global__ __launch_bounds__(64) void gdn_scan_carry_kernel(int64_t BC, int C, int64_t chunks, const float* part,
                                                            const void* first, void* last, DType dtype, float* starts,
                                                            const int32_t* lengths) {
    const int64_t half = BC * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < BC; i += (int64_t)gridDim.x * 64) {
        const int64_t b = i / C, base = b * chunks * C + (i - b * C);
        float h = first ? state_at(first, dtype, i) : 0.0f;
        for (int64_t k = 0; k < chunks; ++k) {
            const int64_t at = base + (REV ? chunks - 1 - k : k) * C;
            const float p = part[at], u = part[half + at];
            starts[at] = h;
            h = fmaf(p, h, u);
        }
        if (last && (REV || !lengths || lengths[b] > 0)) set_state(last, dtype, i, h);
    }
}

// Backward. ENDS: the maps of whole tiles from the last token to the first, r -> alpha (do + r), as above. Otherwise
// the gradients, from the states at the tiles' starts and the adjoints r behind their ends.
template <typename T, int V, bool COUPLED, bool RATE, bool ENDS>
__global__ __launch_bounds__(512) void gdn_scan_backward_kernel(ScanArgs a, float* part, const float* starts,
                                                                const float* behind, float* rates) {
    constexpr int S = 8, W = kScanChunk / S;
    __shared__ float maps[W][3 * V][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t chunks = (a.T + (int64_t)kScanChunk - 1) / kScanChunk, tiles = a.B * chunks * ((a.C + 64 * V - 1) / (64 * V));
    for (int64_t id = blockIdx.x; id < tiles; id += gridDim.x) {
        const Tile t = Tile::at<V, S>(a, id, chunks);
        const bool on = t.c < a.C;
        const int64_t c = on ? t.c : 0, at = (t.b * chunks + t.j) * a.C + c;
        Rows<T, V, S> x, ga, gb, go;
        ga.load(a.a, t.b, t.t0, c, t.n);
        go.load(a.d_o, t.b, t.t0, c, t.n);
        if (!ENDS) {
            x.load(a.x, t.b, t.t0, c, t.n);
            if (!COUPLED) gb.load(a.b, t.b, t.t0, c, t.n);
        }
        float P[V], H[V], R[V], rate[V];
        float m[S][V], hb[S][V], pb[S][V];  // decays; the state before each token: pb h + hb from the segment's start
        float slope[S][V], soft[S][V];      // sigmoid(a) rate, softplus(a)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.0f;
            H[v] = 0.0f;
            R[v] = 0.0f;
            rate[v] = RATE ? a.rate[c + v] : 1.0f;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float av = ga.r[s].get(v);
                const Sigmoid sg(av);
                soft[s][v] = RATE || !rates ? 0.0f : softplus(av, sg.w);
                const Decay d = decay_of<RATE>(av, sg, rate[v], &soft[s][v]);
                m[s][v] = d.m;
                slope[s][v] = sg.up * rate[v];
                pb[s][v] = P[v];
                hb[s][v] = H[v];
                if (s < t.n) {
                    const float keep = keep_of(d.m);
                    P[v] = fmaf(keep, P[v], d.m * P[v]);
                    if (!ENDS) {
                        const float beta = COUPLED ? d.lost : Sigmoid(gb.r[s].get(v)).up;
                        H[v] = fmaf(keep, H[v], fmaf(d.m, H[v], beta * x.r[s].get(v)));
                    }
                }
            }
        }
#pragma unroll
        for (int s = S - 1; s >= 0; --s)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (s < t.n) R[v] = decayed(m[s][v], go.r[s].get(v) + R[v]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            maps[wave][3 * v][lane] = P[v];
            maps[wave][3 * v + 1][lane] = H[v];
            maps[wave][3 * v + 2][lane] = R[v];
        }
        __syncthreads();
        if constexpr (ENDS) {
            if (wave == 0 && on) {
                const int64_t half = a.B * chunks * a.C;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float p = 1.0f, r = 0.0f;
                    for (int w = W - 1; w >= 0; --w) {
                        const float q = maps[w][3 * v][lane];
                        p *= q;
                        r = fmaf(q, r, maps[w][3 * v + 2][lane]);
                    }
                    part[at + v] = p;
                    part[half + at + v] = r;
                }
            }
        } else {
            float h[V], r[V], total[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = starts ? starts[at + v] : (a.state0 ? state_at(a.state0, a.state_dtype, t.b * a.C + c + v) : 0.0f);
                for (int w = 0; w < wave; ++w) h[v] = fmaf(maps[w][3 * v][lane], h[v], maps[w][3 * v + 1][lane]);
                r[v] = behind ? behind[at + v] : (a.dstate ? state_at(a.dstate, a.state_dtype, t.b * a.C + c + v) : 0.0f);
                for (int w = W - 1; w > wave; --w) r[v] = fmaf(maps[w][3 * v][lane], r[v], maps[w][3 * v + 2][lane]);
                total[v] = 0.0f;
            }
#pragma unroll
            for (int s = S - 1; s >= 0; --s) {
                float ox[V], oa[V], ob[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float xv = x.r[s].get(v), g = go.r[s].get(v) + r[v];
                    const float before = fmaf(pb[s][v], h[v], hb[s][v]);
                    const float next = decayed(m[s][v], g);
                    const float e = next * (COUPLED ? xv - before : -before);
                    oa[v] = e * slope[s][v];
                    if (COUPLED) {
                        const float alpha = (int)__float_as_uint(m[s][v]) < 0 ? 0.0f : m[s][v];
                        ox[v] = g * ((int)__float_as_uint(m[s][v]) < 0 ? -m[s][v] : 1.0f - alpha);
                    } else {
                        const Sigmoid sb(gb.r[s].get(v));
                        ox[v] = g * sb.up;
                        ob[v] = g * xv * (sb.up * sb.down);
                    }
                    if (s < t.n) {
                        r[v] = next;
                        total[v] = fmaf(e, soft[s][v], total[v]);
                    }
                }
                x.r[s].set(ox);
                ga.r[s].set(oa);
                if (!COUPLED) gb.r[s].set(ob);
            }
            if (on) {
                x.store(a.dx, t.b, t.t0, c, t.n, t.rows);
                ga.store(a.da, t.b, t.t0, c, t.n, t.rows);
                if (!COUPLED) gb.store(a.db, t.b, t.t0, c, t.n, t.rows);
            }
            if (!behind && a.dstate0 && wave == 0 && on)
#pragma unroll
                for (int v = 0; v < V; ++v) set_state(a.dstate0, a.state_dtype, t.b * a.C + c + v, r[v]);
            if (rates) {
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; ++v) maps[wave][v][lane] = total[v];
                __syncthreads();
                if (wave == 0 && on)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float sum = 0.0f;
                        for (int w = 0; w < W; ++w) sum += maps[w][v][lane];
                        rates[at + v] = sum;
                    }
            }
        }
        __syncthreads();
    }
}

// Sums over the rows of part [n][C], in 64 bits: a lane per channel and a sixteenth of the rows.
__global__ __launch_bounds__(1024) void gdn_scan_rates_kernel(const float* part, int64_t n, int C, float* out) {
    __shared__ double sum[16][64];
    const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < C; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        double v = 0.0;
        if (c < C) {
#pragma unroll 8
            for (int64_t i = row; i < n; i += 16) v += part[i * C + c];
        }
        sum[row][lane] = v;
        __syncthreads();
        if (row == 0 && c < C) {
            for (int i = 1; i < 16; ++i) v += sum[i][lane];
            out[c] = (float)v;
        }
        __syncthreads();
    }
}

// dstate0 of a call without tokens.
__global__ __launch_bounds__(256) void gdn_scan_copy_kernel(int64_t n, const void* from, void* to, DType dtype) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        set_state(to, dtype, i, from ? state_at(from, dtype, i) : 0.0f);
}

// -------------------------------------------------------------------------------------------- launches

unsigned blocks_of(int64_t n) { return (unsigned)(n < 1 ? 1 : (n < kMaxBlocks ? n : kMaxBlocks)); }

hipError_t launch(const void* kernel, int64_t blocks, int threads, hipStream_t s, void** args) {
    return hipLaunchKernel(kernel, dim3(blocks_of(blocks)), dim3((unsigned)threads), args, 0, s);
}

bool fits(const RowsView& v, const ScanArgs& a, size_t bytes) {
    const size_t es = a.act == DType::F32 ? 4 : 2;
    auto whole = [&](int64_t s, int64_t n) { return n <= 1 || (size_t)s * es % bytes == 0; };
    return !v.p || ((uintptr_t)v.p % bytes == 0 && whole(v.sb, a.B) && whole(v.st, a.T));
}

// Whether every row of the call splits into vectors of v values.
bool vector_fits(const ScanArgs& a, int v) {
    const size_t bytes = (size_t)v * (a.act == DType::F32 ? 4 : 2);
    return a.C % v == 0 && fits(a.x, a, bytes) && fits(a.a, a, bytes) && fits(a.b, a, bytes) && fits(a.o, a, bytes) &&
           fits(a.d_o, a, bytes) && fits(a.dx, a, bytes) && fits(a.da, a, bytes) && fits(a.db, a, bytes);
}

template <typename T, int V, bool COUPLED, bool RATE>
hipError_t decode(const ScanArgs& a, hipStream_t s) {
    ScanArgs args = a;
    void* p[] = {&args};
    return launch((const void*)gdn_scan_decode_kernel<T, V, COUPLED, RATE>, (a.B * (a.C / V) + 255) / 256, 256, s, p);
}

hipError_t carry(const ScanArgs& a, bool rev, const float* part, const void* first, void* last, float* starts, hipStream_t s) {
    int64_t BC = a.B * a.C, chunks = scan_chunks(a.T);
    int C = a.C;
    DType dtype = a.state_dtype;
    const int32_t* lengths = a.lengths;
    void* p[] = {&BC, &C, &chunks, &part, &first, &last, &dtype, &starts, &lengths};
    return launch(rev ? (const void*)gdn_scan_carry_kernel<true> : (const void*)gdn_scan_carry_kernel<false>, (BC + 63) / 64, 64, s, p);
}

template <int V>
int64_t tiles_of(const ScanArgs& a) { return a.B * scan_chunks(a.T) * (((int64_t)a.C + 64 * V - 1) / (64 * V)); }

template <typename T, int V, bool COUPLED, bool RATE>
hipError_t forward_ends(const ScanArgs& a, float* part, hipStream_t s) {
    ScanArgs args = a;
    const float* none = nullptr;
    void* p[] = {&args, &part, &none};
    return launch((const void*)gdn_scan_forward_kernel<T, V, COUPLED, RATE, true>, tiles_of<V>(a), 256, s, p);
}

template <typename T, int V, bool COUPLED, bool RATE>
hipError_t prefill(const ScanArgs& a, hipStream_t s) {
    ScanArgs args = a;
    const int64_t chunks = scan_chunks(a.T), n = a.B * chunks * a.C;
    float *part = a.ws, *starts = nullptr;
    if (chunks > 1) {
        starts = a.checkpoints ? a.checkpoints : a.ws + 2 * n;
        hipError_t e = forward_ends<T, V, COUPLED, RATE>(a, part, s);
        if (e != hipSuccess) return e;
        e = carry(a, false, part, a.state, a.state, starts, s);
        if (e != hipSuccess) return e;
    }
    void* p[] = {&args, &part, &starts};
    return launch((const void*)gdn_scan_forward_kernel<T, V, COUPLED, RATE, false>, tiles_of<V>(a), 256, s, p);
}

template <typename T, int V, bool COUPLED, bool RATE>
hipError_t backward(const ScanArgs& a, hipStream_t s) {
    ScanArgs args = a;
    const int64_t chunks = scan_chunks(a.T), n = a.B * chunks * a.C;
    float* part = a.ws;
    const float* starts = a.checkpoints;
    float* behind = nullptr;
    hipError_t e;
    if (chunks > 1) {
        if (!starts) {
            float* made = a.ws + 2 * n;
            e = forward_ends<T, V, COUPLED, RATE>(a, part, s);
            if (e != hipSuccess) return e;
            e = carry(a, false, part, a.state0, nullptr, made, s);
            if (e != hipSuccess) return e;
            starts = made;
        }
        behind = a.ws + 3 * n;
        const float* none = nullptr;
        float* no_rates = nullptr;
        void* p[] = {&args, &part, &none, &none, &no_rates};
        e = launch((const void*)gdn_scan_backward_kernel<T, V, COUPLED, RATE, true>, tiles_of<V>(a), 512, s, p);
        if (e != hipSuccess) return e;
        e = carry(a, true, part, a.dstate, a.dstate0, behind, s);
        if (e != hipSuccess) return e;
    }
    float* rates = a.drate ? a.ws + 4 * n : nullptr;
    const float* after = behind;
    void* p[] = {&args, &part, &starts, &after, &rates};
    e = launch((const void*)gdn_scan_backward_kernel<T, V, COUPLED, RATE, false>, tiles_of<V>(a), 512, s, p);
    if (e != hipSuccess || !rates) return e;
    const float* in = rates;
    int64_t rows = a.B * chunks;
    int C = a.C;
    float* out = a.drate;
    void* p2[] = {&in, &rows, &C, &out};
    return launch((const void*)gdn_scan_rates_kernel, ((int64_t)C + 63) / 64, 1024, s, p2);
}

// f.template run<T, V, COUPLED, RATE>() for the call's type, vector width (wide, 2 or 1) and gates.
template <typename T, int V, typename F>
hipError_t by_gates(const ScanArgs& a, F f) {
    if (a.b.p) return a.rate ? f.template run<T, V, false, true>() : f.template run<T, V, false, false>();
    return a.rate ? f.template run<T, V, true, true>() : f.template run<T, V, true, false>();
}
template <typename T, typename F>
hipError_t by_width(const ScanArgs& a, F f) {
    constexpr int WIDE = F::wide / (int)sizeof(T);
    if constexpr (WIDE > 2) {
        if (vector_fits(a, WIDE)) return by_gates<T, WIDE>(a, f);
    }
    return vector_fits(a, 2) ? by_gates<T, 2>(a, f) : by_gates<T, 1>(a, f);
}
template <typename F>
hipError_t by_type(const ScanArgs& a, F f) {
    switch (a.act) {
        case DType::F32: return by_width<float>(a, f);
        case DType::BF16: return by_width<uint16_t>(a, f);
        default: return by_width<_Float16>(a, f);
    }
}

struct DecodeRun {
    static constexpr int wide = 16;
    const ScanArgs& a;
    hipStream_t s;
    template <typename T, int V, bool COUPLED, bool RATE>
    hipError_t run() { return decode<T, V, COUPLED, RATE>(a, s); }
};
struct PrefillRun {
    static constexpr int wide = 0;
    const ScanArgs& a;
    hipStream_t s;
    template <typename T, int V, bool COUPLED, bool RATE>
    hipError_t run() { return prefill<T, V, COUPLED, RATE>(a, s); }
};
struct BackwardRun {
    static constexpr int wide = 0;
    const ScanArgs& a;
    hipStream_t s;
    template <typename T, int V, bool COUPLED, bool RATE>
    hipError_t run() { return backward<T, V, COUPLED, RATE>(a, s); }
};

}  // namespace

hipError_t launch_scan_decode(const ScanArgs& a, hipStream_t s) { return by_type(a, DecodeRun{a, s}); }

hipError_t launch_scan_prefill(const ScanArgs& a, hipStream_t s) { return by_type(a, PrefillRun{a, s}); }

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
    if (a.B == 0 || a.T == 0) {  // no tokens: dstate0 = dstate, drate = 0
        int64_t n = a.B * a.C;
        if (a.dstate0 && n > 0) {
            const void* from = a.dstate;
            void* to = a.dstate0;
            DType dtype = a.state_dtype;
            void* p[] = {&n, &from, &to, &dtype};
            hipError_t e = launch((const void*)gdn_scan_copy_kernel, (n + 255) / 256, 256, s, p);
            if (e != hipSuccess) return e;
        }
        if (!a.drate) return hipSuccess;
        const float* in = nullptr;
        int64_t rows = 0;
        int C = a.C;
        float* out = a.drate;
        void* p[] = {&in, &rows, &C, &out};
        return launch((const void*)gdn_scan_rates_kernel, ((int64_t)C + 63) / 64, 1024, s, p);
    }
    return by_type(a, BackwardRun{a, s});
}

}  // namespace gdn
