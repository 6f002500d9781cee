// Layer norm of a layer's output on gfx950 (CDNA4), forward and backward. Per row r of x [rows][C]
// with the affine of group r mod G,
//     n = (x - mean) rstd,  mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),  y = n w + b
//     g = dy w,  dx = rstd (g - mean_C(g) - n mean_C(g n)),  dw = sum_rows dy n,  db = sum_rows dy.
// Sums are fp32 where a row's registers hold the terms of one lane (at most 24 of a row), 64 bits over a row
// that is longer; the variance is summed from centred values.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_linear_common.h"
#include "gdn_linear_launch.h"

namespace gdn {
namespace {

// VE elements of a row, 16 bytes, at any element alignment (the hardware takes unaligned vector
// accesses); nv < VE of them at a row's end.
typedef uint32_t words2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t words4_t __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Vec {
    static constexpr int VE = 16 / (int)sizeof(T);
    using words = std::conditional_t<sizeof(T) == 4, words4_t, words2_t>;
    uint32_t w[4];

    __device__ __forceinline__ void load(const T* p, int nv) {
        if (nv >= VE) {
            const words x = *(const words*)p;
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
            w[0] = w[1] = w[2] = w[3] = 0u;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (e >= nv) continue;
                if constexpr (sizeof(T) == 4) w[e] = *(const uint32_t*)(p + e);
                else w[e / 2] |= (uint32_t)*(const uint16_t*)(p + e) << (16 * (e & 1));
            }
        }
    }
    __device__ __forceinline__ float get(int e) const { return Elem<T>::get(w, e); }
    static __device__ __forceinline__ void store(T* p, const float* f, int nv) {
        Run<T, VE> r;
        r.set(f);
        if (nv >= VE) {
            *(words*)p = words{r.w[0], r.w[1], r.w[2], r.w[3]};
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (e >= nv) continue;
                if constexpr (sizeof(T) == 4) *(uint32_t*)(p + e) = r.w[e];
                else *(uint16_t*)(p + e) = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
            }
        }
    }
};

// VE floats of an affine row (fp32, any 4-byte alignment), or a constant without one.
template <int VE>
__device__ __forceinline__ void load_affine(float* f, const float* p, size_t at, int nv, float without) {
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = without;
    if (p == nullptr) return;
    if (nv >= VE) {
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) {
            const words4_t x = *(const words4_t*)(p + at + 4 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = __uint_as_float(x[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (e < nv) f[e] = p[at + e];
    }
}

// A workgroup's sums: N values at once over the LR lanes of a row (a part of a wave, or the whole
// workgroup); every lane of the row gets the same values.
template <int LR, int NT, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*lds)[NT / 64]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane_sum<(LR < 64 ? LR : 64)>(x[i]);
    if constexpr (LR > 64) {
        constexpr int NW = NT / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i][threadIdx.x >> 6] = x[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = lds[i][0];
#pragma unroll
            for (int w = 1; w < NW; ++w) s += lds[i][w];
            x[i] = s;
        }
    }
}

// Forward and backward keep a row in registers: LR lanes of a workgroup of NT hold one, K vectors
// each (vector j of lane l is number l + j LR). A unit is one group of rows (one affine row) and
// one slab of its tokens; a workgroup takes a unit's tokens NT / LR at a time, so that the affine
// row stays in registers and, backward, its gradient is summed there. The next row is loaded while
// the present one is computed.
template <typename T, int LR, int K, int NT>
__global__ __launch_bounds__(NT) void gdn_layer_norm_rows_kernel(
    int64_t tokens, int G, int C, int slabs, const T* x, const float* __restrict__ weight,
    const float* __restrict__ bias, T* y, float* __restrict__ mean, float* __restrict__ rstd, float eps) {
    constexpr int VE = Vec<T>::VE, RB = NT / LR;
    __shared__ float lds[1][NT / 64];
    const int l = threadIdx.x % LR, sub = threadIdx.x / LR;
    int nv[K];
#pragma unroll
    for (int j = 0; j < K; ++j) nv[j] = min(max(C - (l + j * LR) * VE, 0), VE);
    const float inv = 1.0f / (float)C;
    const int64_t units = (int64_t)G * slabs;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int g = (int)(u % G);
        const int64_t step = (int64_t)slabs * RB;
        float w[K][VE], bi[K][VE];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            load_affine<VE>(w[j], weight, (size_t)g * C + (l + j * LR) * VE, nv[j], 1.0f);
            load_affine<VE>(bi[j], bias, (size_t)g * C + (l + j * LR) * VE, nv[j], 0.0f);
        }
        const int64_t first = (u / G) * RB;  // the same trips for every row of the workgroup
        Vec<T> v[K];
        if (first + sub < tokens) {
            const T* p = x + ((size_t)(first + sub) * G + g) * C;
#pragma unroll
            for (int j = 0; j < K; ++j) v[j].load(p + (l + j * LR) * VE, nv[j]);
        }
        for (int64_t t0 = first; t0 < tokens; t0 += step) {
            const int64_t t = t0 + sub;
            Vec<T> next[K];
            if (t + step < tokens) {
                const T* p = x + ((size_t)(t + step) * G + g) * C;
#pragma unroll
                for (int j = 0; j < K; ++j) next[j].load(p + (l + j * LR) * VE, nv[j]);
            }
            float s[1] = {0.0f};
            if (t < tokens) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (nv[j] > 0) {
#pragma unroll
                        for (int e = 0; e < VE; ++e) s[0] += v[j].get(e);  // zeros past the row
                    }
            }
            row_sums<LR, NT, 1>(s, lds);
            const float m = s[0] * inv;
            s[0] = 0.0f;
            if (t < tokens) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (nv[j] == VE) {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const float d = v[j].get(e) - m;
                            s[0] = fmaf(d, d, s[0]);
                        }
                    } else {
                        for (int e = 0; e < nv[j]; ++e) {  // a row's end
                            const float d = to_f32<T>(x[((size_t)t * G + g) * C + (l + j * LR) * VE + e]) - m;
                            s[0] = fmaf(d, d, s[0]);
                        }
                    }
            }
            row_sums<LR, NT, 1>(s, lds);
            const float r = 1.0f / sqrtf(s[0] * inv + eps);
            if (t < tokens) {
                const size_t row = (size_t)t * G + g;
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (nv[j] > 0) {
                        float f[VE];
#pragma unroll
                        for (int e = 0; e < VE; ++e) f[e] = fmaf((v[j].get(e) - m) * r, w[j][e], bi[j][e]);
                        Vec<T>::store(y + row * C + (l + j * LR) * VE, f, nv[j]);
                    }
                if (mean && l == 0) { mean[row] = m; rstd[row] = r; }
            }
#pragma unroll
            for (int j = 0; j < K; ++j) v[j] = next[j];
        }
    }
}

// part[0][slab][G * C] takes the slab's sums of dy n and part[1][slab][G * C] those of dy, if wanted.
template <typename T, int LR, int K, int NT>
__global__ __launch_bounds__(NT) void gdn_layer_norm_rows_backward_kernel(
    int64_t tokens, int G, int C, int slabs, const T* dy, const T* __restrict__ x,
    const float* __restrict__ weight, const float* __restrict__ mean, const float* __restrict__ rstd, T* dx,
    float* __restrict__ part) {
    constexpr int VE = Vec<T>::VE, RB = NT / LR;
    __shared__ float lds[2][NT / 64];
    __shared__ float sums[RB > 1 ? NT * K * VE : 1];
    const int l = threadIdx.x % LR, sub = threadIdx.x / LR;
    int nv[K];
#pragma unroll
    for (int j = 0; j < K; ++j) nv[j] = min(max(C - (l + j * LR) * VE, 0), VE);
    const float inv = 1.0f / (float)C;
    const int64_t units = (int64_t)G * slabs;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int g = (int)(u % G);
        const int64_t slab = u / G, step = (int64_t)slabs * RB;
        float w[K][VE], aw[K][VE], ab[K][VE];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            load_affine<VE>(w[j], weight, (size_t)g * C + (l + j * LR) * VE, nv[j], 1.0f);
#pragma unroll
            for (int e = 0; e < VE; ++e) aw[j][e] = ab[j][e] = 0.0f;
        }
        const int64_t first = slab * RB;
        Vec<T> v[K], d[K];
        float m = 0.0f, r = 0.0f;
        const auto fetch = [&](int64_t t, Vec<T>(&v)[K], Vec<T>(&d)[K], float& m, float& r) {
            const size_t row = (size_t)t * G + g;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                v[j].load(x + row * C + (l + j * LR) * VE, nv[j]);
                d[j].load(dy + row * C + (l + j * LR) * VE, nv[j]);
            }
            m = mean[row];
            r = rstd[row];
        };
        if (first + sub < tokens) fetch(first + sub, v, d, m, r);
        for (int64_t t0 = first; t0 < tokens; t0 += step) {
            const int64_t t = t0 + sub;
            Vec<T> vn[K], dn[K];
            float mn = 0.0f, rn = 0.0f;
            if (t + step < tokens) fetch(t + step, vn, dn, mn, rn);
            float s[2] = {0.0f, 0.0f};
            if (t < tokens) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (nv[j] > 0) {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {  // past the row dy and n are 0 (-m r may be an infinity)
                            const float n = e < nv[j] ? (v[j].get(e) - m) * r : 0.0f;
                            const float dyv = d[j].get(e), gg = dyv * w[j][e];
                            s[0] += gg;
                            s[1] = fmaf(gg, n, s[1]);
                            aw[j][e] = fmaf(dyv, n, aw[j][e]);
                            ab[j][e] += dyv;
                        }
                    }
            }
            row_sums<LR, NT, 2>(s, lds);
            const float sg = s[0] * inv, sn = s[1] * inv;
            if (t < tokens) {
                const size_t row = (size_t)t * G + g;
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (nv[j] > 0) {
                        float f[VE];
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const float n = (v[j].get(e) - m) * r;
                            f[e] = r * (d[j].get(e) * w[j][e] - sg - n * sn);
                        }
                        Vec<T>::store(dx + row * C + (l + j * LR) * VE, f, nv[j]);
                    }
            }
#pragma unroll
            for (int j = 0; j < K; ++j) { v[j] = vn[j]; d[j] = dn[j]; }
            m = mn;
            r = rn;
        }
        if (!part) continue;
        const size_t GC = (size_t)G * C;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float* out = part + ((size_t)which * slabs + slab) * GC + (size_t)g * C;
            if constexpr (RB > 1) {  // join the workgroup's rows, in their order
                __syncthreads();
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        sums[sub * LR * K * VE + (l + j * LR) * VE + e] = which ? ab[j][e] : aw[j][e];
                __syncthreads();
                for (int c = threadIdx.x; c < C; c += NT) {
                    float t = sums[c];
#pragma unroll
                    for (int i = 1; i < RB; ++i) t += sums[i * LR * K * VE + c];
                    out[c] = t;
                }
            } else {
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        if (e < nv[j]) out[(l + j * LR) * VE + e] = which ? ab[j][e] : aw[j][e];
            }
        }
        if constexpr (RB > 1) __syncthreads();
    }
}

// Joins the slabs of part[which][slab][GC]: 64 columns a workgroup, every wave a share of the slabs.
__global__ __launch_bounds__(1024) void gdn_layer_norm_slabs_kernel(int64_t GC, int slabs,
                                                                    const float* __restrict__ part,
                                                                    float* __restrict__ dw,
                                                                    float* __restrict__ db) {
    __shared__ float lds[16][64];
    float* out = blockIdx.y ? db : dw;
    if (!out) return;
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < GC; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + l;
        float s = 0.0f;
        if (c < GC) {
            const float* p = part + (size_t)blockIdx.y * slabs * GC + c;
#pragma unroll 4
            for (int i = wave; i < slabs; i += 16) s += p[(size_t)i * GC];
        }
        lds[wave][l] = s;
        __syncthreads();
        if (wave == 0 && c < GC) {
#pragma unroll
            for (int i = 1; i < 16; ++i) s += lds[i][l];
            out[c] = s;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------ rows too long for registers

// Sum over the workgroup; every thread gets the same value. A lane adds up to C / 1024 values one after
// another: in fp32 the mean of 2^24 values of one sign was off by 1e-5 of itself, of 2^31 by 2%. The loop
// waits for memory: with four loads at a time 2^26 fp32 values in rows of 12288 take 152 us forward and
// 351 backward in 64 bits, one fp32 sum a lane (and loads one at a time) 206 and 332.
template <int NW>
__device__ __forceinline__ double block_sum(double x, double* lds) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) s += lds[i];
    return s;
}

// One workgroup per row at a time, rows in strides of the grid.
template <int NW, typename T>
__global__ __launch_bounds__(64 * NW) void gdn_layer_norm_kernel(
    int64_t rows, int G, int C, const T* x, const float* __restrict__ weight, const float* __restrict__ bias, T* y,
    float* __restrict__ mean, float* __restrict__ rstd, float eps) {
    __shared__ double lds[NW];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + (size_t)row * C;
        T* yr = y + (size_t)row * C;
        const size_t w0 = (size_t)(row % G) * C;
        double s = 0.0;
#pragma unroll 4
        for (uint32_t c = threadIdx.x; c < (uint32_t)C; c += 64 * NW) s += (double)to_f32<T>(xr[c]);
        const float m = (float)(block_sum<NW>(s, lds) / (double)C);
        s = 0.0;
#pragma unroll 4
        for (uint32_t c = threadIdx.x; c < (uint32_t)C; c += 64 * NW) {
            const float d = to_f32<T>(xr[c]) - m;
            s += (double)d * (double)d;
        }
        const float r = 1.0f / sqrtf((float)(block_sum<NW>(s, lds) / (double)C) + eps);
#pragma unroll 4
        for (uint32_t c = threadIdx.x; c < (uint32_t)C; c += 64 * NW) {
            const float n = (to_f32<T>(xr[c]) - m) * r;
            yr[c] = from_f32<T>(fmaf(n, weight ? weight[w0 + c] : 1.0f, bias ? bias[w0 + c] : 0.0f));
        }
        if (mean && threadIdx.x == 0) { mean[row] = m; rstd[row] = r; }
    }
}

template <int NW, typename T>
__global__ __launch_bounds__(64 * NW) void gdn_layer_norm_dx_kernel(
    int64_t rows, int G, int C, const T* dy, const T* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ mean, const float* __restrict__ rstd, T* dx) {
    __shared__ double lds[NW];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + (size_t)row * C;
        const T* dr = dy + (size_t)row * C;
        T* out = dx + (size_t)row * C;
        const size_t w0 = (size_t)(row % G) * C;
        const float m = mean[row], r = rstd[row];
        double tg = 0.0, tn = 0.0;
#pragma unroll 4
        for (uint32_t c = threadIdx.x; c < (uint32_t)C; c += 64 * NW) {
            const float n = (to_f32<T>(xr[c]) - m) * r;
            const float g = to_f32<T>(dr[c]) * (weight ? weight[w0 + c] : 1.0f);
            tg += (double)g;
            tn += (double)g * (double)n;
        }
        const float sg = (float)(block_sum<NW>(tg, lds) / (double)C);
        const float sn = (float)(block_sum<NW>(tn, lds) / (double)C);
#pragma unroll 4
        for (uint32_t c = threadIdx.x; c < (uint32_t)C; c += 64 * NW) {
            const float n = (to_f32<T>(xr[c]) - m) * r;
            const float g = to_f32<T>(dr[c]) * (weight ? weight[w0 + c] : 1.0f);
            out[c] = from_f32<T>(r * (g - sg - n * sn));
        }
    }
}

// Sums over a slab of tokens (G consecutive rows each), to part as above.
template <typename T>
__global__ __launch_bounds__(256) void gdn_layer_norm_dw_kernel(
    int64_t tokens, int G, int C, int slabs, const T* __restrict__ dy, const T* __restrict__ x,
    const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part) {
    const int64_t GC = (int64_t)G * C;
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= GC) return;
    const int g = (int)(c / C);
    float dw = 0.0f, db = 0.0f;
    for (int64_t t = blockIdx.y; t < tokens; t += slabs) {
        const float d = to_f32<T>(dy[t * GC + c]);
        dw = fmaf(d, (to_f32<T>(x[t * GC + c]) - mean[t * G + g]) * rstd[t * G + g], dw);
        db += d;
    }
    part[blockIdx.y * GC + c] = dw;
    part[(slabs + blockIdx.y) * GC + c] = db;
}

constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch (a dispatch covers fewer than 2^32 work-items)

hipError_t launch(const void* kernel, dim3 grid, int threads, hipStream_t s, void** args) {
    return hipLaunchKernel(kernel, grid, dim3((unsigned)threads), args, 0, s);
}

// Lanes per row LR, vectors per lane K and threads NT of the kernels that keep rows in registers:
// f.template run<LR, K, NT>() for rows of `vecs` vectors, or f.loop() for longer ones. Up to 128 vectors
// a wave or less holds a row (no LDS; at 128 a workgroup of two waves takes 56 us forward and 309
// backward against 43 and 150); above that the workgroup grows once K reaches 3, since fewer lanes with
// more registers each hide less (512 vectors, 128 lanes with 4 against 256 with 2: 48 and 197 us against
// 45 and 133; 1536, 256 with 6 against 512 with 3: 58 and 125 against 54 and 103). All of 2^26 bf16
// values. The loop over a row that no workgroup holds reads it again for every sum: rows of 16384 take 52 us
// forward and 105 backward in registers, of 24576 100 and 264 in the loop.
template <typename F>
hipError_t by_width(int64_t vecs, F&& f) {
    if (vecs <= 4) return f.template run<4, 1, 256>();
    if (vecs <= 8) return f.template run<8, 1, 256>();
    if (vecs <= 16) return f.template run<16, 1, 256>();
    if (vecs <= 32) return f.template run<32, 1, 256>();
    if (vecs <= 64) return f.template run<64, 1, 256>();
    if (vecs <= 128) return f.template run<64, 2, 256>();
    if (vecs <= 256) return f.template run<256, 1, 256>();
    if (vecs <= 512) return f.template run<256, 2, 256>();
    if (vecs <= 768) return f.template run<256, 3, 256>();
    if (vecs <= 1024) return f.template run<512, 2, 512>();
    if (vecs <= 1536) return f.template run<512, 3, 512>();
    if (vecs <= 2048) return f.template run<1024, 2, 1024>();
    return f.loop();
}

template <typename T>
struct NormRun {
    const NormArgs& a;
    hipStream_t s;

    template <int LR, int K, int NT>
    hipError_t run() {
        int64_t tokens = a.rows / a.G;
        int G = a.G, C = a.C;
        // workgroups: 16 a CU of 256 threads, 8 where rows take many registers or threads (2^26 bf16 values,
        // 16 and 8: rows of 512 44 and 52 us, of 2048 46 and 55; of 6144 45 and 44, of 16384 52 and 49)
        constexpr int WGS = NT <= 256 && K < 3 ? 4096 : 2048;
        const int64_t trips = (tokens + NT / LR - 1) / (NT / LR), want = (WGS * 256 / NT + G - 1) / G;
        int slabs = (int)(trips < want ? trips : want);
        const T* x = (const T*)a.x;
        T* y = (T*)a.y;
        const float *w = a.weight, *b = a.bias;
        float *m = a.mean, *r = a.rstd, eps = a.eps;
        void* args[] = {&tokens, &G, &C, &slabs, &x, &w, &b, &y, &m, &r, &eps};
        const int64_t units = (int64_t)G * slabs;
        return launch((const void*)gdn_layer_norm_rows_kernel<T, LR, K, NT>,
                      dim3((unsigned)(units < kMaxGrid ? units : kMaxGrid)), NT, s, args);
    }
    hipError_t loop() {
        int64_t rows = a.rows;
        int G = a.G, C = a.C;
        const T* x = (const T*)a.x;
        T* y = (T*)a.y;
        const float *w = a.weight, *b = a.bias;
        float *m = a.mean, *r = a.rstd, eps = a.eps;
        void* args[] = {&rows, &G, &C, &x, &w, &b, &y, &m, &r, &eps};
        return launch((const void*)gdn_layer_norm_kernel<16, T>,
                      dim3((unsigned)(rows < kMaxGrid ? rows : kMaxGrid)), 1024, s, args);
    }
};

hipError_t join_slabs(const NormBackwardArgs& a, int slabs, hipStream_t s) {
    int64_t GC = (int64_t)a.G * a.C;
    const float* part = a.ws;
    float *dw = a.dweight, *db = a.dbias;
    void* args[] = {&GC, &slabs, &part, &dw, &db};
    const int64_t blocks = (GC + 63) / 64;
    return launch((const void*)gdn_layer_norm_slabs_kernel, dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid), 2), 1024,
                  s, args);
}

template <typename T>
struct NormBackwardRun {
    const NormBackwardArgs& a;
    hipStream_t s;

    template <int LR, int K, int NT>
    hipError_t run() {
        const bool params = a.dweight || a.dbias;
        int64_t tokens = a.rows / a.G;
        int G = a.G, C = a.C;
        // workgroups: 8 a CU of 256 threads, and 2 or 1 of more (all resident at once; of two rounds the
        // second runs partly empty: 5000 fp32 rows of 4099 63 us, with twice as many 78)
        constexpr int WGS = NT <= 256 ? 2048 : 1024;
        const int64_t trips = (tokens + NT / LR - 1) / (NT / LR), want = (WGS * 256 / NT + G - 1) / G;
        int slabs = (int)(trips < want ? trips : want);
        if (params && slabs > norm_slabs(a.rows, G, C)) slabs = norm_slabs(a.rows, G, C);
        if (params && NT > 256 && slabs > kNormSlabsLong) slabs = (int)kNormSlabsLong;
        const T *dy = (const T*)a.dy, *x = (const T*)a.x;
        T* dx = (T*)a.dx;
        const float *w = a.weight, *m = a.mean, *r = a.rstd;
        float* part = params ? a.ws : nullptr;
        if (slabs > 0) {
            void* args[] = {&tokens, &G, &C, &slabs, &dy, &x, &w, &m, &r, &dx, &part};
            const int64_t units = (int64_t)G * slabs;
            hipError_t e = launch((const void*)gdn_layer_norm_rows_backward_kernel<T, LR, K, NT>,
                                  dim3((unsigned)(units < kMaxGrid ? units : kMaxGrid)), NT, s, args);
            if (e != hipSuccess) return e;
        }
        return params ? join_slabs(a, slabs, s) : hipSuccess;
    }
    hipError_t loop() {
        int64_t rows = a.rows, tokens = a.rows / a.G;
        int G = a.G, C = a.C;
        const T *dy = (const T*)a.dy, *x = (const T*)a.x;
        T* dx = (T*)a.dx;
        const float *w = a.weight, *m = a.mean, *r = a.rstd;
        if (a.dweight || a.dbias) {  // before dx, which may overwrite dy
            int slabs = norm_slabs(rows, G, C);
            float* part = a.ws;
            if (slabs > 0) {
                void* args[] = {&tokens, &G, &C, &slabs, &dy, &x, &m, &r, &part};
                const unsigned cols = (unsigned)(((int64_t)G * C + 255) / 256);
                hipError_t e = launch((const void*)gdn_layer_norm_dw_kernel<T>, dim3(cols, (unsigned)slabs), 256, s, args);
                if (e != hipSuccess) return e;
            }
            hipError_t e = join_slabs(a, slabs, s);
            if (e != hipSuccess) return e;
        }
        if (rows == 0) return hipSuccess;
        void* args[] = {&rows, &G, &C, &dy, &x, &w, &m, &r, &dx};
        return launch((const void*)gdn_layer_norm_dx_kernel<16, T>,
                      dim3((unsigned)(rows < kMaxGrid ? rows : kMaxGrid)), 1024, s, args);
    }
};

template <typename T>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
    constexpr int VE = Vec<T>::VE;
    return by_width(((int64_t)a.C + VE - 1) / VE, NormRun<T>{a, s});
}

template <typename T>
hipError_t norm_backward_t(const NormBackwardArgs& a, hipStream_t s) {
    constexpr int VE = Vec<T>::VE;
    return by_width(((int64_t)a.C + VE - 1) / VE, NormBackwardRun<T>{a, s});
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s) {
    switch (a.dtype) {
        case DType::F32: return norm_t<float>(a, s);
        case DType::BF16: return norm_t<uint16_t>(a, s);
        default: return norm_t<_Float16>(a, s);
    }
}

hipError_t launch_layer_norm_backward(const NormBackwardArgs& a, hipStream_t s) {
    switch (a.dtype) {
        case DType::F32: return norm_backward_t<float>(a, s);
        case DType::BF16: return norm_backward_t<uint16_t>(a, s);
        default: return norm_backward_t<_Float16>(a, s);
    }
}

}  // namespace gdn
