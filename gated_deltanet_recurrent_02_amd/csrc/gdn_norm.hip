// Layer norm of a layer's output on gfx950 (CDNA4), forward and backward. Per row r of x [rows][C]
// with the affine of group r mod G,
//     n = (x - mean) rstd,  mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),  y = n w + b
//     g = dy w,  dx = rstd (g - mean_C(g) - n mean_C(g n)),  dw = sum_rows dy n,  db = sum_rows dy.
// All sums are fp32; the variance is summed from centred values.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_linear_common.h"
#include "gdn_linear_launch.h"

namespace gdn {
namespace {

// Sum over the workgroup's NW waves; every thread gets the same value.
template <int NW>
__device__ __forceinline__ float block_sum(float x, float* lds) {
    x = lane_sum<64>(x);
    if constexpr (NW == 1) return x;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = lds[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) s += lds[i];
    return s;
}

// One workgroup per row at a time, rows in strides of the grid.
template <int NW, typename T>
__global__ __launch_bounds__(64 * NW) void gdn_layer_norm_kernel(
    int64_t rows, int G, int C, const T* x, const float* __restrict__ weight, const float* __restrict__ bias, T* y,
    float* __restrict__ mean, float* __restrict__ rstd, float eps) {
    __shared__ float lds[NW];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + (size_t)row * C;
    T* yr = y + (size_t)row * C;
    const size_t w0 = (size_t)(row % G) * C;
    float s = 0.0f;
    for (int c = threadIdx.x; c < C; c += 64 * NW) s += to_f32<T>(xr[c]);
    const float m = block_sum<NW>(s, lds) / (float)C;
    s = 0.0f;
    for (int c = threadIdx.x; c < C; c += 64 * NW) {
        const float d = to_f32<T>(xr[c]) - m;
        s = fmaf(d, d, s);
    }
    const float r = 1.0f / sqrtf(block_sum<NW>(s, lds) / (float)C + eps);
    for (int c = threadIdx.x; c < C; c += 64 * NW) {
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
    __shared__ float lds[NW];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + (size_t)row * C;
    const T* dr = dy + (size_t)row * C;
    T* out = dx + (size_t)row * C;
    const size_t w0 = (size_t)(row % G) * C;
    const float m = mean[row], r = rstd[row];
    float sg = 0.0f, sn = 0.0f;
    for (int c = threadIdx.x; c < C; c += 64 * NW) {
        const float n = (to_f32<T>(xr[c]) - m) * r;
        const float g = to_f32<T>(dr[c]) * (weight ? weight[w0 + c] : 1.0f);
        sg += g;
        sn = fmaf(g, n, sn);
    }
    sg = block_sum<NW>(sg, lds) / (float)C;
    sn = block_sum<NW>(sn, lds) / (float)C;
    for (int c = threadIdx.x; c < C; c += 64 * NW) {
        const float n = (to_f32<T>(xr[c]) - m) * r;
        const float g = to_f32<T>(dr[c]) * (weight ? weight[w0 + c] : 1.0f);
        out[c] = from_f32<T>(r * (g - sg - n * sn));
    }
    }
}

// Partial sums over a slab of tokens (G consecutive rows each): part[0][slab][G * C] of dy n and
// part[1][slab][G * C] of dy.
constexpr int kSlabs = kNormSlabs;

template <typename T>
__global__ __launch_bounds__(256) void gdn_layer_norm_dw_kernel(
    int64_t tokens, int G, int C, const T* __restrict__ dy, const T* __restrict__ x,
    const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part) {
    const int64_t GC = (int64_t)G * C;
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= GC) return;
    const int g = (int)(c / C);
    float dw = 0.0f, db = 0.0f;
    for (int64_t t = blockIdx.y; t < tokens; t += kSlabs) {
        const float d = to_f32<T>(dy[t * GC + c]);
        dw = fmaf(d, (to_f32<T>(x[t * GC + c]) - mean[t * G + g]) * rstd[t * G + g], dw);
        db += d;
    }
    part[blockIdx.y * GC + c] = dw;
    part[(kSlabs + blockIdx.y) * GC + c] = db;
}

__global__ __launch_bounds__(256) void gdn_layer_norm_dw_sum_kernel(int64_t GC, int slabs,
                                                                    const float* __restrict__ part,
                                                                    float* __restrict__ dw,
                                                                    float* __restrict__ db) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= GC) return;
    float sw = 0.0f, sb = 0.0f;
    for (int i = 0; i < slabs; ++i) {
        sw += part[i * GC + c];
        sb += part[(kSlabs + i) * GC + c];
    }
    if (dw) dw[c] = sw;
    if (db) db[c] = sb;
}

constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch (a dispatch covers fewer than 2^32 work-items)

hipError_t launch(const void* kernel, dim3 grid, int threads, hipStream_t s, void** args) {
    return hipLaunchKernel(kernel, grid, dim3((unsigned)threads), args, 0, s);
}

template <typename T>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
    int G = a.G, C = a.C;
    const T* x = (const T*)a.x;
    T* y = (T*)a.y;
    const float *w = a.weight, *b = a.bias;
    float *m = a.mean, *r = a.rstd, eps = a.eps;
    int64_t rows = a.rows;
    void* args[] = {&rows, &G, &C, &x, &w, &b, &y, &m, &r, &eps};
    const dim3 grid((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid));
    return C <= 512 ? launch((const void*)gdn_layer_norm_kernel<1, T>, grid, 64, s, args)
                    : launch((const void*)gdn_layer_norm_kernel<4, T>, grid, 256, s, args);
}

template <typename T>
hipError_t norm_backward_t(const NormBackwardArgs& a, hipStream_t s) {
    int G = a.G, C = a.C;
    const T *dy = (const T*)a.dy, *x = (const T*)a.x;
    T* dx = (T*)a.dx;
    const float *w = a.weight, *m = a.mean, *r = a.rstd;
    hipError_t e;
    float* part = a.ws;
    int64_t tokens = a.rows / a.G, GC = (int64_t)a.G * a.C;
    const unsigned cols = (unsigned)((GC + 255) / 256);
    int slabs = (int)(tokens < kSlabs ? tokens : kSlabs);
    if ((a.dweight || a.dbias) && slabs > 0) {  // before dx, which may overwrite dy
        void* args[] = {&tokens, &G, &C, &dy, &x, &m, &r, &part};
        e = launch((const void*)gdn_layer_norm_dw_kernel<T>, dim3(cols, (unsigned)slabs), 256, s, args);
        if (e != hipSuccess) return e;
    }
    if (a.dweight || a.dbias) {
        float *dw = a.dweight, *db = a.dbias;
        void* args[] = {&GC, &slabs, &part, &dw, &db};
        e = launch((const void*)gdn_layer_norm_dw_sum_kernel, dim3(cols), 256, s, args);
        if (e != hipSuccess) return e;
    }
    if (a.rows == 0) return hipSuccess;
    int64_t rows = a.rows;
    void* args[] = {&rows, &G, &C, &dy, &x, &w, &m, &r, &dx};
    const dim3 grid((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid));
    return C <= 512 ? launch((const void*)gdn_layer_norm_dx_kernel<1, T>, grid, 64, s, args)
                    : launch((const void*)gdn_layer_norm_dx_kernel<4, T>, grid, 256, s, args);
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
