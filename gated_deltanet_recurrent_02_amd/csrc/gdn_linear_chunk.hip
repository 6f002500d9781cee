// The chunked form of linear attention's sweeps (gdn_linear.hip) on the matrix cores of gfx950.
//
// A sweep N <- l N + z_t y_t^T, out_t = N x_t over a chunk of C tokens i = 0 .. C-1 from the state
// N before it regroups into dense products,
//     out_i  = l^(i+1-e) N x_i + sum_{j <= i} l^(i-j) (x_i . y_j) z_j
//     N_next = l^C N + sum_j l^(C-1-j+e) z_j y_j^T
// with e = 0 forward in time (the decay comes before a token) and e = 1 backward (after it). Every
// power of l is a product, never a quotient, so l = 0 is exact and nothing overflows for l <= 1;
// the powers are formed in 64 bits and rounded once. The last chunk of a sequence takes its
// number of tokens n for C; tokens past it enter as zeros.
//
// A workgroup of W waves owns one head's state columns z in [z0, z0 + 16 W NV) (16 NV a wave) for the whole sweep
// and walks over its chunks. Layout (lane = 16 g + n; 16x16x32 bf16 MFMA: operand row or column n,
// k = 8 g + 0..7, result column n, rows 4 g + 0..3):
//   * the state is held as N^T (rows y's dimension, columns z) in fp32 result tiles, which the
//     update accumulates into; the same registers, split into bf16 parts, are the operand of N x;
//   * x, y, z tiles of the chunk are staged in LDS by rows of tokens; products that contract over
//     tokens read y and z transposed (ds_read_b64_tr_b16);
//   * the weighted scores are formed once per workgroup, a share of the 16x16 tiles on or below
//     the diagonal per wave, and exchanged through LDS.
// Precision: operands of the matrix cores are bf16, so fp16 and fp32 inputs enter as two and three
// bf16 parts whose sum is exact. State and scores enter the outputs as two parts for 16-bit
// outputs (2^-16 of a term, against their own rounding of 2^-9 and 2^-12) and three for fp32 ones;
// the weighted z enters the state as three parts (exact). Products of parts below the last kept
// one are dropped.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_linear_common.h"
#include "gdn_linear_launch.h"

namespace gdn {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Four 16-bit values of one column: within each group of 16 lanes, lane i passes the address of row
// i / 4, columns 4 (i % 4) .. + 3 of a 4 x 16 block and gets column i's rows 0..3 (checked on the device).
__device__ __forceinline__ u32x2 read_tr(const uint16_t* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)p));
}

// The high halves of two words packed into one, x's in the low half.
__device__ __forceinline__ uint32_t hi_halves(uint32_t x, uint32_t y) {
    return __builtin_amdgcn_perm(y, x, 0x07060302u);
}

// Two floats as NP packed pairs of bf16 parts. The leading parts are truncated, so each remainder
// is exact; three parts hold all 24 bits, and the last of two rounds to nearest.
template <int NP>
__device__ __forceinline__ void split(float a, float b, uint32_t (&w)[NP]) {
    constexpr uint32_t HI = 0xffff0000u;
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    w[0] = hi_halves(ua, ub);
    if constexpr (NP >= 2) {
        const float ra = a - __uint_as_float(ua & HI), rb = b - __uint_as_float(ub & HI);
        if constexpr (NP == 2) {
            w[1] = Elem<uint16_t>::pack(ra, rb);
        } else {
            const uint32_t va = __float_as_uint(ra), vb = __float_as_uint(rb);
            w[1] = hi_halves(va, vb);
            w[2] = hi_halves(__float_as_uint(ra - __uint_as_float(va & HI)),
                             __float_as_uint(rb - __uint_as_float(vb & HI)));
        }
    }
}

// The parts of one activation type, and how many parts the fp32 factors of its outputs take.
template <typename AT> struct Parts;
template <> struct Parts<uint16_t> { static constexpr int A = 1, O = 2, LIM = 2, C = 64; };
template <> struct Parts<_Float16> { static constexpr int A = 2, O = 2, LIM = 2, C = 32; };
template <> struct Parts<float> { static constexpr int A = 3, O = 3, LIM = 3, C = 32; };

template <int D_, typename AT_, int W_, int NV_>
struct ChunkGeo {
    static constexpr int D = D_, W = W_, NV = NV_;
    using AT = AT_;
    static constexpr int A = Parts<AT>::A, O = Parts<AT>::O, LIM = Parts<AT>::LIM, C = Parts<AT>::C;
    static constexpr int DP = D < 32 ? 32 : D;       // contraction over D in steps of 32 (zeros past D)
    static constexpr int ZW = 16 * W * NV;           // state columns of a workgroup
    static constexpr int ZS = D / ZW;                // workgroups per head and segment
    static constexpr int NT = 64 * W;
    static constexpr int CT = C / 16, CK = C / 32, DT = DP / 16, DK = DP / 32;
    static constexpr int TILES = CT * (CT + 1) / 2;  // score tiles on or below the diagonal
    // row strides in LDS, in 16-bit elements: rows 4 or 8 banks apart spread reads by rows and
    // transposed reads over the banks
    static constexpr int XS = DP + 8, YS = DP + 16, ZSTR = ZW + 16, PS = C + 8;
    static constexpr int VE = 16 / (int)sizeof(AT);  // elements per 16-byte load
    static constexpr int XV = C * (D / VE) / NT, ZV = C * (ZW / VE) / NT;  // loads per thread
    static_assert(D % ZW == 0 && C * (D / VE) % NT == 0 && C * (ZW / VE) % NT == 0, "geometry");
};

template <class G, bool STATE_ONLY>
struct ChunkLds {
    alignas(16) uint16_t x[STATE_ONLY ? 1 : G::A][STATE_ONLY ? 1 : G::C][G::XS];
    alignas(16) uint16_t y[G::A][G::C][G::YS];
    alignas(16) uint16_t z[G::A][G::C][G::ZSTR];
    alignas(16) uint16_t p[STATE_ONLY ? 1 : G::O][STATE_ONLY ? 1 : G::C][G::PS];
    float pw[G::C + 1];  // l^0 .. l^C
};

// l^n in 64 bits.
__device__ __forceinline__ double power(float l, int n) {
    double p = 1.0, b = (double)l;
    for (; n > 0; n >>= 1) {
        if (n & 1) p *= b;
        b *= b;
    }
    return p;
}

// A chunk's rows of one tensor on their way from memory to LDS: WIDTH columns from column c0.
template <class G, int WIDTH, int N>
struct Stage {
    using AT = typename G::AT;
    static constexpr int VPR = WIDTH / G::VE;
    Run<AT, G::VE> r[N];

    // rows of tokens [i0, i0 + n) of the sweep; row i is token i, or len - 1 - i backward
    __device__ __forceinline__ void load(const AT* p, size_t stride, int i0, int n, int len, bool reverse, int c0) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int e = threadIdx.x + u * G::NT, row = e / VPR, c = (e % VPR) * G::VE;
            if (row < n) {
                const int t = reverse ? len - 1 - (i0 + row) : i0 + row;
                r[u].load(p + (size_t)t * stride + c0 + c);
            } else {
                r[u].zero();
            }
        }
    }
    template <int STRIDE>
    __device__ __forceinline__ void store(uint16_t (*lds)[G::C][STRIDE]) const {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int e = threadIdx.x + u * G::NT, row = e / VPR, c = (e % VPR) * G::VE;
            if constexpr (G::A == 1) {
                *(u32x4*)&lds[0][row][c] = u32x4{r[u].w[0], r[u].w[1], r[u].w[2], r[u].w[3]};
            } else {
                uint32_t w[G::VE / 2][G::A];
#pragma unroll
                for (int j = 0; j < G::VE / 2; ++j) split<G::A>(r[u].get(2 * j), r[u].get(2 * j + 1), w[j]);
#pragma unroll
                for (int a = 0; a < G::A; ++a) {
                    if constexpr (G::VE == 8) *(u32x4*)&lds[a][row][c] = u32x4{w[0][a], w[1][a], w[2][a], w[3][a]};
                    else *(u32x2*)&lds[a][row][c] = u32x2{w[0][a], w[1][a]};
                }
            }
        }
    }
};

__device__ __forceinline__ float state_value(const void* p, DType t, size_t i) {
    return t == DType::F32 ? ((const float*)p)[i]
                           : (t == DType::BF16 ? to_f32<uint16_t>(((const uint16_t*)p)[i])
                                               : (float)((const _Float16*)p)[i]);
}

struct ChunkArgs {
    Sweep s[3];
    int64_t BH;     // B * H
    int seg_tokens; // tokens of a segment (a multiple of C)
    int nseg;
    float* ws;      // [sweep][B * H][nseg][D][D] fp32, if nseg > 1: the segments' states
};

// Loads four consecutive values (y's dimension d .. d + 3 of row z) of a state.
template <int D>
__device__ __forceinline__ f32x4 load_state4(const void* p, DType t, bool transposed, size_t base, int z, int d) {
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        v[r] = state_value(p, t, base + (transposed ? (size_t)(d + r) * D + z : (size_t)z * D + d + r));
    return v;
}

template <int D>
__device__ __forceinline__ void store_state4(void* p, DType t, size_t base, int z, int d, f32x4 v) {
    const size_t i = base + (size_t)z * D + d;
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (t == DType::F32) {
        *(f32x4*)((float*)p + i) = v;
    } else if (t == DType::BF16) {
        Run<uint16_t, 4> r;
        r.set(f);
        r.store((uint16_t*)p + i);
    } else {
        Run<_Float16, 4> r;
        r.set(f);
        r.store((_Float16*)p + i);
    }
}

// STATE_ONLY: each segment's own state from zero, for the scan that gives every segment its start.
template <class G, bool STATE_ONLY>
__global__ __launch_bounds__(G::NT) void gdn_linear_chunk_kernel(ChunkArgs a) {
    using AT = typename G::AT;
    constexpr int D = G::D, C = G::C, A = G::A, O = G::O, LIM = G::LIM, NV = G::NV;
    __shared__ ChunkLds<G, STATE_ONLY> L;
    const Sweep& s = a.s[blockIdx.y];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, n16 = lane & 15;
    uint32_t id = blockIdx.x;
    const int zs = (int)(id % G::ZS);
    id /= G::ZS;
    const int seg = (int)(id % (uint32_t)a.nseg);
    const int64_t bh = id / (uint32_t)a.nseg;
    const int64_t b = bh / s.H;
    const int h = (int)(bh % s.H);
    const int T = s.T, len = tokens_of(s.lengths, b, T);
    const int begin = min(seg * a.seg_tokens, len);
    const int end = (seg == a.nseg - 1) ? len : min((seg + 1) * a.seg_tokens, len);
    const bool reverse = s.reverse;
    const int e = reverse ? 1 : 0;
    const int z0 = zs * G::ZW, zw = z0 + wave * 16 * NV;  // the workgroup's and the wave's columns
    const float lam = s.decay[h];
    float* wst = a.ws + ((size_t)blockIdx.y * a.BH + bh) * a.nseg * D * D + (size_t)seg * D * D;

    if constexpr (!STATE_ONLY) {
        // outputs past the sequence's end: this segment's share
        const int r0 = max(seg * a.seg_tokens, len), r1 = seg == a.nseg - 1 ? T : min((seg + 1) * a.seg_tokens, T);
        if (r0 < r1) {
            const size_t es = s.out_f32 ? 4 : sizeof(AT);
            char* o = (char*)s.out + (((size_t)b * T * s.H + h) * D + z0) * es;
            const size_t row = (size_t)s.H * D * es;
            const int words = (int)(G::ZW * es / 8);
            for (int64_t i = tid; i < (int64_t)(r1 - r0) * words; i += G::NT)
                *(u32x2*)(o + (size_t)(r0 + i / words) * row + (i % words) * 8) = u32x2{0u, 0u};
        }
        // a segment without tokens; the last one still hands on the state
        if (begin == end && !(a.nseg == 1 && s.last != nullptr && s.last != s.first)) return;
    }

    for (int i = tid; i <= C; i += G::NT) L.pw[i] = (float)power(lam, i);
    if constexpr (!STATE_ONLY) {
        // the score tiles above the diagonal that products over 32 tokens touch stay zero
        for (int i = tid; i < O * C * G::PS / 2; i += G::NT) ((uint32_t*)L.p)[i] = 0u;
    }
    if constexpr (G::DP > D) {
        for (int i = tid; i < A * C * G::YS / 2; i += G::NT) ((uint32_t*)L.y)[i] = 0u;
        if constexpr (!STATE_ONLY)
            for (int i = tid; i < A * C * G::XS / 2; i += G::NT) ((uint32_t*)L.x)[i] = 0u;
        __syncthreads();
    }

    // N^T: tile (dt, v), element r is N[z = zw + 16 v + n16][d = 16 dt + 4 g + r]
    f32x4 N[G::DT][NV];
#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            N[dt][v] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (!STATE_ONLY) {
                if (16 * dt < D) {
                    const int z = zw + 16 * v + n16, d = 16 * dt + 4 * g;
                    if (a.nseg > 1) N[dt][v] = *(const f32x4*)(wst + (size_t)z * D + d);
                    else if (s.first) N[dt][v] = load_state4<D>(s.first, s.state_dtype, s.transposed, (size_t)bh * D * D, z, d);
                }
            }
        }

    const int Hx = s.H / s.gx, Hy = s.H / s.gy, Hz = s.H / s.gz;
    const size_t xst = (size_t)Hx * D, yst = (size_t)Hy * D, zst = (size_t)Hz * D;
    const AT* xp = (const AT*)s.x + ((size_t)b * T * Hx + h / s.gx) * D;
    const AT* yp = (const AT*)s.y + ((size_t)b * T * Hy + h / s.gy) * D;
    const AT* zp = (const AT*)s.z + ((size_t)b * T * Hz + h / s.gz) * D;
    Stage<G, D, STATE_ONLY ? 1 : G::XV> sx;
    Stage<G, D, G::XV> sy;
    Stage<G, G::ZW, G::ZV> sz;
    const auto fetch = [&](int i0) {
        const int n = min(C, end - i0);
        if constexpr (!STATE_ONLY) sx.load(xp, xst, i0, n, len, reverse, 0);
        sy.load(yp, yst, i0, n, len, reverse, 0);
        sz.load(zp, zst, i0, n, len, reverse, z0);
    };
    if (begin < end) fetch(begin);

    for (int i0 = begin; i0 < end; i0 += C) {
        const int n = min(C, end - i0);
        if constexpr (!STATE_ONLY) sx.template store<G::XS>(L.x);
        sy.template store<G::YS>(L.y);
        sz.template store<G::ZSTR>(L.z);
        __syncthreads();
        if (i0 + C < end) fetch(i0 + C);

        f32x4 acc[STATE_ONLY ? 1 : NV][STATE_ONLY ? 1 : G::CT];
        if constexpr (!STATE_ONLY) {
            // scores: tile (ti, si), lane (g, n16) holds s = 16 si + 4 g + r of t = 16 ti + n16
            const float ps = s.oscale * s.zscale;
            for (int tile = wave; tile < G::TILES; tile += G::W) {
                int ti = 0, si = tile;
                while (si > ti) { si -= ti + 1; ++ti; }
                f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < G::DK; ++kk) {
                    u32x4 yf[A], xf[A];
#pragma unroll
                    for (int p = 0; p < A; ++p) {
                        yf[p] = *(const u32x4*)&L.y[p][16 * si + n16][32 * kk + 8 * g];
                        xf[p] = *(const u32x4*)&L.x[p][16 * ti + n16][32 * kk + 8 * g];
                    }
#pragma unroll
                    for (int p = A - 1; p >= 0; --p)
#pragma unroll
                        for (int u = A - 1; u >= 0; --u)
                            if (p + u < LIM) c = mfma(yf[p], xf[u], c);
                }
                const int t = 16 * ti + n16, s0 = 16 * si + 4 * g;
                float w[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r] = t >= s0 + r ? ps * L.pw[max(t - s0 - r, 0)] * c[r] : 0.0f;
                uint32_t lo[O], hi[O];
                split<O>(w[0], w[1], lo);
                split<O>(w[2], w[3], hi);
#pragma unroll
                for (int p = 0; p < O; ++p) *(u32x2*)&L.p[p][t][s0] = u32x2{lo[p], hi[p]};
            }

            // out^T = N x: rows z = zw + 16 v + 4 g + r, column t = 16 ct + n16
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int ct = 0; ct < G::CT; ++ct) acc[v][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < G::DK; ++kk) {
                u32x4 nf[NV][O];
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    uint32_t w[4][O];
                    split<O>(N[2 * kk][v].x, N[2 * kk][v].y, w[0]);
                    split<O>(N[2 * kk][v].z, N[2 * kk][v].w, w[1]);
                    split<O>(N[2 * kk + 1][v].x, N[2 * kk + 1][v].y, w[2]);
                    split<O>(N[2 * kk + 1][v].z, N[2 * kk + 1][v].w, w[3]);
#pragma unroll
                    for (int p = 0; p < O; ++p) nf[v][p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
                }
#pragma unroll
                for (int ct = 0; ct < G::CT; ++ct) {
                    u32x4 xf[A];
#pragma unroll
                    for (int u = 0; u < A; ++u) {
                        const u32x2 x0 = *(const u32x2*)&L.x[u][16 * ct + n16][32 * kk + 4 * g];
                        const u32x2 x1 = *(const u32x2*)&L.x[u][16 * ct + n16][32 * kk + 16 + 4 * g];
                        xf[u] = u32x4{x0.x, x0.y, x1.x, x1.y};
                    }
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int p = O - 1; p >= 0; --p)
#pragma unroll
                            for (int u = A - 1; u >= 0; --u)
                                if (p + u < LIM) acc[v][ct] = mfma(nf[v][p], xf[u], acc[v][ct]);
                }
            }
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) {
                const float f = s.oscale * L.pw[16 * ct + n16 + 1 - e];
#pragma unroll
                for (int v = 0; v < NV; ++v) acc[v][ct] *= f;
            }
            __syncthreads();
        }

        // z transposed, its products with the scores, and the state's update, 32 tokens at a time
        const float carry = L.pw[n];
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
            for (int v = 0; v < NV; ++v) N[dt][v] *= carry;
        const int tr = n16 >> 2, tc = (n16 & 3) * 4;
#pragma unroll
        for (int kk = 0; kk < G::CK; ++kk) {
            u32x4 zf[NV][A];
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int u = 0; u < A; ++u) {
                    const uint16_t* p = &L.z[u][32 * kk + 8 * g + tr][wave * 16 * NV + 16 * v + tc];
                    const u32x2 a0 = read_tr(p), a1 = read_tr(p + 4 * G::ZSTR);
                    zf[v][u] = u32x4{a0.x, a0.y, a1.x, a1.y};
                }
            if constexpr (!STATE_ONLY) {
#pragma unroll
                for (int ct = 2 * kk; ct < G::CT; ++ct) {
                    u32x4 pf[O];
#pragma unroll
                    for (int p = 0; p < O; ++p) pf[p] = *(const u32x4*)&L.p[p][16 * ct + n16][32 * kk + 8 * g];
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int p = O - 1; p >= 0; --p)
#pragma unroll
                            for (int u = A - 1; u >= 0; --u)
                                if (p + u < LIM) acc[v][ct] = mfma(zf[v][u], pf[p], acc[v][ct]);
                }
            }
            // weighted z in three parts
            u32x4 wf[NV][3];
            float wt[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) wt[j] = s.zscale * L.pw[max(n - 1 - (32 * kk + 8 * g + j), 0) + e];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                uint32_t w[4][3];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float z[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int u = A - 1; u >= 0; --u) {
                        z[0] += __uint_as_float(zf[v][u][j] << 16);
                        z[1] += __uint_as_float(zf[v][u][j] & 0xffff0000u);
                    }
                    split<3>(z[0] * wt[2 * j], z[1] * wt[2 * j + 1], w[j]);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) wf[v][p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
            }
#pragma unroll
            for (int dt = 0; dt < G::DT; ++dt) {
                if (16 * dt >= D) continue;
                u32x4 yf[A];
#pragma unroll
                for (int u = 0; u < A; ++u) {
                    const uint16_t* p = &L.y[u][32 * kk + 8 * g + tr][16 * dt + tc];
                    const u32x2 a0 = read_tr(p), a1 = read_tr(p + 4 * G::YS);
                    yf[u] = u32x4{a0.x, a0.y, a1.x, a1.y};
                }
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
#pragma unroll
                        for (int u = A - 1; u >= 0; --u)
                            if (p + u < 3) N[dt][v] = mfma(yf[u], wf[v][p], N[dt][v]);
            }
        }

        if constexpr (!STATE_ONLY) {
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) {
                const int i = 16 * ct + n16;
                if (i < n) {
                    const int t = reverse ? len - 1 - (i0 + i) : i0 + i;
                    const size_t o = (((size_t)b * T + t) * s.H + h) * D + zw + 4 * g;
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const float f[4] = {acc[v][ct].x, acc[v][ct].y, acc[v][ct].z, acc[v][ct].w};
                        if (s.out_f32) {
                            *(f32x4*)((float*)s.out + o + 16 * v) = acc[v][ct];
                        } else {
                            Run<AT, 4> r;
                            r.set(f);
                            r.store((AT*)s.out + o + 16 * v);
                        }
                    }
                }
            }
        }
        __syncthreads();
    }

#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (16 * dt < D) {
                const int z = zw + 16 * v + n16, d = 16 * dt + 4 * g;
                if constexpr (STATE_ONLY) *(f32x4*)(wst + (size_t)z * D + d) = N[dt][v];
                else if (a.nseg == 1 && s.last) store_state4<D>(s.last, s.state_dtype, (size_t)bh * D * D, z, d, N[dt][v]);
            }
}

// The segments' starts from their own states, in place: start[0] is the sweep's first state,
// start[i + 1] = l^(tokens of i) start[i] + own[i]; the one after the last segment is the last state.
template <int D>
__global__ __launch_bounds__(256) void gdn_linear_scan_kernel(ChunkArgs a) {
    const Sweep& s = a.s[blockIdx.y];
    constexpr int PER = D * D / 4;  // vectors of a state
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t bh = id / PER;
    if (bh >= a.BH) return;
    const int z = (int)(id % PER) / (D / 4), d = (int)(id % (D / 4)) * 4;
    const int len = tokens_of(s.lengths, bh / s.H, s.T);
    const float lam = s.decay[bh % s.H];
    f32x4 N = {0.f, 0.f, 0.f, 0.f};
    if (s.first) N = load_state4<D>(s.first, s.state_dtype, s.transposed, (size_t)bh * D * D, z, d);
    float* w = a.ws + ((size_t)blockIdx.y * a.BH + bh) * a.nseg * D * D + (size_t)z * D + d;
    const float whole = (float)power(lam, a.seg_tokens);
    for (int seg = 0; seg < a.nseg; ++seg, w += D * D) {
        const int begin = min(seg * a.seg_tokens, len);
        const int end = (seg == a.nseg - 1) ? len : min((seg + 1) * a.seg_tokens, len);
        const f32x4 own = *(const f32x4*)w;
        *(f32x4*)w = N;
        N = N * (end - begin == a.seg_tokens ? whole : (float)power(lam, end - begin)) + own;
    }
    if (s.last && !(s.last == s.first && len == 0)) store_state4<D>(s.last, s.state_dtype, (size_t)bh * D * D, z, d, N);
}

template <typename F>
hipError_t launch(F kernel, dim3 grid, int threads, hipStream_t st, ChunkArgs a) {
    void* args[] = {&a};
    return hipLaunchKernel((const void*)kernel, grid, dim3((unsigned)threads), args, 0, st);
}

template <int D, typename AT>
hipError_t chunk_t(const Sweep* sweeps, int n, int64_t B, float* ws, hipStream_t st) {
    constexpr int W = D >= 64 ? 4 : D / 16, NV = D / 16 / W;
    using G = ChunkGeo<D, AT, W, NV>;
    ChunkArgs a;
    for (int i = 0; i < n; ++i) a.s[i] = sweeps[i];
    const int T = sweeps[0].T, H = sweeps[0].H;
    a.BH = B * H;
    a.nseg = linear_segments(B, T, H, D, n);
    a.seg_tokens = ((T + a.nseg - 1) / a.nseg + 63) / 64 * 64;
    a.ws = ws;
    const dim3 grid((unsigned)(a.BH * a.nseg * G::ZS), (unsigned)n);
    if (a.nseg > 1) {
        hipError_t e = launch(gdn_linear_chunk_kernel<G, true>, grid, G::NT, st, a);
        if (e != hipSuccess) return e;
        e = launch(gdn_linear_scan_kernel<D>, dim3((unsigned)((a.BH * D * D / 4 + 255) / 256), (unsigned)n), 256, st, a);
        if (e != hipSuccess) return e;
    }
    return launch(gdn_linear_chunk_kernel<G, false>, grid, G::NT, st, a);
}

template <int D>
hipError_t chunk_d(const Sweep* s, int n, int64_t B, DType act, float* ws, hipStream_t st) {
    switch (act) {
        case DType::F32: return chunk_t<D, float>(s, n, B, ws, st);
        case DType::BF16: return chunk_t<D, uint16_t>(s, n, B, ws, st);
        default: return chunk_t<D, _Float16>(s, n, B, ws, st);
    }
}

}  // namespace

hipError_t launch_linear_chunk(const Sweep* s, int n, int64_t B, int D, DType act, float* ws, hipStream_t st) {
    switch (D) {
        case 16: return chunk_d<16>(s, n, B, act, ws, st);
        case 32: return chunk_d<32>(s, n, B, act, ws, st);
        case 64: return chunk_d<64>(s, n, B, act, ws, st);
        default: return chunk_d<128>(s, n, B, act, ws, st);
    }
}

}  // namespace gdn
