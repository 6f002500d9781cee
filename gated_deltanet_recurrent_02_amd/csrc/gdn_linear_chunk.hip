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
// A workgroup of W waves owns one head's state, 16 NV columns z a wave, and walks over its chunks. Layout (lane = 16 g + n; 16x16x32 bf16 MFMA: operand row or column n,
// k = 8 g + 0..7, result column n, rows 4 g + 0..3):
//   * the state is held as N^T (rows y's dimension, columns z) in fp32 result tiles, which the
//     update accumulates into; the same registers, split into bf16 parts, are the operand of N x;
//   * x, y, z tiles of the chunk are staged in LDS by rows of tokens; products that contract over
//     tokens read y and z transposed (ds_read_b64_tr_b16);
//   * the weighted scores are formed once per workgroup, a share of the 16x16 tiles on or below
//     the diagonal per wave, and exchanged through LDS.
// Precision: operands of the matrix cores are bf16, so fp16 and fp32 inputs enter as two and three
// bf16 parts whose sum is exact, and the fp32 factors that a chunk forms (state, scores, weighted z) as
// three whatever the outputs' type: sums of large terms that cancel keep fp32's precision, as in the
// recurrent form. Products of parts below the last kept one are dropped. (Two parts for 16-bit
// outputs took 292 and 631 us in the cases below.)
//
// What bounds it. B = 4, T = 4096, H = 48, D = 128, bf16: prefill 316 us (830 MB, 2.6 TB/s; the parts'
// matrix instructions alone take 170 us at the rate of a large product); the gradients 806 us (three
// sweeps, 2.4 GB, 3.0 TB/s). A chunk takes 11,400 cycles of a workgroup alone on its CU: the matrix cores are
// busy for 3,800 of them and vector instructions, most of them taking factors apart, issue for 5,300; the steps
// wait for each other's operands (state in parts, scores through LDS) more than for memory. A second
// workgroup on a CU fills part of that (15,100 cycles a chunk for both), a third does not fit: the state, its parts and
// the operands a step ahead take all 256 registers (so the loads of the next x wait for the first steps of N x, and
// parts are made for one column tile at a time; else it spills). Tried with two parts and slower: 8 waves with 16
// columns each, two workgroups a head, all loads of the next chunk at the start or one in every step, matrix
// and vector instructions interleaved by hand (spills).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_linear_common.h"
#include "gdn_linear_launch.h"

// A value the compiler may not look through: what is computed from it inside the loop over chunks is
// not kept in registers across chunks, where hundreds of such values would crowd out the state.
#define OPAQUE(x) asm volatile("" : "+v"(x))
#define STEP __builtin_amdgcn_sched_barrier(0)

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
__device__ __forceinline__ u32x2 read_tr(const uint8_t* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)p));
}

// Two floats as NP packed pairs of bf16 parts, each rounded to nearest: every remainder is exact, so two parts
// hold an fp16 value and three an fp32 one whole. Cutting parts off instead costs as many instructions and
// doubles each remainder, with the value's sign: the dropped products of parts then take 2^-21 of a term,
// here 2^-26. Values that round to 2^128 in bf16 become infinities.
template <int NP>
__device__ __forceinline__ void split(float a, float b, uint32_t (&w)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        w[p] = Elem<uint16_t>::pack(a, b);
        a -= __uint_as_float(w[p] << 16);
        b -= __uint_as_float(w[p] & 0xffff0000u);
    }
}

// The parts of an fp32 factor; products of parts p and u are kept for p + u < kParts (of two fp16 values all).
constexpr int kParts = 3;

// The parts A of one activation type and the tokens C of a chunk: 64 in one part; 32 in two or three, whose x,
// y and z rows would fill a CU's LDS with one workgroup at 64 (D = 128, three parts: 147 KB).
template <typename AT> struct Parts;
template <> struct Parts<uint16_t> { static constexpr int A = 1, C = 64; };
template <> struct Parts<_Float16> { static constexpr int A = 2, C = 32; };
template <> struct Parts<float> { static constexpr int A = 3, C = 32; };

template <int D_, typename AT_, int W_, int NV_>
struct ChunkGeo {
    static constexpr int D = D_, W = W_, NV = NV_;
    using AT = AT_;
    static constexpr int A = Parts<AT>::A, O = kParts, C = Parts<AT>::C;
    static constexpr int DP = D < 32 ? 32 : D;       // contraction over D in steps of 32 (zeros past D)
    static_assert(16 * W * NV == D, "a workgroup owns a head's state");
    static constexpr int NT = 64 * W;
    static constexpr int CT = C / 16, CK = C / 32, DT = DP / 16, DK = DP / 32;
    // score tiles on or below the diagonal, then those above it that products over 32 tokens touch (zeros)
    static constexpr int LOWER = CT * (CT + 1) / 2, TILES = LOWER + CT / 2, TPW = (TILES + W - 1) / W;
    // bytes of a row in LDS: x and y, z, scores
    static constexpr int XB = 2 * DP, ZB = 2 * D, PB = 2 * C;
    static constexpr int VE = 16 / (int)sizeof(AT);  // elements per 16-byte load
    static constexpr int XV = C * (D / VE) / NT;  // loads per thread
    static_assert(C * (D / VE) % NT == 0, "geometry");
    // Waves a SIMD that the registers are held to: two (512 places of workgroups of four waves), but one for a
    // head of one wave and 64 tokens, of which a CU's LDS holds four.
    static constexpr int WAVES = W == 1 && C == 64 ? 1 : 2;
};

// Rows in LDS are not padded; the 16- or 32-byte unit of a row is exchanged with the row's number
// instead, so that reads of one unit of 16 (or, transposed, 8) consecutive rows use every bank.
template <int ROW_BYTES>
__device__ __forceinline__ int swizzle16(int row) {
    static_assert(ROW_BYTES >= 32 && ROW_BYTES <= 256, "row");
    return ((row / (256 / ROW_BYTES)) & (ROW_BYTES / 16 - 1)) << 4;
}
template <int ROW_BYTES>
__device__ __forceinline__ int swizzle32(int row) {
    static_assert(ROW_BYTES >= 32 && ROW_BYTES <= 256, "row");
    return ((row / (256 / ROW_BYTES)) & (ROW_BYTES / 32 - 1)) << 5;
}

template <class G, bool STATE_ONLY>
struct ChunkLds {
    static constexpr int XBYTES = G::A * G::C * G::XB, PBYTES = G::O * G::C * G::PB;
    // x, then the scores in its place (16-byte units exchanged); beside it where x has columns of
    // zeros, which have to stay
    static constexpr int PAT = G::DP > G::D ? XBYTES : 0;
    alignas(16) uint8_t x[STATE_ONLY ? 16 : (XBYTES > PAT + PBYTES ? XBYTES : PAT + PBYTES)];
    alignas(16) uint8_t y[G::A * G::C * G::XB];  // 32-byte units exchanged
    alignas(16) uint8_t z[G::A * G::C * G::ZB];
    alignas(16) float w[G::C];  // the update's weights: zscale l^(n - 1 - j + e) of token j
    float pw[G::C + 1];         // l^0 .. l^C
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

// A chunk's rows of one tensor on their way from memory to LDS: WIDTH columns. Row i of a chunk is
// the sweep's token i0 + i, which lies i rows after (or, backward, before) the chunk's first. Loads
// take a base that is the same for the workgroup and a 32-bit offset per thread (the launcher keeps
// the rows of a chunk within 32 bits).
template <class G, int WIDTH, int N>
struct Stage {
    using AT = typename G::AT;
    static constexpr int VPR = WIDTH / G::VE;
    static constexpr int RSTEP = G::NT / VPR;  // rows of the workgroup's one load
    static_assert(G::NT % VPR == 0, "a thread's loads are in one column");
    Run<AT, G::VE> r[N];
    const char* p;      // the lowest row of the next chunk's first load
    int64_t row;        // bytes between the sweep's tokens, signed
    uint32_t at;        // the thread's offset
    int first;          // the thread's row of the first load

    __device__ __forceinline__ void start(const AT* base, int64_t stride, int i0, int len, bool reverse) {
        first = threadIdx.x / VPR;
        const int t = reverse ? len - RSTEP - i0 : i0;  // may lie before the tensor; such rows are not read
        row = (reverse ? -stride : stride) * (int)sizeof(AT);
        p = (const char*)base + (int64_t)t * stride * (int)sizeof(AT);
        at = (uint32_t)(reverse ? RSTEP - 1 - first : first) * (uint32_t)(stride * sizeof(AT)) +
             (threadIdx.x % VPR) * 16;
    }
    // the next chunk, n of its tokens
    __device__ __forceinline__ void load(int n) {
        OPAQUE(at);
        OPAQUE(first);
        if (n >= G::C) {
#pragma unroll
            for (int u = 0; u < N; ++u) r[u].load((const AT*)(p + u * (RSTEP * row) + at));
        } else {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                if (first + u * RSTEP < n) r[u].load((const AT*)(p + u * (RSTEP * row) + at));
                else r[u].zero();
            }
        }
        p += G::C * row;
    }
    // to rows of ROW_BYTES, units of 16 or 32 bytes exchanged
    template <int ROW_BYTES, int UNIT>
    __device__ __forceinline__ void store(uint8_t* lds) const {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int row = first + u * RSTEP, c = (threadIdx.x % VPR) * G::VE * 2;
            uint8_t* q = lds + row * ROW_BYTES + (c ^ (UNIT == 16 ? swizzle16<ROW_BYTES>(row) : swizzle32<ROW_BYTES>(row)));
            if constexpr (G::A == 1) {
                *(u32x4*)q = u32x4{r[u].w[0], r[u].w[1], r[u].w[2], r[u].w[3]};
            } else {
                uint32_t w[G::VE / 2][G::A];
#pragma unroll
                for (int j = 0; j < G::VE / 2; ++j) split<G::A>(r[u].get(2 * j), r[u].get(2 * j + 1), w[j]);
#pragma unroll
                for (int a = 0; a < G::A; ++a) {
                    if constexpr (G::VE == 8) *(u32x4*)(q + a * G::C * ROW_BYTES) = u32x4{w[0][a], w[1][a], w[2][a], w[3][a]};
                    else *(u32x2*)(q + a * G::C * ROW_BYTES) = u32x2{w[0][a], w[1][a]};
                }
            }
        }
    }
};

// A 16-bit state value.
__device__ __forceinline__ float half_value(uint32_t bits, bool f16) {
    const float h = (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    return f16 ? h : __uint_as_float(bits << 16);
}

// Four consecutive values (y's dimension d .. d + 3 of row z) of head bh's state, of type t (one of two
// forms: the 16-bit types are told apart by a selection, not a branch).
template <int D>
__device__ __forceinline__ f32x4 load_state4(const void* p, DType t, int64_t bh, int z, int d) {
    const size_t i = (size_t)bh * D * D + (size_t)z * D + d;
    if (t == DType::F32) return *(const f32x4*)((const float*)p + i);
    const u32x2 w = *(const u32x2*)((const uint16_t*)p + i);
    const bool f16 = t == DType::F16;
    return f32x4{half_value(w.x & 0xffffu, f16), half_value(w.x >> 16, f16), half_value(w.y & 0xffffu, f16),
                 half_value(w.y >> 16, f16)};
}

// The same values of the transposed state.
template <int D>
__device__ __forceinline__ f32x4 load_state4_transposed(const void* p, DType t, int64_t bh, int z, int d) {
    const size_t i = (size_t)bh * D * D + (size_t)d * D + z;
    f32x4 v;
    if (t == DType::F32) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = ((const float*)p)[i + r * D];
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = half_value(((const uint16_t*)p)[i + r * D], t == DType::F16);
    }
    return v;
}

template <int D>
__device__ __forceinline__ void store_state4(void* p, DType t, int64_t bh, int z, int d, f32x4 v) {
    const size_t i = (size_t)bh * D * D + (size_t)z * D + d;
    if (t == DType::F32) {
        *(f32x4*)((float*)p + i) = v;
    } else {
        const bool f16 = t == DType::F16;
        const uint32_t h0 = Elem<_Float16>::pack(v.x, v.y), h1 = Elem<_Float16>::pack(v.z, v.w);
        const uint32_t b0 = Elem<uint16_t>::pack(v.x, v.y), b1 = Elem<uint16_t>::pack(v.z, v.w);
        *(u32x2*)((uint16_t*)p + i) = u32x2{f16 ? h0 : b0, f16 ? h1 : b1};
    }
}

struct ChunkArgs {
    Sweep s[3];
    int64_t BH;     // B * H
    int seg_tokens; // tokens of a segment (a multiple of C)
    int nseg;
    bool from_ws;   // first states are read from ws: with several segments, or transposed
    float* ws;      // [sweep][B * H][nseg][D][D] fp32, then: the segments' states
    bool mirror;    // sweep 1's states are sweep 2's transposed
};

// STATE_ONLY: each segment's own state from zero, for the scan that gives every segment its start.
// MIXED: a sweep's outputs may be fp32 (else all are of the activations' type).
template <class G, bool MIXED, bool STATE_ONLY>
__global__ __launch_bounds__(G::NT, G::WAVES) void gdn_linear_chunk_kernel(ChunkArgs a) {
    using AT = typename G::AT;
    constexpr int D = G::D, C = G::C, A = G::A, O = G::O, NV = G::NV;
    __shared__ ChunkLds<G, STATE_ONLY> L;
    const int sweep = STATE_ONLY && a.mirror && blockIdx.y == 1 ? 2 : blockIdx.y;
    const Sweep& s = a.s[sweep];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    int g = lane >> 4, n16 = lane & 15;
    const uint32_t id = blockIdx.x;
    const uint32_t segs = STATE_ONLY ? a.nseg - 1 : a.nseg;  // the last segment's own state is not wanted
    const int seg = (int)(id % segs);
    const uint32_t head = id / segs;  // B * H < 2^32 / (8 D)
    const int64_t bh = head, b = head / (uint32_t)s.H;
    const int h = (int)(head % (uint32_t)s.H);
    const int T = s.T, len = tokens_of(s.lengths, b, T);
    const int begin = min(seg * a.seg_tokens, len);
    const int end = (seg == a.nseg - 1) ? len : min((seg + 1) * a.seg_tokens, len);
    const bool reverse = s.reverse;
    const int e = reverse ? 1 : 0;
    const int zw = wave * 16 * NV;  // the wave's columns
    const float lam = s.decay[h];
    float* wst = a.ws + ((size_t)sweep * a.BH + bh) * a.nseg * D * D + (size_t)seg * D * D;

    if constexpr (!STATE_ONLY) {
        // outputs past the sequence's end: this segment's share
        const int r0 = max(seg * a.seg_tokens, len), r1 = seg == a.nseg - 1 ? T : min((seg + 1) * a.seg_tokens, T);
        if (r0 < r1) {
            const int es = MIXED && s.out_f32 ? 4 : (int)sizeof(AT), words = D * es / 8;
            char* o = (char*)s.out + ((size_t)b * T * s.H + h) * D * es;
            const size_t row = (size_t)s.H * D * es;
            for (int64_t i = tid; i < (int64_t)(r1 - r0) * words; i += G::NT)
                *(u32x2*)(o + (size_t)(r0 + i / words) * row + (i % words) * 8) = u32x2{0u, 0u};
        }
        // a segment without tokens; a sequence without any still hands on its state
        if (begin == end && !(len == 0 && seg == 0 && s.last != nullptr && s.last != s.first)) return;
    }

    for (int i = tid; i <= C; i += G::NT) L.pw[i] = (float)power(lam, i);
    for (int i = tid; i < C; i += G::NT) L.w[i] = s.zscale * (float)power(lam, C - 1 - i + e);
    if constexpr (G::DP > D) {  // the contraction's columns past D
        for (int i = tid; i < A * C * G::XB / 4; i += G::NT) {
            ((uint32_t*)L.y)[i] = 0u;
            if constexpr (!STATE_ONLY) ((uint32_t*)L.x)[i] = 0u;
        }
        __syncthreads();
    }

    // N^T: tile (dt, v), element r is N[z = zw + 16 v + n16][d = 16 dt + 4 g + r]
    f32x4 N[G::DT][NV];
    const auto each_tile = [&](auto&& f) {
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (16 * dt < D) {
                    f(N[dt][v], zw + 16 * v + n16, 16 * dt + 4 * g);
                    __builtin_amdgcn_sched_barrier(0);  // few addresses at a time
                }
    };
#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
        for (int v = 0; v < NV; ++v) N[dt][v] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (!STATE_ONLY) {
        if (a.from_ws) {
            each_tile([&](f32x4& t, int z, int d) { t = *(const f32x4*)(wst + (size_t)z * D + d); });
        } else if (s.first) {
            each_tile([&](f32x4& t, int z, int d) { t = load_state4<D>(s.first, s.state_dtype, bh, z, d); });
        }
    }

    const int Hx = s.H / s.gx, Hy = s.H / s.gy, Hz = s.H / s.gz;
    const int64_t xst = (int64_t)Hx * D, yst = (int64_t)Hy * D, zst = (int64_t)Hz * D;
    const AT* xp = (const AT*)s.x + ((size_t)b * T * Hx + h / s.gx) * D;
    const AT* yp = (const AT*)s.y + ((size_t)b * T * Hy + h / s.gy) * D;
    const AT* zp = (const AT*)s.z + ((size_t)b * T * Hz + h / s.gz) * D;
    Stage<G, D, STATE_ONLY ? 1 : G::XV> sx;
    Stage<G, D, G::XV> sy;
    Stage<G, D, G::XV> sz;
    if constexpr (!STATE_ONLY) sx.start(xp, xst, begin, len, reverse);
    sy.start(yp, yst, begin, len, reverse);
    sz.start(zp, zst, begin, len, reverse);
    const auto fetch = [&](int n) {
        if constexpr (!STATE_ONLY) sx.load(n);
        sy.load(n);
        sz.load(n);
    };
    const auto stage = [&] {
        if constexpr (!STATE_ONLY) sx.template store<G::XB, 16>(L.x);
        sy.template store<G::XB, 32>(L.y);
        sz.template store<G::ZB, 32>(L.z);
    };
    if (begin < end) {
        fetch(end - begin);
        stage();
    }

    // the lane's addresses in LDS; parts and rows 16 i are added to them, units within a row are
    // exclusive-ored (OPAQUE keeps the compiler from holding a register for each of those)
    const int tr = n16 >> 2, tc = (n16 & 3) * 8;  // transposed reads: row and bytes of a 4 x 16 block
    int xb = n16 * G::XB | ((8 * g) ^ swizzle16<G::XB>(n16));
    int xsb = n16 * G::XB | ((16 * g) ^ swizzle16<G::XB>(n16)), ysb = n16 * G::XB | ((16 * g) ^ swizzle32<G::XB>(n16));
    int yb = (4 * g + tr) * G::XB | (tc ^ swizzle32<G::XB>(4 * g + tr));
    int zb = (4 * g + tr) * G::ZB | (tc ^ swizzle32<G::ZB>(4 * g + tr));
    int pb = n16 * G::PB | ((8 * g) ^ swizzle16<G::PB>(n16));

    // outputs: the lowest of 16 tokens of the chunk's first column tile, and the lane's offset
    const bool f32 = MIXED && s.out_f32;
    const int es = f32 ? 4 : (int)sizeof(AT);
    const int64_t ostride = (int64_t)s.H * D * es, orow = reverse ? -ostride : ostride;
    char* out = (char*)s.out + ((int64_t)b * T + (reverse ? len - 16 - begin : begin)) * ostride + (int64_t)h * D * es;
    uint32_t oat = (uint32_t)(reverse ? 15 - n16 : n16) * (uint32_t)ostride + (uint32_t)((zw + (NV == 2 && sizeof(AT) == 2 && !f32 ? 8 * (g >> 1) + 16 * (g & 1) : 4 * g)) * es);

    // one chunk of n tokens (FULL: n = C); `left` tokens of the segment remain after it
    const auto chunk = [&](auto full, int n, int left) {
        constexpr bool FULL = decltype(full)::value;
        OPAQUE(g); OPAQUE(n16); OPAQUE(oat); OPAQUE(xb); OPAQUE(xsb); OPAQUE(ysb); OPAQUE(yb); OPAQUE(zb); OPAQUE(pb);
        if constexpr (!FULL) {
            for (int i = tid; i < C; i += G::NT) L.w[i] = s.zscale * (float)power(lam, max(n - 1 - i, 0) + e);
        }
        __syncthreads();

        // The next chunk's loads are issued a tensor at a time between the steps: a burst of all of them
        // fills the memory pipeline and stops the wave until it drains.
        if constexpr (STATE_ONLY) {
            if (left > 0) { sy.load(left); sz.load(left); }
        }
        // The steps below are fenced (STEP) so that each step's loads from LDS are in flight while
        // the step before them computes.
        f32x4 acc[STATE_ONLY ? 1 : NV][STATE_ONLY ? 1 : G::CT];
        u32x2 sc[STATE_ONLY ? 1 : G::TPW][O];
        int sat[STATE_ONLY ? 1 : G::TPW];
        if constexpr (!STATE_ONLY) {
            // scores: tile (ti, si), lane (g, n16) holds s = 16 si + 4 g + r of t = 16 ti + n16
            const float ps = s.oscale * s.zscale;
            int ti[G::TPW], si[G::TPW];
            f32x4 c[G::TPW];
#pragma unroll
            for (int i = 0; i < G::TPW; ++i) {
                const int tile = min(wave + i * G::W, G::TILES - 1);
                ti[i] = (int)((C == 64 ? 0x203333222110ull : 0x0110ull) >> (4 * tile)) & 15;
                si[i] = (int)((C == 64 ? 0x313210210100ull : 0x1100ull) >> (4 * tile)) & 15;
                c[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            u32x4 yf[2][G::TPW][A], xf[2][G::TPW][A];
            const auto load_scores = [&](int kk) {
#pragma unroll
                for (int i = 0; i < G::TPW; ++i)
#pragma unroll
                    for (int p = 0; p < A; ++p) {
                        yf[kk & 1][i][p] = *(const u32x4*)&L.y[p * C * G::XB + ((16 * si[i] * G::XB + ysb) ^ (64 * kk))];
                        xf[kk & 1][i][p] = *(const u32x4*)&L.x[p * C * G::XB + ((16 * ti[i] * G::XB + xsb) ^ (64 * kk))];
                    }
            };
            u32x4 qf[2][G::CT][A];  // x, columns t
            u32x4 nf[2][O];         // N in parts: 32 rows of one column tile
            const auto load_x = [&](int kk) {
#pragma unroll
                for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                    for (int u = 0; u < A; ++u) {
                        const u32x2 x0 = *(const u32x2*)&L.x[(u * C + 16 * ct) * G::XB + (xb ^ (64 * kk))];
                        const u32x2 x1 = *(const u32x2*)&L.x[(u * C + 16 * ct) * G::XB + (xb ^ (64 * kk + 32))];
                        qf[kk & 1][ct][u] = u32x4{x0.x, x0.y, x1.x, x1.y};
                    }
            };
            const auto split_state = [&](int step) {
                const int kk = step / NV, v = step % NV;
                uint32_t w[4][O];
                split<O>(N[2 * kk][v].x, N[2 * kk][v].y, w[0]);
                split<O>(N[2 * kk][v].z, N[2 * kk][v].w, w[1]);
                split<O>(N[2 * kk + 1][v].x, N[2 * kk + 1][v].y, w[2]);
                split<O>(N[2 * kk + 1][v].z, N[2 * kk + 1][v].w, w[3]);
#pragma unroll
                for (int p = 0; p < O; ++p) nf[step & 1][p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
            };
            load_scores(0);
            float lag[G::TPW][4];  // l^(t - s)
#pragma unroll
            for (int i = 0; i < G::TPW; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) lag[i][r] = L.pw[max(16 * ti[i] + n16 - (16 * si[i] + 4 * g + r), 0)];
            STEP;
#pragma unroll
            for (int kk = 0; kk < G::DK; ++kk) {
                if (kk + 1 < G::DK) {
                    load_scores(kk + 1);
                } else {
                    load_x(0);
                    split_state(0);
                }
#pragma unroll
                for (int p = A - 1; p >= 0; --p)
#pragma unroll
                    for (int u = A - 1; u >= 0; --u)
#pragma unroll
                        for (int i = 0; i < G::TPW; ++i)
                            if (p + u < kParts) c[i] = mfma(yf[kk & 1][i][p], xf[kk & 1][i][u], c[i]);
                STEP;
            }

            // out^T = N x: rows z = zw + 16 v + 4 g + r, column t = 16 ct + n16
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int ct = 0; ct < G::CT; ++ct) acc[v][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int step = 0; step < G::DK * NV; ++step) {
                const int kk = step / NV, v = step % NV;
                if (step == G::DK * NV / 4 && left > 0) sx.load(left);
                if (step == G::DK * NV * 3 / 4 && left > 0) sy.load(left);
                if (v == 0 && kk + 1 < G::DK) load_x(kk + 1);
                if (step + 1 < G::DK * NV) split_state(step + 1);
                if (step == 0) {  // weights of the scores
#pragma unroll
                    for (int i = 0; i < G::TPW; ++i) {
                        const int t = 16 * ti[i] + n16, s0 = 16 * si[i] + 4 * g;
                        float w[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) w[r] = lag[i][r] * c[i][r];
#pragma unroll
                        for (int r = 0; r < 4; ++r) w[r] = t >= s0 + r ? w[r] : 0.0f;
                        uint32_t lo[O], hi[O];
                        split<O>(ps * w[0], ps * w[1], lo);
                        split<O>(ps * w[2], ps * w[3], hi);
#pragma unroll
                        for (int p = 0; p < O; ++p) sc[i][p] = u32x2{lo[p], hi[p]};
                        sat[i] = t * G::PB + ((32 * si[i] + 8 * g) ^ swizzle16<G::PB>(t));
                    }
                }
#pragma unroll
                for (int p = O - 1; p >= 0; --p)
#pragma unroll
                    for (int u = A - 1; u >= 0; --u)
#pragma unroll
                        for (int ct = 0; ct < G::CT; ++ct)
                            if (p + u < kParts) acc[v][ct] = mfma(nf[step & 1][p], qf[kk & 1][ct][u], acc[v][ct]);
                STEP;
            }
        }

        // z transposed: tokens 32 kk + 16 (j / 4) + 4 g + j % 4, j = 0..7, of column n16; y likewise
        u32x4 zf[G::CK][NV][A];
#pragma unroll
        for (int kk = 0; kk < G::CK; ++kk)
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int u = 0; u < A; ++u) {
                    const uint8_t* p = &L.z[(u * C + 32 * kk) * G::ZB + (zb ^ (32 * (wave * NV + v)))];
                    const u32x2 a0 = read_tr(p), a1 = read_tr(p + 16 * G::ZB);
                    zf[kk][v][u] = u32x4{a0.x, a0.y, a1.x, a1.y};
                }
        constexpr int YG = A == 1 && G::DT >= 4 ? 4 : 2, YS = G::DT / YG;  // y tiles of a step, steps of 32 tokens
        u32x4 yt[2][YG][A];
        const auto load_y = [&](int step) {
#pragma unroll
            for (int i = 0; i < YG; ++i)
#pragma unroll
                for (int u = 0; u < A; ++u) {
                    const uint8_t* p = &L.y[(u * C + 32 * (step / YS)) * G::XB + (yb ^ (32 * (step % YS * YG + i)))];
                    const u32x2 a0 = read_tr(p), a1 = read_tr(p + 16 * G::XB);
                    yt[step & 1][i][u] = u32x4{a0.x, a0.y, a1.x, a1.y};
                }
        };
        load_y(0);
        u32x4 wf[NV][O];  // weighted z in parts
        const auto weigh = [&](int kk) {
            const f32x4 w0 = *(const f32x4*)&L.w[32 * kk + 4 * g], w1 = *(const f32x4*)&L.w[32 * kk + 16 + 4 * g];
            const float wl[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                uint32_t w[4][O];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4(&zz)[A] = zf[kk][v];
                    float z0 = __uint_as_float(zz[A - 1][j] << 16), z1 = __uint_as_float(zz[A - 1][j] & 0xffff0000u);
#pragma unroll
                    for (int u = A - 2; u >= 0; --u) {
                        z0 += __uint_as_float(zz[u][j] << 16);
                        z1 += __uint_as_float(zz[u][j] & 0xffff0000u);
                    }
                    split<O>(z0 * wl[2 * j], z1 * wl[2 * j + 1], w[j]);
                }
#pragma unroll
                for (int p = 0; p < O; ++p) wf[v][p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
            }
        };

        if constexpr (!STATE_ONLY) {
            float f[G::CT];
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) f[ct] = s.oscale * L.pw[16 * ct + n16 + 1 - e];
            __syncthreads();  // x has been read
#pragma unroll
            for (int i = 0; i < G::TPW; ++i)
#pragma unroll
                for (int p = 0; p < O; ++p) *(u32x2*)&L.x[L.PAT + p * C * G::PB + sat[i]] = sc[i][p];
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                for (int v = 0; v < NV; ++v) acc[v][ct] *= f[ct];
            __syncthreads();
            if (left > 0) sz.load(left);
            // out^T += z^T scores^T
            u32x4 pf[2][G::CT];  // one part of the scores of 32 tokens
            const auto load_weighted = [&](int step) {
                const int kk = step / O, p = O - 1 - step % O;
#pragma unroll
                for (int ct = 2 * kk; ct < G::CT; ++ct) {
                    const u32x2 p0 = *(const u32x2*)&L.x[L.PAT + (p * C + 16 * ct) * G::PB + (pb ^ (64 * kk))];
                    const u32x2 p1 = *(const u32x2*)&L.x[L.PAT + (p * C + 16 * ct) * G::PB + (pb ^ (64 * kk + 32))];
                    pf[step & 1][ct] = u32x4{p0.x, p0.y, p1.x, p1.y};
                }
            };
            load_weighted(0);
#pragma unroll
            for (int step = 0; step < G::CK * O; ++step) {
                const int kk = step / O, p = O - 1 - step % O;
                if (step + 1 < G::CK * O) load_weighted(step + 1);
#pragma unroll
                for (int u = A - 1; u >= 0; --u)
#pragma unroll
                    for (int ct = 2 * kk; ct < G::CT; ++ct)
#pragma unroll
                        for (int v = 0; v < NV; ++v)
                            if (p + u < kParts) acc[v][ct] = mfma(zf[kk][v][u], pf[step & 1][ct], acc[v][ct]);
                STEP;
            }
        }
        weigh(0);
        const float carry = FULL ? L.pw[C] : L.pw[n];
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
            for (int v = 0; v < NV; ++v) N[dt][v] *= carry;
        STEP;
        if constexpr (!STATE_ONLY) {
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) {
                char* o = out + 16 * ct * orow + oat;
                if constexpr (NV == 2 && sizeof(AT) == 2) {
                    if (!f32) {
                        // two tiles' halves exchanged between lanes of neighbouring g: 16 bytes a lane (even
                        // g: columns 4 g .. + 7 of the first tile, odd g: 4 (g - 1) .. + 7 of the second)
                        uint32_t w[2][2];
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            w[v][0] = Elem<AT>::pack(acc[v][ct].x, acc[v][ct].y);
                            w[v][1] = Elem<AT>::pack(acc[v][ct].z, acc[v][ct].w);
                        }
                        const auto s0 = __builtin_amdgcn_permlane16_swap(w[0][0], w[1][0], false, false);
                        const auto s1 = __builtin_amdgcn_permlane16_swap(w[0][1], w[1][1], false, false);
                        if (FULL || 16 * ct + n16 < n) *(u32x4*)o = u32x4{s0[0], s1[0], s0[1], s1[1]};
                        continue;
                    }
                }
                if (FULL || 16 * ct + n16 < n) {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const float f[4] = {acc[v][ct].x, acc[v][ct].y, acc[v][ct].z, acc[v][ct].w};
                        if (f32) {
                            *(f32x4*)((float*)o + 16 * v) = acc[v][ct];
                        } else {
                            Run<AT, 4> r;
                            r.set(f);
                            r.store((AT*)o + 16 * v);
                        }
                    }
                }
            }
            out += C * orow;
        }
        // the state's update
#pragma unroll
        for (int step = 0; step < G::CK * YS; ++step) {
            const int dt0 = step % YS * YG;
            if (step + 1 < G::CK * YS) load_y(step + 1);
#pragma unroll
            for (int p = O - 1; p >= 0; --p)
#pragma unroll
                for (int u = A - 1; u >= 0; --u)
#pragma unroll
                    for (int i = 0; i < YG; ++i)
#pragma unroll
                        for (int v = 0; v < NV; ++v)
                            if (p + u < kParts && 16 * (dt0 + i) < D)
                                N[dt0 + i][v] = mfma(yt[step & 1][i][u], wf[v][p], N[dt0 + i][v]);
            if (step + 1 < G::CK * YS && (step + 1) % YS == 0) weigh((step + 1) / YS);
            STEP;
        }
        __syncthreads();
        if (left > 0) stage();
    };
    int i0 = begin;
    for (; end - i0 >= C; i0 += C) chunk(std::true_type{}, C, end - i0 - C);
    if (i0 < end) chunk(std::false_type{}, end - i0, 0);

    if constexpr (STATE_ONLY) {
        each_tile([&](f32x4& t, int z, int d) { *(f32x4*)(wst + (size_t)z * D + d) = t; });
    } else if (s.last && end == len && (begin < len || seg == 0)) {
        each_tile([&](f32x4& t, int z, int d) { store_state4<D>(s.last, s.state_dtype, bh, z, d, t); });
    }
}

// The segments' starts from their own states, in place: start[0] is the sweep's first state,
// start[i + 1] = l^(tokens of i) start[i] + own[i]; with `mirror`, sweep 1's from sweep 2's.
template <int D>
__global__ __launch_bounds__(256) void gdn_linear_scan_kernel(ChunkArgs a) {
    const int sweep = a.mirror && blockIdx.y == 1 ? 2 : blockIdx.y;
    const Sweep& s = a.s[sweep];
    constexpr int PER = D * D / 4;  // vectors of a state
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < a.BH * PER; id += (int64_t)gridDim.x * 256) {
        const int64_t bh = id / PER;
        const uint32_t b = (uint32_t)bh / (uint32_t)s.H, h = (uint32_t)bh % (uint32_t)s.H;
        const int z = (int)(id % PER) / (D / 4), d = (int)(id % (D / 4)) * 4;
        const int len = tokens_of(s.lengths, b, s.T);
        const float lam = s.decay[h];
        f32x4 N = {0.f, 0.f, 0.f, 0.f};
        if (s.first)
            N = s.transposed ? load_state4_transposed<D>(s.first, s.state_dtype, bh, z, d)
                             : load_state4<D>(s.first, s.state_dtype, bh, z, d);
        const size_t base = (size_t)bh * a.nseg * D * D, sweeps = (size_t)a.BH * a.nseg * D * D;
        float* w = a.ws + sweep * sweeps + base + (size_t)z * D + d;
        float* m = a.ws + sweeps + base + (size_t)d * D + z;
        const float whole = (float)power(lam, a.seg_tokens);
        constexpr int AHEAD = 8;  // states read ahead of the sums
        for (int s0 = 0; s0 < a.nseg; s0 += AHEAD) {
            f32x4 own[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                own[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (s0 + i + 1 < a.nseg) own[i] = *(const f32x4*)(w + (size_t)i * D * D);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int seg = s0 + i;
                if (seg >= a.nseg) break;
                *(f32x4*)(w + (size_t)i * D * D) = N;
                if (sweep == 2) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) m[(size_t)i * D * D + (size_t)r * D] = N[r];
                }
                const int n = min((seg + 1) * a.seg_tokens, len) - min(seg * a.seg_tokens, len);
                N = N * (n == a.seg_tokens ? whole : (float)power(lam, n)) + own[i];
            }
            w += AHEAD * D * D;
            m += AHEAD * D * D;
        }
    }
}

// ------------------------------------------------------------------------ the decay's gradient

// With M_t = dS_t / dl = l M_{t-1} + S_{t-1} the loss's derivative is sum_t scale do_t . (M_t q_t) +
// <dS_T, M_T>. A chunk of n tokens from S and M regroups (differentiating the chunked form) into
//     M_i q_i = l^(i+1) M q_i + (i+1) l^i S q_i + sum_{j < i} (i-j) l^(i-j-1) (q_i . k_j) v_j
//     M_next  = l^n M + n l^(n-1) S + sum_j (n-1-j) l^(n-2-j) v_j k_j^T
// A forward sweep (x = q, y = k, z = v) with both states in registers, 16 state columns a wave. Its terms
// cancel in the sum, so every factor keeps three parts (2^-24) whatever the activations' type. Each
// workgroup writes one partial sum.
struct TangentArgs {
    Sweep s;              // forward; out unused, first: S before the call (or nullptr)
    const void* d_o;      // act [B][T][H][D]
    const void* dstate;   // state_dtype [B][H][D][D] or nullptr
    int64_t BH;
    int seg_tokens, nseg;
    float* ws;            // [2][B * H][nseg][D][D]: the segments' S and M, if nseg > 1
    float* part;          // [nseg][B * H]
};

template <class G, bool STATE_ONLY>
struct TangentLds {
    static constexpr int XBYTES = G::A * G::C * G::XB, PBYTES = 3 * G::C * G::PB;
    static constexpr int PAT = G::DP > G::D ? XBYTES : 0;
    alignas(16) uint8_t x[STATE_ONLY ? 16 : (XBYTES > PAT + PBYTES ? XBYTES : PAT + PBYTES)];
    alignas(16) uint8_t y[G::A * G::C * G::XB];
    alignas(16) uint8_t z[G::A * G::C * G::ZB];
    alignas(16) float w[G::C];   // l^(n - 1 - j)
    alignas(16) float wd[G::C];  // its derivative
    float pw[G::C + 1];          // l^i
    float pd[G::C + 1];          // i l^(i - 1)
    double sum[G::W];
};

template <class G, bool STATE_ONLY>
__global__ __launch_bounds__(G::NT, G::WAVES) void gdn_linear_tangent_chunk_kernel(TangentArgs a) {
    using AT = typename G::AT;
    constexpr int D = G::D, C = G::C, A = G::A, O = 3;
    static_assert(G::NV == 1, "16 columns a wave");
    __shared__ TangentLds<G, STATE_ONLY> L;
    const Sweep& s = a.s;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int g = lane >> 4, n16 = lane & 15;
    const uint32_t id = blockIdx.x;
    const uint32_t segs = STATE_ONLY ? a.nseg - 1 : a.nseg;
    const int seg = (int)(id % segs);
    const uint32_t head = id / segs;  // B * H < 2^32 / (8 D)
    const int64_t bh = head, b = head / (uint32_t)s.H;
    const int h = (int)(head % (uint32_t)s.H);
    const int T = s.T, len = tokens_of(s.lengths, b, T);
    const int begin = min(seg * a.seg_tokens, len);
    const int end = (seg == a.nseg - 1) ? len : min((seg + 1) * a.seg_tokens, len);
    const int zw = wave * 16;
    const float lam = s.decay[h];
    float* ws = a.ws + (bh * a.nseg + seg) * D * D;
    const size_t wm = (size_t)a.BH * a.nseg * D * D;  // M's states after S's

    for (int i = tid; i <= C; i += G::NT) {
        L.pw[i] = (float)power(lam, i);
        L.pd[i] = i ? (float)((double)i * power(lam, i - 1)) : 0.0f;
    }
    if constexpr (G::DP > D) {
        for (int i = tid; i < A * C * G::XB / 4; i += G::NT) {
            ((uint32_t*)L.y)[i] = 0u;
            if constexpr (!STATE_ONLY) ((uint32_t*)L.x)[i] = 0u;
        }
    }
    __syncthreads();

    f32x4 S[G::DT], M[G::DT];
#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt) {
        S[dt] = M[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (!STATE_ONLY) {
            if (16 * dt < D) {
                const int z = zw + n16, d = 16 * dt + 4 * g;
                if (a.nseg > 1) {
                    S[dt] = *(const f32x4*)(ws + (size_t)z * D + d);
                    M[dt] = *(const f32x4*)(ws + wm + (size_t)z * D + d);
                } else if (s.first) {
                    S[dt] = load_state4<D>(s.first, s.state_dtype, bh, z, d);
                }
            }
        }
    }

    const int Hx = s.H / s.gx, Hz = s.H / s.gz;
    Stage<G, D, STATE_ONLY ? 1 : G::XV> sx;
    Stage<G, D, G::XV> sy;
    Stage<G, D, G::XV> sz;
    if constexpr (!STATE_ONLY) sx.start((const AT*)s.x + ((size_t)b * T * Hx + h / s.gx) * D, (int64_t)Hx * D, begin, len, false);
    sy.start((const AT*)s.y + ((size_t)b * T * Hx + h / s.gx) * D, (int64_t)Hx * D, begin, len, false);
    sz.start((const AT*)s.z + ((size_t)b * T * Hz + h / s.gz) * D, (int64_t)Hz * D, begin, len, false);
    const AT* dop = (const AT*)a.d_o + (((size_t)b * T + begin + n16) * s.H + h) * D + zw + 4 * g;
    const auto fetch = [&](int n) {
        if constexpr (!STATE_ONLY) sx.load(n);
        sy.load(n);
        sz.load(n);
    };
    if (begin < end) fetch(end - begin);

    const int tr = n16 >> 2, tc = (n16 & 3) * 8;
    const int xb = n16 * G::XB | ((8 * g) ^ swizzle16<G::XB>(n16));
    const int xsb = n16 * G::XB | ((16 * g) ^ swizzle16<G::XB>(n16)), ysb = n16 * G::XB | ((16 * g) ^ swizzle32<G::XB>(n16));
    const int yb = (4 * g + tr) * G::XB | (tc ^ swizzle32<G::XB>(4 * g + tr));
    const int zb = (4 * g + tr) * G::ZB | (tc ^ swizzle32<G::ZB>(4 * g + tr));
    const int pb = n16 * G::PB | ((8 * g) ^ swizzle16<G::PB>(n16));
    double total = 0.0;

    for (int i0 = begin; i0 < end; i0 += C) {
        const int n = min(C, end - i0);
        if constexpr (!STATE_ONLY) sx.template store<G::XB, 16>(L.x);
        sy.template store<G::XB, 32>(L.y);
        sz.template store<G::ZB, 32>(L.z);
        if (i0 == begin || n < C) {
            for (int i = tid; i < C; i += G::NT) {
                L.w[i] = L.pw[max(n - 1 - i, 0)];
                L.wd[i] = L.pd[max(n - 1 - i, 0)];
            }
        }
        __syncthreads();
        if (i0 + C < end) fetch(end - i0 - C);

        if constexpr (!STATE_ONLY) {
            f32x4 dv[G::CT];  // scale do
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) {
                dv[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (16 * ct + n16 < n) {
                    Run<AT, 4> r;
                    r.load(dop + (size_t)16 * ct * s.H * D);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dv[ct][j] = s.oscale * r.get(j);
                }
            }
            dop += (size_t)C * s.H * D;
            u32x2 sc[G::TPW][O];
            int sat[G::TPW];
#pragma unroll
            for (int i = 0; i < G::TPW; ++i) {
                const int tile = min(wave + i * G::W, G::TILES - 1);
                const int ti = (int)((C == 64 ? 0x203333222110ull : 0x0110ull) >> (4 * tile)) & 15;
                const int si = (int)((C == 64 ? 0x313210210100ull : 0x1100ull) >> (4 * tile)) & 15;
                f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < G::DK; ++kk) {
                    u32x4 yf[A], xf[A];
#pragma unroll
                    for (int p = 0; p < A; ++p) {
                        yf[p] = *(const u32x4*)&L.y[p * C * G::XB + ((16 * si * G::XB + ysb) ^ (64 * kk))];
                        xf[p] = *(const u32x4*)&L.x[p * C * G::XB + ((16 * ti * G::XB + xsb) ^ (64 * kk))];
                    }
#pragma unroll
                    for (int p = A - 1; p >= 0; --p)
#pragma unroll
                        for (int u = A - 1; u >= 0; --u)
                            if (p + u < 3) c = mfma(yf[p], xf[u], c);
                }
                const int t = 16 * ti + n16, s0 = 16 * si + 4 * g;
                float w[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r] = L.pd[max(t - s0 - r, 0)] * c[r];
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r] = t > s0 + r ? w[r] : 0.0f;
                uint32_t lo[O], hi[O];
                split<O>(w[0], w[1], lo);
                split<O>(w[2], w[3], hi);
#pragma unroll
                for (int p = 0; p < O; ++p) sc[i][p] = u32x2{lo[p], hi[p]};
                sat[i] = t * G::PB + ((32 * si + 8 * g) ^ swizzle16<G::PB>(t));
            }
            f32x4 as[G::CT], am[G::CT];
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) as[ct] = am[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < G::DK; ++kk) {
                u32x4 sf[O], mf[O];
                uint32_t w[4][O];
                split<O>(S[2 * kk].x, S[2 * kk].y, w[0]);
                split<O>(S[2 * kk].z, S[2 * kk].w, w[1]);
                split<O>(S[2 * kk + 1].x, S[2 * kk + 1].y, w[2]);
                split<O>(S[2 * kk + 1].z, S[2 * kk + 1].w, w[3]);
#pragma unroll
                for (int p = 0; p < O; ++p) sf[p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
                split<O>(M[2 * kk].x, M[2 * kk].y, w[0]);
                split<O>(M[2 * kk].z, M[2 * kk].w, w[1]);
                split<O>(M[2 * kk + 1].x, M[2 * kk + 1].y, w[2]);
                split<O>(M[2 * kk + 1].z, M[2 * kk + 1].w, w[3]);
#pragma unroll
                for (int p = 0; p < O; ++p) mf[p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
#pragma unroll
                for (int ct = 0; ct < G::CT; ++ct) {
                    u32x4 xf[A];
#pragma unroll
                    for (int u = 0; u < A; ++u) {
                        const u32x2 x0 = *(const u32x2*)&L.x[(u * C + 16 * ct) * G::XB + (xb ^ (64 * kk))];
                        const u32x2 x1 = *(const u32x2*)&L.x[(u * C + 16 * ct) * G::XB + (xb ^ (64 * kk + 32))];
                        xf[u] = u32x4{x0.x, x0.y, x1.x, x1.y};
                    }
#pragma unroll
                    for (int p = O - 1; p >= 0; --p)
#pragma unroll
                        for (int u = A - 1; u >= 0; --u)
                            if (p + u < 3) {
                                as[ct] = mfma(sf[p], xf[u], as[ct]);
                                am[ct] = mfma(mf[p], xf[u], am[ct]);
                            }
                }
            }
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct)
                am[ct] = am[ct] * L.pw[16 * ct + n16 + 1] + as[ct] * L.pd[16 * ct + n16 + 1];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < G::TPW; ++i)
#pragma unroll
                for (int p = 0; p < O; ++p) *(u32x2*)&L.x[L.PAT + p * C * G::PB + sat[i]] = sc[i][p];
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < G::CK; ++kk) {
                u32x4 zf[A];
#pragma unroll
                for (int u = 0; u < A; ++u) {
                    const uint8_t* p = &L.z[(u * C + 32 * kk) * G::ZB + (zb ^ (32 * wave))];
                    const u32x2 a0 = read_tr(p), a1 = read_tr(p + 16 * G::ZB);
                    zf[u] = u32x4{a0.x, a0.y, a1.x, a1.y};
                }
#pragma unroll
                for (int ct = 2 * kk; ct < G::CT; ++ct)
#pragma unroll
                    for (int p = O - 1; p >= 0; --p) {
                        const u32x2 p0 = *(const u32x2*)&L.x[L.PAT + (p * C + 16 * ct) * G::PB + (pb ^ (64 * kk))];
                        const u32x2 p1 = *(const u32x2*)&L.x[L.PAT + (p * C + 16 * ct) * G::PB + (pb ^ (64 * kk + 32))];
#pragma unroll
                        for (int u = A - 1; u >= 0; --u)
                            if (p + u < 3) am[ct] = mfma(zf[u], u32x4{p0.x, p0.y, p1.x, p1.y}, am[ct]);
                    }
            }
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) {
                const f32x4 m = am[ct] * dv[ct];
                const float sum = (m.x + m.y) + (m.z + m.w);
                total += 16 * ct + n16 < n ? (double)sum : 0.0;  // past n a growing power may be an infinity
            }
        }

        const float ln = L.pw[n], dn = L.pd[n];
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt) {
            M[dt] = M[dt] * ln + S[dt] * dn;
            S[dt] *= ln;
        }
#pragma unroll
        for (int kk = 0; kk < G::CK; ++kk) {
            u32x4 zf[A], wf[3], df[3];
#pragma unroll
            for (int u = 0; u < A; ++u) {
                const uint8_t* p = &L.z[(u * C + 32 * kk) * G::ZB + (zb ^ (32 * wave))];
                const u32x2 a0 = read_tr(p), a1 = read_tr(p + 16 * G::ZB);
                zf[u] = u32x4{a0.x, a0.y, a1.x, a1.y};
            }
            const f32x4 w0 = *(const f32x4*)&L.w[32 * kk + 4 * g], w1 = *(const f32x4*)&L.w[32 * kk + 16 + 4 * g];
            const f32x4 d0 = *(const f32x4*)&L.wd[32 * kk + 4 * g], d1 = *(const f32x4*)&L.wd[32 * kk + 16 + 4 * g];
            const float wl[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            const float dl[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
            uint32_t w[4][3], d[4][3];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v0 = __uint_as_float(zf[A - 1][j] << 16), v1 = __uint_as_float(zf[A - 1][j] & 0xffff0000u);
#pragma unroll
                for (int u = A - 2; u >= 0; --u) {
                    v0 += __uint_as_float(zf[u][j] << 16);
                    v1 += __uint_as_float(zf[u][j] & 0xffff0000u);
                }
                split<3>(v0 * wl[2 * j], v1 * wl[2 * j + 1], w[j]);
                split<3>(v0 * dl[2 * j], v1 * dl[2 * j + 1], d[j]);
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                wf[p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
                df[p] = u32x4{d[0][p], d[1][p], d[2][p], d[3][p]};
            }
#pragma unroll
            for (int dt = 0; dt < G::DT; ++dt) {
                if (16 * dt >= D) continue;
#pragma unroll
                for (int u = A - 1; u >= 0; --u) {
                    const uint8_t* p = &L.y[(u * C + 32 * kk) * G::XB + (yb ^ (32 * dt))];
                    const u32x2 a0 = read_tr(p), a1 = read_tr(p + 16 * G::XB);
                    const u32x4 yf = {a0.x, a0.y, a1.x, a1.y};
#pragma unroll
                    for (int q = 2; q >= 0; --q)
                        if (q + u < 3) {
                            S[dt] = mfma(yf, wf[q], S[dt]);
                            M[dt] = mfma(yf, df[q], M[dt]);
                        }
                }
            }
        }
        __syncthreads();
    }

    if constexpr (STATE_ONLY) {
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt)
            if (16 * dt < D) {
                const size_t i = (size_t)(zw + n16) * D + 16 * dt + 4 * g;
                *(f32x4*)(ws + i) = S[dt];
                *(f32x4*)(ws + wm + i) = M[dt];
            }
    } else {
        if (a.dstate && end == len && begin < len) {  // the sequence's end (without tokens M is 0, whatever dstate holds)
#pragma unroll
            for (int dt = 0; dt < G::DT; ++dt)
                if (16 * dt < D) {
                    const f32x4 r = load_state4<D>(a.dstate, s.state_dtype, bh, zw + n16, 16 * dt + 4 * g) * M[dt];
                    total += (double)((r.x + r.y) + (r.z + r.w));
                }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m);
        if (lane == 0) L.sum[wave] = total;
        __syncthreads();
        if (tid == 0) {
#pragma unroll
            for (int i = 1; i < G::W; ++i) total += L.sum[i];
            a.part[(size_t)seg * a.BH + bh] = (float)total;
        }
    }
}

// The segments' starts of S and M: M's takes the derivative of the decay over the segment times S's.
template <int D>
__global__ __launch_bounds__(256) void gdn_linear_tangent_scan_kernel(TangentArgs a) {
    const Sweep& s = a.s;
    constexpr int PER = D * D / 4;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t bh = id / PER;
    if (bh >= a.BH) return;
    const int z = (int)(id % PER) / (D / 4), d = (int)(id % (D / 4)) * 4;
    const int len = tokens_of(s.lengths, (uint32_t)bh / (uint32_t)s.H, s.T);
    const float lam = s.decay[(uint32_t)bh % (uint32_t)s.H];
    f32x4 S = {0.f, 0.f, 0.f, 0.f}, M = {0.f, 0.f, 0.f, 0.f};
    if (s.first) S = load_state4<D>(s.first, s.state_dtype, bh, z, d);
    float* w = a.ws + (size_t)bh * a.nseg * D * D + (size_t)z * D + d;
    const size_t wm = (size_t)a.BH * a.nseg * D * D;
    for (int seg = 0; seg < a.nseg; ++seg, w += D * D) {
        f32x4 own = {0.f, 0.f, 0.f, 0.f}, mown = own;
        if (seg + 1 < a.nseg) {
            own = *(const f32x4*)w;
            mown = *(const f32x4*)(w + wm);
        }
        *(f32x4*)w = S;
        *(f32x4*)(w + wm) = M;
        const int n = min((seg + 1) * a.seg_tokens, len) - min(seg * a.seg_tokens, len);
        const float ln = (float)power(lam, n), dn = n ? (float)((double)n * power(lam, n - 1)) : 0.0f;
        M = M * ln + S * dn + mown;
        S = S * ln + own;
    }
}

// ------------------------------------------------------------------------ dispatch

template <typename F, typename Args>
hipError_t launch(F kernel, dim3 grid, int threads, hipStream_t st, Args a) {
    void* args[] = {&a};
    return hipLaunchKernel((const void*)kernel, grid, dim3((unsigned)threads), args, 0, st);
}

template <class G>
hipError_t chunk_g(const ChunkArgs& a, int n, bool mixed, hipStream_t st) {
    constexpr int D = G::D;
    const unsigned heads = (unsigned)a.BH, own = a.mirror ? 2 : n;
    if (a.nseg > 1) {
        hipError_t e = launch(gdn_linear_chunk_kernel<G, false, true>, dim3(heads * (a.nseg - 1), own), G::NT, st, a);
        if (e != hipSuccess) return e;
    }
    if (a.from_ws) {
        const int64_t blocks = (a.BH * D * D / 4 + 255) / 256, most = 1 << 20;  // a dispatch covers fewer than 2^32 work-items
        hipError_t e = launch(gdn_linear_scan_kernel<D>, dim3((unsigned)(blocks < most ? blocks : most), own), 256, st, a);
        if (e != hipSuccess) return e;
    }
    const dim3 grid(heads * a.nseg, (unsigned)n);
    if constexpr (G::A != 3) {
        if (mixed) return launch(gdn_linear_chunk_kernel<G, true, false>, grid, G::NT, st, a);
    }
    return launch(gdn_linear_chunk_kernel<G, false, false>, grid, G::NT, st, a);
}

// Four waves a head where D has the columns, two column tiles each at D = 128 (eight waves of one tile read
// every operand from LDS twice as often and took as long).
template <int D, typename AT>
hipError_t chunk_t(const Sweep* sweeps, int n, int64_t B, float* ws, hipStream_t st) {
    constexpr int W = D >= 64 ? 4 : D / 16, NV = D / 16 / W;
    using G = ChunkGeo<D, AT, W, NV>;
    ChunkArgs a;
    bool mixed = false;  // is an output fp32?
    for (int i = 0; i < n; ++i) {
        a.s[i] = sweeps[i];
        mixed = mixed || sweeps[i].out_f32;
    }
    const int T = sweeps[0].T, H = sweeps[0].H;
    a.BH = B * H;
    a.nseg = linear_segments(B, T, H, n);
    a.seg_tokens = ((T + a.nseg - 1) / a.nseg + 63) / 64 * 64;
    a.nseg = (T + a.seg_tokens - 1) / a.seg_tokens;
    a.from_ws = a.nseg > 1;
    for (int i = 0; i < n; ++i) a.from_ws = a.from_ws || (sweeps[i].transposed && sweeps[i].first);
    a.ws = ws;
    a.mirror = n == 3;
    return chunk_g<G>(a, n, mixed, st);
}

// One column tile a wave: S and M of two would not fit its registers.
template <int D, typename AT>
hipError_t tangent_t(TangentArgs a, int64_t B, int64_t* parts, hipStream_t st) {
    constexpr int W = D / 16;
    using G = ChunkGeo<D, AT, W, 1>;
    a.BH = B * a.s.H;
    a.nseg = linear_segments(B, a.s.T, a.s.H, 1);
    a.seg_tokens = ((a.s.T + a.nseg - 1) / a.nseg + 63) / 64 * 64;
    a.nseg = (a.s.T + a.seg_tokens - 1) / a.seg_tokens;
    const unsigned heads = (unsigned)a.BH;
    if (a.nseg > 1) {
        hipError_t e = launch(gdn_linear_tangent_chunk_kernel<G, true>, dim3(heads * (a.nseg - 1)), G::NT, st, a);
        if (e != hipSuccess) return e;
        e = launch(gdn_linear_tangent_scan_kernel<D>, dim3((unsigned)((a.BH * D * D / 4 + 255) / 256)), 256, st, a);
        if (e != hipSuccess) return e;
    }
    a.part = a.ws + linear_tangent_state_floats(B, a.s.T, a.s.H, D);
    *parts = a.nseg;
    return launch(gdn_linear_tangent_chunk_kernel<G, false>, dim3(heads * a.nseg), G::NT, st, a);
}

template <int D>
hipError_t tangent_d(const TangentArgs& a, int64_t B, DType act, int64_t* parts, hipStream_t st) {
    switch (act) {
        case DType::F32: return tangent_t<D, float>(a, B, parts, st);
        case DType::BF16: return tangent_t<D, uint16_t>(a, B, parts, st);
        default: return tangent_t<D, _Float16>(a, B, parts, st);
    }
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

hipError_t launch_linear_tangent(const LinearBackwardArgs& b, float* ws, int64_t* parts, hipStream_t st) {
    const int g = b.H / b.Hk;
    TangentArgs a{};
    a.s = Sweep{b.T, b.H, g, g, 1, b.q, b.k, b.v, b.decay, b.lengths, b.state0, nullptr, nullptr, 1.0f, b.scale,
                false, false, false, b.state_dtype};
    a.d_o = b.d_o;
    a.dstate = b.dstate;
    a.ws = ws;
    switch (b.D) {
        case 16: return tangent_d<16>(a, b.B, b.act, parts, st);
        case 32: return tangent_d<32>(a, b.B, b.act, parts, st);
        case 64: return tangent_d<64>(a, b.B, b.act, parts, st);
        default: return tangent_d<128>(a, b.B, b.act, parts, st);
    }
}

}  // namespace gdn
