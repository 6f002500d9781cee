// The gated linear recurrence h <- alpha h + beta x of every channel, over a few tokens, over prompts, and its
// gradients.
//
// A token is the map h -> alpha h + u of its channel, and maps compose: (P, H) after (p, u) is (P p, P u + H). A
// tile of 64 tokens is split over the waves of a workgroup along the tokens; each lane composes its tokens' maps
// in registers, the waves' maps meet in LDS, and a state at the tile's start then gives every token's. So every input
// is read once and the tokens of a sequence are worked on at once; only the state at its start waits for the tile before.
// (With the tiles' maps, the states between them and the outputs in launches of their own, which read the inputs twice,
// 4 x 4096 tokens of 6144 bf16 channels took 368 us forward and 762 backward; now 178 and 334.)
// Where states grow, products of decays can leave fp32's range although the states do not; such channels are walked
// through token by token (walk_forward, walk_backward).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_linear_common.h"
#include "gdn_scan_launch.h"

namespace gdn {
namespace {

constexpr int64_t kMaxBlocks = 1 << 20;  // of a launch; more work is taken in a loop

// -------------------------------------------------------------------------------------------- gates

constexpr float kMost = 3.402823466385288598e38f;  // fp32's largest number
constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.925963033500011e-8f, kLn2 = 0.693147182464599609375f;

// 2^-|p| for p = x log2 e. Of the product's rounding error, 2^-24 |x| of the result, fp32 inputs take the part that was
// lost along; next to the rounding of a 16-bit result it is nothing.
template <bool EXACT>
__device__ __forceinline__ float exp_neg(float x, float p) {
    const float w = __builtin_amdgcn_exp2f(-fabsf(p));
    if constexpr (!EXACT) return w;
    const float low = fmaf(fabsf(x), kLog2eLow, fmaf(fabsf(x), kLog2e, -fabsf(p)));
    return w == 0.0f ? w : fmaf(w, low * -kLn2, w);
}

// sigmoid(b)
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float b) {
    if constexpr (EXACT) {
        const float w = exp_neg<true>(b, b * kLog2e), r = __builtin_amdgcn_rcpf(1.0f + w);
        return b >= 0.0f ? r : w * r;
    } else {
        return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(b * -kLog2e));
    }
}

// A sigmoid beside its complement: the smaller of sigmoid(b) and sigmoid(-b), with its sign bit set where that is the latter
// (the bit, not the comparison with 0: from b = 88 on it is -0, and sigmoid(b) 1).
template <bool EXACT>
__device__ __forceinline__ float smaller_sigmoid(float b) {
    const float w = exp_neg<EXACT>(b, b * kLog2e), s = w * __builtin_amdgcn_rcpf(1.0f + w);
    return b >= 0.0f ? -s : s;
}
__device__ __forceinline__ float sigmoid_of(float z) { return __builtin_signbitf(z) ? 1.0f + z : z; }
__device__ __forceinline__ float sigmoid_slope_of(float z) { return fabsf(z) * (1.0f - fabsf(z)); }

// A token's decay alpha = exp(-rate softplus(a)), and 1 - alpha without cancellation. Within a tile's 64 tokens
// alpha v is a product with alpha; over a long memory alpha's rounding, step after step, would add up where it is
// next to 1, so the products P of alphas, which carry states from tile to tile, take P - (1 - alpha) P there. Away from 1
// that difference would round at P's size, not at what is left of it, so they take alpha P: where a token leaves
// 2e-6 of a state, the difference is off by 2^-24 of the state, 3 % of what is left.
struct Decay {
    float alpha, lost;  // lost: 1 - alpha
    bool near;          // alpha is next to 1
    float step;         // - (1 - alpha) where it is, else alpha
    float e;            // alpha = 2^-e (with a rate)
    float soft;         // softplus(a) log2 e
    float up;           // sigmoid(a)
    __device__ __forceinline__ float of(float p) const { return fmaf(step, p, near ? p : 0.0f); }
    // alpha v, alpha h + u and (1 - alpha) x token by token, where a rate below 0 (grows) may also take alpha itself past
    // fp32's range and the product not: in four parts, which pass it only if the product does.
    __device__ __forceinline__ float grown(float v) const {
        const float q = __builtin_amdgcn_exp2f(e * -0.25f);
        return v == 0.0f ? v : v * q * q * q * q;
    }
    __device__ __forceinline__ float times(bool grows, float v) const { return grows && alpha > kMost ? grown(v) : alpha * v; }
    __device__ __forceinline__ float next(bool grows, float h, float u) const {
        if (grows && alpha > kMost) return grown(h) + u;
        return (near ? h : 0.0f) + fmaf(step, h, u);  // the larger terms last where the state stays as it is
    }
    __device__ __forceinline__ float lost_of(bool grows, float x) const {
        return grows && alpha > kMost ? x - grown(x) : lost * x;
    }
};

// log2(1 + w) with what 1 + w rounds away added back, + max(p, 0): softplus in units of ln 2, for p = a log2 e and
// w = 2^-|p|. It stays finite for an infinite a (or one whose p is), so that its products with a gradient or a rate of 0 are 0.
__device__ __forceinline__ float softplus2(float p, float w) {
    const float u = 1.0f + w, lost = w - (u - 1.0f);
    return fmaf(lost, kLog2e, __builtin_amdgcn_logf(u)) + __builtin_amdgcn_fmed3f(p, 0.0f, kMost);  // (w keeps a NaN)
}

// Without a rate (1) alpha = sigmoid(-a). soft: softplus is wanted there too. What is not used is not computed.
template <bool EXACT, bool RATE>
__device__ __forceinline__ Decay decay_of(float a, float rate, bool soft) {
    Decay d;
    const float p = a * kLog2e, w = exp_neg<EXACT>(a, p);
    if constexpr (!RATE) {
        const float r = __builtin_amdgcn_rcpf(1.0f + w), s = w * r;
        d.lost = d.up = a >= 0.0f ? r : s;
        d.alpha = a >= 0.0f ? s : r;
        d.near = !(a >= 0.0f);
        d.step = a >= 0.0f ? s : -s;
        d.soft = soft ? softplus2(p, w) : 0.0f;
    } else {
        d.soft = softplus2(p, w);
        const float e = d.e = rate * d.soft;
        d.alpha = __builtin_amdgcn_exp2f(-e);
        // 1 - 2^-e as its series up to (e ln 2)^5 / 120 for |e ln 2| < 1/8 (the next term is below 2^-24 of it)
        const float series = e * fmaf(e, fmaf(e, fmaf(e, fmaf(e, 1.33335581464284434e-3f, -9.61812910762847716e-3f),
                                                      5.55041086648215800e-2f), -2.40226506959100712e-1f), kLn2);
        d.near = fabsf(e) < 0.18f;
        d.lost = d.near ? series : 1.0f - d.alpha;
        d.step = d.near ? -series : d.alpha;
        const float r = __builtin_amdgcn_rcpf(1.0f + w);
        d.up = a >= 0.0f ? r : w * r;
    }
    return d;
}

// Whether a wave has a channel whose states may grow.
template <int V>
__device__ __forceinline__ bool any_below_0(const float* rate) {
    bool below = false;
#pragma unroll
    for (int v = 0; v < V; ++v) below = below || rate[v] < 0.0f;
    return __any(below);
}

// Whether a wave has a product of decays past fp32's range.
template <int V>
__device__ __forceinline__ bool any_past(const float* p) {
    bool past = false;
#pragma unroll
    for (int v = 0; v < V; ++v) past = past || !(p[v] <= kMost);
    return __any(past);
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

// A row's address, the same for the wave, kept in scalar registers: with the lane's offset it is the address of a load
// or store, without vector arithmetic or a pair of vector registers for each.
struct RowAt {
    uint64_t p;
    int64_t step;  // bytes to the next row
    template <typename T>
    __device__ __forceinline__ RowAt(const T* base, int64_t st) : p((uint64_t)base), step(st * (int64_t)sizeof(T)) {}
    template <typename T>
    __device__ __forceinline__ T* at(unsigned& lane_bytes) const {
        typedef __attribute__((address_space(1))) char global_char;
        global_char* q = (global_char*)p;
        asm("" : "+s"(q), "+v"(lane_bytes));  // (no instruction: the sum is made where it is used, not before)
        return (T*)(q + lane_bytes);
    }
};

// S rows of a wave's segment, V channels a lane. base: the segment's first row and the tile's first channel; at: the
// lane's channel within the tile.
template <typename T, int V, int S>
struct Rows {
    Run<T, V> r[S];
    // The rows from n on are not read: `fill` is put in their place.
    __device__ __forceinline__ void load(const T* base, int64_t st, unsigned at, int n, uint32_t fill) {
        RowAt row(base, st);
        unsigned off = at * (unsigned)sizeof(T);
        if (n == S) {
#pragma unroll
            for (int s = 0; s < S; ++s, row.p += row.step) r[s].template load<true>(row.at<const T>(off));
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s, row.p += row.step) {
#pragma unroll
                for (int i = 0; i < Run<T, V>::WORDS; ++i) r[s].w[i] = fill;
                if (s < n) r[s].template load<true>(row.at<const T>(off));
            }
        }
    }
    // Stores the first `rows` rows; those from n on as zeros.
    __device__ __forceinline__ void store(T* base, int64_t st, unsigned at, int n, int rows) {
        RowAt row(base, st);
        unsigned off = at * (unsigned)sizeof(T);
        if (n == S) {
#pragma unroll
            for (int s = 0; s < S; ++s, row.p += row.step) r[s].store(row.at<T>(off));
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s, row.p += row.step) {
                if (s >= n) r[s].zero();
                if (s < rows) r[s].store(row.at<T>(off));
            }
        }
    }
};

// -infinity in every value of a word: as a gate `a` it leaves the state as it is, bit for bit, with x = 0.
template <typename T> constexpr uint32_t kShut = 0xff800000u;
template <> constexpr uint32_t kShut<uint16_t> = 0xff80ff80u;
template <> constexpr uint32_t kShut<_Float16> = 0xfc00fc00u;

// -------------------------------------------------------------------------------------------- few tokens

// A lane takes V channels of a sequence through its tokens. Bound by the launch and, with many channels, by memory: one
// token of 256 sequences of 6144 bf16 channels with fp32 states (25 MB) takes 6.7 us, 3.7 TB/s.
template <typename T, int V, bool COUPLED, bool RATE>
__global__ __launch_bounds__(256) void gdn_scan_decode_kernel(ScanArgs a) {
    constexpr bool EXACT = sizeof(T) == 4;
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
                bool far = false;  // a decay past fp32's range: the token is taken again with care
                const auto token = [&](bool grows) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const Decay d = decay_of<EXACT, RATE>(ga.get(v), rate[v], false);
                        const float xv = x.get(v), u = COUPLED ? d.lost_of(grows, xv) : sigmoid<EXACT>(gb.get(v)) * xv;
                        o[v] = d.next(grows, h[v], u);
                        far = far || d.alpha > kMost;
                    }
                };
                token(false);
                if (RATE && __builtin_expect(__any(far), 0)) token(true);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = o[v];
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

__device__ __forceinline__ int64_t scan_chunks_of(int T) { return ((int64_t)T + kScanChunk - 1) / kScanChunk; }

// The tile of a workgroup: sequence, TT tokens and 64 V channels, and the wave's segment of S tokens in it.
template <int V, int S, int TT>
struct Tile {
    int64_t b, j, c0;  // sequence, tile along the tokens, first channel
    int64_t t0;        // the segment's first token
    int n, rows;       // tokens of the segment within the sequence, and within T
    unsigned at;       // the lane's channel within the tile; 0 for lanes past C
    bool on;           // the lane has channels
    int len;

    // `chain`: sequence and channels; `along`: the tile's place among the chain's (REV: from the last).
    template <bool REV>
    __device__ __forceinline__ static Tile of(const ScanArgs& a, unsigned chain, unsigned along, int wave) {
        const unsigned width = ((unsigned)a.C + 64 * V - 1) / (64 * V), tiles = ((unsigned)a.T + TT - 1) / TT;
        Tile t;
        t.b = chain / width;
        t.c0 = (int64_t)(chain - (unsigned)t.b * width) * (64 * V);
        t.j = REV ? tiles - 1 - along : along;
        t.len = __builtin_amdgcn_readfirstlane(tokens_of(a.lengths, t.b, a.T));
        const int t0 = (int)t.j * TT + wave * S;   // T < 2^30
        t.t0 = t0;
        t.n = max(0, min(t.len - t0, S));
        t.rows = max(0, min(a.T - t0, S));
        t.at = (threadIdx.x & 63) * V;
        t.on = t.c0 + t.at < a.C;
        if (!t.on) t.at = 0;
        return t;
    }
    template <typename T>
    __device__ __forceinline__ T* base(const RowsView& v) const { return (T*)v.p + b * v.sb + t0 * v.st + c0; }
};

// What passes from tile to tile along the tokens: one fp32 value for each channel and tile boundary. kNothing, a NaN
// that no computed value is, marks the ones still to come.
constexpr uint32_t kNothing = 0xffffffffu;

__device__ __forceinline__ void publish(float* p, float h) {
    const uint32_t bits = h == h ? __float_as_uint(h) : 0x7fc00000u;
    __hip_atomic_store((uint32_t*)p, bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// V values from the tile before. Asked for while the tile's own work goes on (look) and waited for after it (get):
// whoever publishes them has an earlier ticket and so is running already, and the wait ends by itself. (Its bound,
// tens of seconds, only keeps a workspace that is written to meanwhile from stopping the card.)
template <int V>
struct Passed {
    uint32_t bits[V];
    __device__ __forceinline__ bool look(const float* p) {
        bool all = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bits[v] = __hip_atomic_load((const uint32_t*)p + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            all = all && bits[v] != kNothing;
        }
        return all;
    }
    __device__ __forceinline__ bool here() const {
        bool all = true;
#pragma unroll
        for (int v = 0; v < V; ++v) all = all && bits[v] != kNothing;
        return all;
    }
    __device__ __forceinline__ void get(const float* p, float* h) {
        bool all = here();
        for (int tries = 0; !all && tries < (1 << 25); ++tries) {
            __builtin_amdgcn_s_sleep(1);
            all = look(p);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __uint_as_float(bits[v]);
    }
    // In a group of tiles only the first tile's value is passed on, from group to group. A tile that is number i of its
    // group takes it (edge) through the maps of the i tiles before it, which are there as soon as those tiles' own work
    // is done; they are composed in order, whenever they come. map: P of the tile before, map + half its H, - k step
    // those before it. p, u: the composed map.
    __device__ __forceinline__ static void maps_before(const float* map, int64_t step, int64_t half, int i, float* p, float* u) {
#pragma unroll
        for (int v = 0; v < V; ++v) { p[v] = 1.0f; u[v] = 0.0f; }
        Passed<V> mp[2], mu[2];
        const float* m = map - (i - 1) * step;
        if (i > 0) { mp[0].look(m); mu[0].look(m + half); }
        for (int k = 0; k < i; k += 2) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (k + e < i) {
                    const float* next = m + step;
                    if (k + e + 1 < i) { mp[1 - e].look(next); mu[1 - e].look(next + half); }
                    float q[V], w[V];
                    mp[e].get(m, q);
                    mu[e].get(m + half, w);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        p[v] *= q[v];
                        u[v] = fmaf(q[v], u[v], w[v]);
                    }
                    m = next;
                }
            }
        }
    }
    // Where a rate below 0 takes p past fp32's range, h goes through the maps (they are there) one by one; p and u become the
    // map to where it ends.
    __device__ __forceinline__ static void one_by_one(const float* map, int64_t step, int64_t half, int i, const float* h, float* p,
                                                      float* u) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (p[v] <= kMost) continue;
            p[v] = 0.0f;
            u[v] = h[v];
            const float* m = map - (i - 1) * step + v;
            for (int k = 0; k < i; ++k, m += step) {
                Passed<1> q, w;
                q.look(m);
                w.look(m + half);
                u[v] = fmaf(__uint_as_float(q.bits[0]), u[v], __uint_as_float(w.bits[0]));
            }
        }
    }
};

// How the tiles are handed out: the chains (a sequence's 64 V channels) in groups with a ticket counter each, and
// within a group the tiles of all its chains step by step along the tokens. Tickets are drawn by workgroups that run,
// so of a group's tiles not done yet the first is always in work, and waiting for the tile before one's own ends. (A
// ticket takes some 18 ns of its counter: with one counter the 1024 workgroups that run at once start over 18 us. A
// workgroup that took several chains' tiles per ticket had more tiles of each chain under way than the chain serves.)
// One tile along the tokens waits for nothing: the workgroups share those out without counters.
constexpr unsigned kGroups = 8;
static_assert(2 * kGroups * kScanCounterStride == kScanCounterFloats, "counters of both directions");
struct Tickets {
    unsigned* counters;       // kScanCounterStride apart, or nullptr
    unsigned groups;          // no more than kGroups, nor than chains
    unsigned chains, along;   // chains of the call, tiles of each
    static constexpr unsigned kNone = 0xffffffffu;
    struct Draw { unsigned chain, along; bool done; };
    // `last`: the ticket before, kNone at first; `turn` is in LDS.
    __device__ __forceinline__ Draw next(unsigned* last, unsigned* turn) const {
        Draw d;
        __syncthreads();
        if (!counters) {
            const unsigned n = *last == kNone ? blockIdx.x : *last + gridDim.x;
            *last = n;
            d.chain = n;
            d.along = 0;
            d.done = n >= chains;
            return d;
        }
        const unsigned g = blockIdx.x % groups;
        if (threadIdx.x == 0)
            *turn = __hip_atomic_fetch_add(counters + g * kScanCounterStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        const unsigned n = (unsigned)__builtin_amdgcn_readfirstlane((int)*turn);
        const unsigned mine = (chains + groups - 1 - g) / groups;  // the group's chains: g, g + groups, ...
        d.along = n / mine;
        d.chain = g + groups * (n - d.along * mine);
        d.done = d.along >= along;
        return d;
    }
};

// Clears the edges of a call, its tiles' maps and its ticket counters.
__global__ __launch_bounds__(256) void gdn_scan_clear_kernel(uint32_t* edges, int64_t n, uint32_t* maps, int64_t m,
                                                             unsigned* counters) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    if (i0 < 2 * kGroups) counters[i0 * kScanCounterStride] = 0;  // of both directions
    const u32x4 none = {kNothing, kNothing, kNothing, kNothing};
    for (int64_t i = i0; i < n / 4; i += step) ((u32x4*)edges)[i] = none;
    if (i0 < n % 4) edges[n / 4 * 4 + i0] = kNothing;
    for (int64_t i = i0; i < m / 4; i += step) ((u32x4*)maps)[i] = none;
    if (i0 < m % 4) maps[m / 4 * 4 + i0] = kNothing;
}

// Tiles in a group where a value passes from group to group (GROUP), for calls with few chains: a step from tile to
// tile takes some 0.65 us, whatever the tiles hold.
constexpr int kGroup = 8;

// The arguments of the tiles' kernels. starts: the states at the chunks' starts; behind: the adjoints behind their ends;
// rates: the rates' gradient of every chunk, or nullptr; ends: the tiles' maps.
struct TileArgs {
    ScanArgs a;
    Tickets tickets;
    float *starts, *behind, *rates, *ends;
};

// A kernel's only argument, read anew: what a rare path needs of it then holds no registers before.
__device__ __forceinline__ TileArgs arguments_again() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    TileArgs g;
    __builtin_memcpy(&g, (const void*)p, sizeof(g));
    return g;
}
__device__ __forceinline__ unsigned again(unsigned x) {
    asm volatile("" : "+s"(x));
    return x;
}

// Forward: o (OUT), and the state before every 64th token in starts [B][chunks][C]; between tiles the states pass
// through it. One workgroup takes one tile after the other in the order of its tickets. A lane keeps P and H after each of
// its 16 tokens, so that one product and sum gives the output once the tile's first state is known, with no second pass
// over the gates. Bound by memory, with the vector units half busy on the gates (33 vector instructions a value): 812 MB in 178 us,
// 4.6 TB/s. When it took 190 us, one chunk a sequence, without tickets, took 160, and four channels a lane and half the tokens 298.
// One wave takes the channels of a tile that are set in `walk` token by token, from the states in `first`, and passes on
// the states at their end; within a group as the map h -> 0 h + end.
template <typename T, int V, int W, bool GROUP, bool COUPLED, bool OUT>
__device__ __forceinline__ void walk_forward(unsigned chain, unsigned along, unsigned walk, const float (*first)[64]) {
    constexpr int S = 16, TT = S * W, PER = TT / kScanChunk;
    constexpr bool EXACT = sizeof(T) == 4;
    const TileArgs g = arguments_again();
    const ScanArgs& a = g.a;
    const Tile<V, S, TT> t = Tile<V, S, TT>::template of<false>(a, chain, along, 0);
    const int n = (int)min(t.len - t.t0, (int64_t)TT), rows = (int)min(a.T - t.t0, (int64_t)TT);
#pragma unroll 1
    for (int v = 0; v < V; ++v) {
        if (!(walk >> v & 1)) continue;
        const int64_t c = t.c0 + t.at + v;
        const auto row = [&](const RowsView& w, int s) { return (T*)w.p + t.b * w.sb + (t.t0 + s) * w.st + c; };
        float* start = g.starts ? g.starts + (t.b * scan_chunks_of(a.T) + t.j * PER) * a.C + c : nullptr;
        float h = first[v][threadIdx.x & 63];
        for (int s = 0; s < rows; ++s) {
            if (s > 0 && s % kScanChunk == 0 && start) start[s / kScanChunk * (int64_t)a.C] = h;
            if (s >= n) continue;
            const Decay d = decay_of<EXACT, true>(to_f32<T>(*row(a.a, s)), a.rate[c], false);
            const float x = to_f32<T>(*row(a.x, s));
            h = d.next(true, h, COUPLED ? d.lost_of(true, x) : sigmoid<EXACT>(to_f32<T>(*row(a.b, s))) * x);
            if (OUT) *row(a.o, s) = from_f32<T>(h);
        }
        if (t.t0 + TT >= a.T) {
            if (OUT && t.len > 0) set_state(a.state, a.state_dtype, t.b * a.C + c, h);
        } else if (GROUP && t.j % kGroup < kGroup - 1) {
            float* map = g.ends + (t.b * g.tickets.along + t.j) * a.C + c;
            publish(map, 0.0f);
            publish(map + a.B * g.tickets.along * a.C, h);
        } else {
            publish(start + PER * (int64_t)a.C, h);
        }
    }
}

template <typename T, int V, int W, bool GROUP, bool COUPLED, bool RATE, bool OUT>
__global__ __launch_bounds__(64 * W) void gdn_scan_forward_kernel(TileArgs g) {
    const ScanArgs& a = g.a;
    const Tickets& tickets = g.tickets;
    float *const starts = g.starts, *const ends = g.ends;
    constexpr int S = 16, TT = S * W;
    constexpr bool EXACT = sizeof(T) == 4;
    __shared__ float maps[W][2 * V][64], first[V][64];
    __shared__ unsigned turn, walks, walk_of[64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t chunks = scan_chunks_of(a.T);
    for (unsigned last = Tickets::kNone;;) {
        const Tickets::Draw draw = tickets.next(&last, &turn);
        if (draw.done) break;
        const Tile<V, S, TT> t = Tile<V, S, TT>::template of<false>(a, draw.chain, draw.along, wave);
        float rate[V];  // first: it is waited for before the rows are there
#pragma unroll
        for (int v = 0; v < V; ++v) rate[v] = RATE ? a.rate[t.c0 + t.at + v] : 1.0f;
        Rows<T, V, S> x, ga, gb;
        ga.load(t.template base<const T>(a.a), a.a.st, t.at, t.n, kShut<T>);
        if (!COUPLED) gb.load(t.template base<const T>(a.b), a.b.st, t.at, t.n, 0u);
        x.load(t.template base<const T>(a.x), a.x.st, t.at, t.n, 0u);
        float P[V], H[V], ps[S][V], hs[S][V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.0f;
            H[v] = 0.0f;
        }
        float* mine = starts + (t.b * chunks + t.j * (TT / kScanChunk)) * a.C + t.c0 + t.at;
        const int in_group = GROUP ? (int)(t.j % kGroup) : 0;
        const bool grows = RATE && any_below_0<V>(rate);
        float* edge = mine - in_group * (TT / kScanChunk) * (int64_t)a.C;
        Passed<V> passed;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s == S / 2 && t.j > 0 && wave == W - 1) {
                __builtin_amdgcn_sched_barrier(0);
                passed.look(edge);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay d = decay_of<EXACT, RATE>(ga.r[s].get(v), rate[v], false);
                const float beta = COUPLED ? d.lost : sigmoid<EXACT>(gb.r[s].get(v));
                P[v] = d.of(P[v]);
                H[v] = fmaf(d.alpha, H[v], beta * x.r[s].get(v));
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
        // The tile's map, its first state, the next tile's; by itself where no states grow (one sequence of 65536
        // tokens of 2048 channels 215 us; 223 with the questions in between).
        const auto join = [&](auto grow) {
            constexpr bool growing = decltype(grow)::value;
            const int64_t i = t.b * a.C + t.c0 + t.at;
            float h[V], p[V], u[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = maps[0][2 * v][lane];
                u[v] = maps[0][2 * v + 1][lane];
                for (int w = 1; w < W; ++w) {
                    const float q = maps[w][2 * v][lane];
                    p[v] *= q;
                    u[v] = fmaf(q, u[v], maps[w][2 * v + 1][lane]);
                }
            }
            const bool last_tile = (t.j + 1) * TT >= a.T;
            const int64_t half = a.B * tickets.along * a.C;
            float* map = ends + (t.b * tickets.along + t.j) * a.C + t.c0 + t.at;
            unsigned pass = t.on ? (1u << V) - 1 : 0;  // bit v: the channel has a map to pass on
            if constexpr (growing) {
#pragma unroll
                for (int v = 0; v < V; ++v) pass &= p[v] <= kMost ? ~0u : ~(1u << v);
                const bool walked = __any(t.on && pass + 1 != 1u << V);
                if (lane == 0) walks = walked;
                if (walked) walk_of[lane] = t.on ? ~pass : 0;
            }
            if (GROUP && in_group < kGroup - 1 && !last_tile && t.on) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (!growing || (pass >> v & 1)) {
                        publish(map + v, p[v]);
                        publish(map + half + v, u[v]);
                    }
            }
            if (t.j > 0) {
                if constexpr (GROUP) {
                    float bp[V], bu[V];
                    Passed<V>::maps_before(map - a.C, a.C, half, in_group, bp, bu);
                    passed.get(edge, h);
                    if (growing && any_past<V>(bp)) Passed<V>::one_by_one(map - a.C, a.C, half, in_group, h, bp, bu);
#pragma unroll
                    for (int v = 0; v < V; ++v) h[v] = fmaf(bp[v], h[v], bu[v]);
                } else {
                    passed.get(edge, h);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = a.state ? state_at(a.state, a.state_dtype, i + v) : 0.0f;
            }
            if (t.on) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float end = fmaf(p[v], h[v], u[v]);
                    if (!growing || (pass >> v & 1)) {
                        if (last_tile) {
                            if (OUT && t.len > 0) set_state(a.state, a.state_dtype, i + v, end);
                        } else if (!GROUP || in_group == kGroup - 1) {
                            publish(mine + (TT / kScanChunk) * (int64_t)a.C + v, end);
                        }
                    }
                    if (starts && (t.j == 0 || in_group > 0)) publish(mine + v, h[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) first[v][lane] = h[v];
        };
        if (wave == W - 1) {
            if (RATE && __builtin_expect(grows, 0)) join(std::bool_constant<RATE>{}); else join(std::false_type{});
        }
        __syncthreads();
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = first[v][lane];
            for (int w = 0; w < wave; ++w) h[v] = fmaf(maps[w][2 * v][lane], h[v], maps[w][2 * v + 1][lane]);
        }
        if (TT > kScanChunk && wave > 0 && wave % (kScanChunk / S) == 0 && starts && t.on && t.t0 < a.T)
#pragma unroll
            for (int v = 0; v < V; ++v) mine[wave / (kScanChunk / S) * (int64_t)a.C + v] = h[v];
        if constexpr (OUT) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = fmaf(ps[s][v], h[v], hs[s][v]);
                x.r[s].set(o);
            }
            if (t.on) x.store(t.template base<T>(a.o), a.o.st, t.at, t.n, t.rows);
        }
        // States that grow (a rate below 0) can take the tile's product of decays past fp32's range where they, 0 or tiny, stay
        // within it. Such channels are walked through here, over the rows and states that were stored from that product.
        if (__builtin_expect(grows && __builtin_amdgcn_readfirstlane((int)walks), 0)) {
            __syncthreads();
            if (wave == W - 1)
                walk_forward<T, V, W, GROUP, COUPLED, OUT>(again(draw.chain), again(draw.along), walk_of[lane], first);
        }
    }
}

// One wave takes the channels of a tile that are set in `walk` through their states (states: kept, in LDS) to the tile's
// end and back, from the adjoints in `after`, and passes on the adjoints before the tile.
template <typename T, int V, bool GROUP, bool COUPLED>
__device__ __forceinline__ void walk_backward(unsigned chain, unsigned along, unsigned walk, const float (*after)[64],
                                              float* states) {
    constexpr int S = 16;
    constexpr bool EXACT = sizeof(T) == 4;
    const TileArgs g = arguments_again();
    const ScanArgs& a = g.a;
    const Tile<V, S, kScanChunk> t = Tile<V, S, kScanChunk>::template of<true>(a, chain, along, 0);
    const int64_t chunks = scan_chunks_of(a.T);
    const int n = (int)min(t.len - t.t0, (int64_t)kScanChunk);
    states += threadIdx.x & 63;
#pragma unroll 1
    for (int v = 0; v < V; ++v) {
        if (!(walk >> v & 1)) continue;
        const int64_t c = t.c0 + t.at + v, i = t.b * a.C + c, at = (t.b * chunks + t.j) * a.C + c;
        const float rate = a.rate[c];
        const auto row = [&](const RowsView& w, int s) { return (T*)w.p + t.b * w.sb + (t.t0 + s) * w.st + c; };
        float h = g.starts ? g.starts[at] : (a.state0 ? state_at(a.state0, a.state_dtype, i) : 0.0f);
        for (int s = 0; s < n; ++s) {
            states[64 * s] = h;
            const Decay d = decay_of<EXACT, true>(to_f32<T>(*row(a.a, s)), rate, false);
            const float x = to_f32<T>(*row(a.x, s));
            h = d.next(true, h, COUPLED ? d.lost_of(true, x) : sigmoid<EXACT>(to_f32<T>(*row(a.b, s))) * x);
        }
        float r = after[v][threadIdx.x & 63], sum = 0.0f;
        for (int s = n - 1; s >= 0; --s) {
            const Decay d = decay_of<EXACT, true>(to_f32<T>(*row(a.a, s)), rate, true);
            const float x = to_f32<T>(*row(a.x, s)), now = to_f32<T>(*row(a.d_o, s)) + r;
            r = d.times(true, now);
            const float e = r * (COUPLED ? x - states[64 * s] : -states[64 * s]);
            *row(a.da, s) = from_f32<T>(e * d.up * rate);
            if constexpr (COUPLED) {
                *row(a.dx, s) = from_f32<T>(d.lost_of(true, now));
            } else {
                const float z = smaller_sigmoid<EXACT>(to_f32<T>(*row(a.b, s)));
                *row(a.dx, s) = from_f32<T>(now * sigmoid_of(z));
                *row(a.db, s) = from_f32<T>(now * x * sigmoid_slope_of(z));
            }
            sum = fmaf(e, d.soft, sum);
        }
        if (g.rates) g.rates[at] = sum * kLn2;
        if (t.j == 0) {
            if (a.dstate0) set_state(a.dstate0, a.state_dtype, i, r);
        } else if (GROUP && along % kGroup < kGroup - 1) {
            publish(g.ends + at, 0.0f);
            publish(g.ends + a.B * chunks * a.C + at, r);
        } else {
            publish(g.behind + at - a.C, r);
        }
    }
}

// (Bound by memory and issue: 1.42 GB in 334 us, 4.2 TB/s, the vector units 55% busy. A lane has one channel and 16 tokens,
// a workgroup four waves (385 us when it was made so; with two channels, 8 tokens and eight waves, whose maps each wave folds, it
// had been 466); at 128 registers four waves fit a SIMD, for which sigmoid(a) and softplus(a) wait in LDS.)
// Backward: the gradients of a tile from the state at its start (`starts`, or state0 for a call of one chunk) and the
// adjoint r behind its end, which passes from tile to tile through `behind` [B][chunks][C]; r -> alpha (do + r) for
// each token from the last to the first.
template <typename T, int V, bool GROUP, bool COUPLED, bool RATE>
__global__ __launch_bounds__(256, 4) void gdn_scan_backward_kernel(TileArgs g) {
    const ScanArgs& a = g.a;
    const Tickets& tickets = g.tickets;
    const float* const starts = g.starts;
    float *const behind = g.behind, *const rates = g.rates, *const ends = g.ends;
    constexpr int S = 16, W = kScanChunk / S;
    constexpr bool EXACT = sizeof(T) == 4;
    __shared__ float maps[W][3 * V][64], after[V][64];
    __shared__ float2 aside[S * V][64 * W];  // sigmoid(a), softplus(a): registers for more waves
    __shared__ unsigned turn, walks, walk_of[64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t chunks = scan_chunks_of(a.T);
    for (unsigned last = Tickets::kNone;;) {
        const Tickets::Draw draw = tickets.next(&last, &turn);
        if (draw.done) break;
        const Tile<V, S, kScanChunk> t = Tile<V, S, kScanChunk>::template of<true>(a, draw.chain, draw.along, wave);
        Rows<T, V, S> x, ga, gb, go;
        ga.load(t.template base<const T>(a.a), a.a.st, t.at, t.n, kShut<T>);
        go.load(t.template base<const T>(a.d_o), a.d_o.st, t.at, t.n, 0u);
        if (!COUPLED) gb.load(t.template base<const T>(a.b), a.b.st, t.at, t.n, 0u);
        x.load(t.template base<const T>(a.x), a.x.st, t.at, t.n, 0u);
        float P[V], H[V], R[V], rate[V];
        float alpha[S][V];
        float z[S][V];                     // sigmoid(b) and its complement; without b 1 - alpha
        float before[S][V];                // the states before the tokens
        float first[V];                    // the state at the tile's start
        const int64_t i = t.b * a.C + t.c0 + t.at, at = (t.b * chunks + t.j) * a.C + t.c0 + t.at;
        const int in_group = GROUP ? (int)(draw.along % kGroup) : 0;
        float* edge = behind + at + in_group * (int64_t)a.C;
        Passed<V> passed;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.0f;
            H[v] = 0.0f;
            R[v] = 0.0f;
            rate[v] = RATE ? a.rate[t.c0 + t.at + v] : 1.0f;
            first[v] = starts ? starts[at + v] : (a.state0 ? state_at(a.state0, a.state_dtype, i + v) : 0.0f);
        }
        const bool grows = RATE && any_below_0<V>(rate);
        // The gates of a first, those of b and the states after them, so that b and x arrive meanwhile; four tokens at a time, since
        // more at once take registers (as one loop 340 us; in two loops without the barriers 336; so 333).
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (s % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                const Decay d = decay_of<EXACT, RATE>(ga.r[s].get(v), rate[v], rates != nullptr);
                alpha[s][v] = d.alpha;
                aside[s * V + v][threadIdx.x] = make_float2(d.up, d.soft);
                if (COUPLED) z[s][v] = d.lost;
                P[v] = d.of(P[v]);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s == S / 2 && t.j + 1 < chunks && wave == 0) {
                __builtin_amdgcn_sched_barrier(0);
                passed.look(edge);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (s % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                if (!COUPLED) z[s][v] = smaller_sigmoid<EXACT>(gb.r[s].get(v));
                const float beta = COUPLED ? z[s][v] : sigmoid_of(z[s][v]);
                H[v] = fmaf(alpha[s][v], H[v], beta * x.r[s].get(v));
            }
        }
#pragma unroll
        for (int s = S - 1; s >= 0; --s)
#pragma unroll
            for (int v = 0; v < V; ++v) R[v] = alpha[s][v] * (go.r[s].get(v) + R[v]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            maps[wave][3 * v][lane] = P[v];
            maps[wave][3 * v + 1][lane] = H[v];
            maps[wave][3 * v + 2][lane] = R[v];
        }
        __syncthreads();
        if (wave == 0) {  // the tile's map, the adjoint behind it, the one behind the tile before
            float r[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                P[v] = 1.0f;
                R[v] = 0.0f;
                for (int w = W - 1; w >= 0; --w) {
                    const float q = maps[w][3 * v][lane];
                    P[v] *= q;
                    R[v] = fmaf(q, R[v], maps[w][3 * v + 2][lane]);
                }
            }
            const int64_t half = a.B * chunks * a.C;
            unsigned pass = t.on ? (1u << V) - 1 : 0;  // bit v: the channel has a map to pass on
            bool walked = false;                       // not all have
            if (__builtin_expect(grows, 0)) {
#pragma unroll
                for (int v = 0; v < V; ++v) pass &= P[v] <= kMost ? ~0u : ~(1u << v);
                walked = __any(t.on && pass + 1 != 1u << V);
                if (lane == 0) walks = walked;
                if (walked) walk_of[lane] = t.on ? ~pass : 0;
            }
            if (GROUP && in_group < kGroup - 1 && t.j > 0 && t.on) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (!walked || (pass >> v & 1)) {
                        publish(ends + at + v, P[v]);
                        publish(ends + half + at + v, R[v]);
                    }
            }
            if (t.j + 1 < chunks) {
                if constexpr (GROUP) {
                    float bp[V], bu[V];
                    Passed<V>::maps_before(ends + at + a.C, -(int64_t)a.C, half, in_group, bp, bu);
                    const bool past = grows && any_past<V>(bp);
                    passed.get(edge, r);
                    if (__builtin_expect(past, 0)) Passed<V>::one_by_one(ends + at + a.C, -(int64_t)a.C, half, in_group, r, bp, bu);
#pragma unroll
                    for (int v = 0; v < V; ++v) r[v] = fmaf(bp[v], r[v], bu[v]);
                } else {
                    passed.get(edge, r);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) r[v] = a.dstate ? state_at(a.dstate, a.state_dtype, i + v) : 0.0f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float end = fmaf(P[v], r[v], R[v]);
                if (t.on) {
                    if (!walked || (pass >> v & 1)) {
                        if (t.j == 0) {
                            if (a.dstate0) set_state(a.dstate0, a.state_dtype, i + v, end);
                        } else if (!GROUP || in_group == kGroup - 1) {
                            publish(behind + at - a.C + v, end);
                        }
                    }
                    if (GROUP && t.j + 1 == chunks && t.j > 0) publish(behind + at + v, r[v]);
                }
                after[v][lane] = r[v];
            }
        }
        float total[V], r[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float h = first[v];
            for (int w = 0; w < wave; ++w) h = fmaf(maps[w][3 * v][lane], h, maps[w][3 * v + 1][lane]);
            total[v] = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                before[s][v] = h;
                h = fmaf(alpha[s][v], h, (COUPLED ? z[s][v] : sigmoid_of(z[s][v])) * x.r[s].get(v));
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            r[v] = after[v][lane];
            for (int w = W - 1; w > wave; --w) r[v] = fmaf(maps[w][3 * v][lane], r[v], maps[w][3 * v + 2][lane]);
        }
        // Each row's gradients are stored as they come, from the last to the first; without conditions where the segment is
        // whole, so that rows overlap.
        const auto finish = [&](auto whole) {
            unsigned off = t.at * (unsigned)sizeof(T);
            RowAt rx(t.template base<T>(a.dx), a.dx.st), ra(t.template base<T>(a.da), a.da.st), rb(t.template base<T>(a.db), a.db.st);
            rx.p += (S - 1) * rx.step;
            ra.p += (S - 1) * ra.step;
            rb.p += (S - 1) * rb.step;
#pragma unroll
            for (int s = S - 1; s >= 0; --s, rx.p -= rx.step, ra.p -= ra.step, rb.p -= rb.step) {
                float ox[V], oa[V], ob[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float xv = x.r[s].get(v), g = go.r[s].get(v) + r[v];
                    r[v] = alpha[s][v] * g;
                    const float e = r[v] * (COUPLED ? xv - before[s][v] : -before[s][v]);
                    const float2 kept = aside[s * V + v][threadIdx.x];
                    oa[v] = e * kept.x * rate[v];
                    ox[v] = g * (COUPLED ? z[s][v] : sigmoid_of(z[s][v]));
                    if (!COUPLED) ob[v] = g * xv * sigmoid_slope_of(z[s][v]);
                    if (whole || s < t.n) total[v] = fmaf(e, kept.y, total[v]);
                }
                Run<T, V> qx, qa, qb;
                qx.set(ox);
                qa.set(oa);
                if (!COUPLED) qb.set(ob);
                if (!whole && s >= t.n) {
                    qx.zero();
                    qa.zero();
                    qb.zero();
                }
                if (whole || s < t.rows) {
                    qx.store(rx.at<T>(off));
                    qa.store(ra.at<T>(off));
                    if (!COUPLED) qb.store(rb.at<T>(off));
                }
            }
        };
        if (t.on) {
            if (t.n == S) finish(std::true_type{}); else finish(std::false_type{});
        }
        if (rates) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v) maps[wave][v][lane] = total[v];
            __syncthreads();
            if (wave == 0 && t.on)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float sum = 0.0f;
                    for (int w = 0; w < W; ++w) sum += maps[w][v][lane];
                    rates[at + v] = sum * kLn2;  // softplus came in units of ln 2
                }
        }
        // As in the forward pass: channels whose product of decays passes fp32's range.
        if (__builtin_expect(grows && __builtin_amdgcn_readfirstlane((int)walks), 0)) {
            __syncthreads();
            if (wave == 0) {
                static_assert(sizeof(aside) >= V * sizeof(float) * 64 * kScanChunk, "the states of a tile");
                walk_backward<T, V, GROUP, COUPLED>(again(draw.chain), again(draw.along), walk_of[lane], after, (float*)aside);
            }
        }
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

// Workgroups of a launch: as many as run at once, four a CU, where they draw tickets (4096 instead took 2 % longer in the
// backward pass of 4 x 4096 tokens of 6144 channels), several times as many where they share the tiles out.
constexpr int64_t kTurns = 1024, kShares = 4096;

// The call's tiles (less than 2^31: the caller has checked it for tiles of 64 tokens and channels).
template <int V>
Tickets tickets_of(const ScanArgs& a, int tokens, unsigned* counters) {
    Tickets t;
    t.chains = (unsigned)(a.B * (((int64_t)a.C + 64 * V - 1) / (64 * V)));
    t.groups = t.chains < kGroups ? t.chains : kGroups;
    t.along = ((unsigned)a.T + tokens - 1) / tokens;
    t.counters = t.along > 1 ? counters : nullptr;
    return t;
}
// Whether the chains are so few, fewer than `limit`, that passing states on from tile to tile, not moving the data, would
// bound the call. All bf16 with b, in us, tile by tile and in groups. Forward, chains of 128 channels: 4 chains of 65536 tokens
// 675 and 102, 16 chains 757 and 263, 48 of 16384 277 and 192, 96 of 4096 108 and 103, 192 of 4096 178 and 184.
// Backward, chains of 64: 8 of 65536 471 and 160, 32 681 and 537, 64 of 1024 25.4 and 25.6, 96 of 4096 94 and 104, 384 329 and 383.
// Short prompts have few steps: 16 chains of 256 tokens 11.4 and 13.2.
template <int V>
bool few_chains(const ScanArgs& a, int limit) {
    return scan_chunks(a.T) > kGroup && a.B * (((int64_t)a.C + 64 * V - 1) / (64 * V)) < limit;
}
int64_t blocks_of(const Tickets& t) {
    const int64_t n = (int64_t)t.chains * t.along, most = t.counters ? kTurns : kShares;  // (at least one for every group)
    return n < most ? n : most;
}

hipError_t clear(float* edges, int64_t n, float* maps, int64_t m, unsigned* counters, hipStream_t s) {
    uint32_t *p = (uint32_t*)edges, *q = (uint32_t*)maps;
    void* args[] = {&p, &n, &q, &m, &counters};
    const int64_t blocks = ((n > m ? n : m) / 4 + 255) / 256;
    return launch((const void*)gdn_scan_clear_kernel, blocks < 2048 ? blocks : 2048, 256, s, args);
}

// The workspace: counters of both directions; the edges' values, the adjoints first; the tiles' maps of both directions;
// the rates' gradient of every chunk.
unsigned* counters_of(const ScanArgs& a, int direction) { return (unsigned*)a.ws + direction * kGroups * kScanCounterStride; }
float* values_of(const ScanArgs& a) { return a.ws + kScanCounterFloats; }

// What a forward pass over the chunks has besides its arguments. `cleared`: its edges, maps and counters are.
struct Pass {
    float *starts, *maps;
    unsigned* counters;
    bool cleared;
};

template <typename T, int V, int W, bool GROUP, bool COUPLED, bool RATE, bool OUT>
hipError_t forward_w(const ScanArgs& a, Pass pass, hipStream_t s) {
    const Tickets tickets = tickets_of<V>(a, 16 * W, pass.counters);
    TileArgs args{a, tickets, pass.starts, nullptr, nullptr, pass.maps};
    if (tickets.counters && !pass.cleared) {
        hipError_t e = clear(pass.starts, a.B * scan_chunks(a.T) * a.C, pass.maps, GROUP ? 2 * a.B * tickets.along * a.C : 0,
                             pass.counters, s);
        if (e != hipSuccess) return e;
    }
    void* p[] = {&args};
    return launch((const void*)gdn_scan_forward_kernel<T, V, W, GROUP, COUPLED, RATE, OUT>, blocks_of(tickets), 64 * W, s, p);
}

constexpr int kFewForward = 128, kFewBackward = 48;

template <typename T, int V, bool COUPLED, bool RATE, bool OUT>
hipError_t forward(const ScanArgs& a, const Pass& pass, hipStream_t s) {
    if (few_chains<V>(a, kFewForward)) return forward_w<T, V, 8, true, COUPLED, RATE, OUT>(a, pass, s);
    return forward_w<T, V, 4, false, COUPLED, RATE, OUT>(a, pass, s);
}

template <typename T, int V, bool COUPLED, bool RATE>
hipError_t prefill(const ScanArgs& a, hipStream_t s) {
    float* between = scan_chunks(a.T) > 1 ? values_of(a) : nullptr;
    const Pass pass{a.checkpoints ? a.checkpoints : between, between ? between + scan_values(a.B, a.T, a.C) : nullptr,
                    counters_of(a, 0), false};
    return forward<T, V, COUPLED, RATE, true>(a, pass, s);
}

template <typename T, int V, bool COUPLED, bool RATE>
hipError_t backward(const ScanArgs& a, hipStream_t s) {
    const int64_t chunks = scan_chunks(a.T), n = a.B * chunks * a.C, stride = (int64_t)scan_values(a.B, a.T, a.C);
    float* starts = a.checkpoints;
    float *behind = values_of(a), *made = behind + stride, *ends = made + stride, *made_maps = ends + 2 * stride;
    float* rates = a.drate ? made_maps + 2 * stride : nullptr;
    const bool make = !starts && chunks > 1, few = few_chains<V>(a, kFewBackward);
    const Tickets tickets = tickets_of<V>(a, kScanChunk, counters_of(a, 0));
    hipError_t e = hipSuccess;
    if (tickets.counters) {  // both passes' at once
        const bool maps = few || (make && few_chains<V>(a, kFewForward));
        e = clear(behind, make ? stride + n : n, ends, maps ? 4 * stride : 0, tickets.counters, s);
        if (e != hipSuccess) return e;
    }
    if (make) {
        ScanArgs f = a;
        f.state = const_cast<void*>(a.state0);
        e = forward<T, V, COUPLED, RATE, false>(f, Pass{made, made_maps, counters_of(a, 1), true}, s);
        if (e != hipSuccess) return e;
        starts = made;
    }
    TileArgs args{a, tickets, starts, behind, rates, ends};
    void* p[] = {&args};
    e = launch(few ? (const void*)gdn_scan_backward_kernel<T, V, true, COUPLED, RATE>
                   : (const void*)gdn_scan_backward_kernel<T, V, false, COUPLED, RATE>,
               blocks_of(tickets), 256, s, p);
    if (e != hipSuccess || !rates) return e;
    const float* in = rates;
    int64_t rows = a.B * chunks;
    int C = a.C;
    float* out = a.drate;
    void* p2[] = {&in, &rows, &C, &out};
    return launch((const void*)gdn_scan_rates_kernel, ((int64_t)C + 63) / 64, 1024, s, p2);
}

// f.template run<T, V, COUPLED, RATE>() for the call's type, vector width (f.wide values, 2 or 1) and gates.
template <typename T, int V, typename F>
hipError_t by_gates(const ScanArgs& a, F f) {
    if (a.b.p) return a.rate ? f.template run<T, V, false, true>() : f.template run<T, V, false, false>();
    return a.rate ? f.template run<T, V, true, true>() : f.template run<T, V, true, false>();
}
template <typename T, typename F>
hipError_t by_width(const ScanArgs& a, F f) {
    constexpr int WIDE = F::template wide<T>();
    if constexpr (WIDE > 2) {
        if (vector_fits(a, WIDE)) return by_gates<T, WIDE>(a, f);
    }
    if constexpr (WIDE > 1) {
        if (vector_fits(a, 2)) return by_gates<T, 2>(a, f);
    }
    return by_gates<T, 1>(a, f);
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
    template <typename T> static constexpr int wide() { return 2; }  // (256 x 6144 bf16: 13.2 us with 8, 9.0 with 4, 7.9 with 2, 9.1 with 1)
    const ScanArgs& a;
    hipStream_t s;
    template <typename T, int V, bool COUPLED, bool RATE>
    hipError_t run() { return decode<T, V, COUPLED, RATE>(a, s); }
};
struct PrefillRun {
    template <typename T> static constexpr int wide() { return 2; }
    const ScanArgs& a;
    hipStream_t s;
    template <typename T, int V, bool COUPLED, bool RATE>
    hipError_t run() { return prefill<T, V, COUPLED, RATE>(a, s); }
};
struct BackwardRun {
    template <typename T> static constexpr int wide() { return 1; }
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
