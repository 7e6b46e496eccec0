// nvq_decode.hip -- a whole mixture-of-experts layer for a few tokens (up to
// 64, single tokens being decoded): router, chosen experts and weighted combine
// on bf16, int8 or NVFP4 weights, in two launches.
//
//   k_decode_router   logits = x Wr^T
//   k_decode_layer    ids, weights = top-k of the logits;
//                     h = silu(g) * u of every (expert, token) pair;
//                     out = residual + sum_s weight * (W2 h)
//
// Bound by reading the chosen experts' weights once. The activations are not
// quantized: they are a few rows, and it would save nothing. A weight reaches
// the matrix pipe as a 16-bit value that holds it exactly (int8 codes have 8
// significant bits: bf16; e2m1 * e4m3 has 6 and lies in [2^-10, 2688]: fp16);
// the channel's or tensor's fp32 scale is applied to the fp32 sum.
//
// The other operand. bf16 and int8 weights: x as it is, and h as two bf16 parts,
// its rounding and the rounding of what that left (2^-17 of it in all; one part
// would be 2^-9, as much as out's own rounding), which costs only products and
// these are far from the limit. NVFP4 weights: x in fp16 times a power of two
// per token that takes its largest value to [2^14, 2^15), which holds its 8 bits
// down to 2^-29 of that and is off by at most 2^-40 of it below; and h rounded to
// fp16 once (2^-12 of it), times a power of two that no h of the token and expert
// can exceed, from the 1-norm of x and the expert's largest possible weight.
#include "nvq_argmax.hpp"
#include "nvq_device.hpp"
#include "nvq_host.hpp"

#include <algorithm>
#include <type_traits>

namespace nvq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum { kBf16 = 0, kInt8 = 1, kNvfp4 = 2 };

constexpr int kMaxT = 64;       // tokens: an expert's are one 64-bit mask
constexpr int kMaxE = 1024;
constexpr int kMaxK = 64;
constexpr int kMaxA = kMaxT * kMaxK;
constexpr int kMaxV = kMaxE + kMaxA / 16;  // blocks of at most 16 tokens of one expert
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr uint32_t kNowhere = 0xFFFFFFE0u;
constexpr int kAgentScope = 16;  // buffer loads: the sc1 bit, as an agent-scope atomic load has it
constexpr int64_t kMaxBytes = 0xFFFFFE00ll;

// Device-wide counters of one call, cleared by k_decode_router.
struct Counters {
    uint32_t pick, picked;  // tasks of the choice taken, finished
    uint32_t fc1, tail;     // shares of fc1 taken, tasks taken of its tail
    uint32_t fc2;           // shares of fc2 taken
    uint32_t done;          // tasks of fc1 finished
    uint32_t pad[26];
    uint32_t block[64];     // the same of each block of tokens, where there are few
};
// x of a token for NVFP4 weights is its fp16 values times 2^shift; the sum of these values' magnitudes is below 2^norm.
struct TokenScale {
    int32_t shift, norm;
};

struct Args {
    const uint16_t* x;
    const uint16_t* wr;
    const float* bias;
    const void *w1, *w2;
    const void *s1, *s2;      // int8: fp32 per row; NVFP4: E4M3 bytes per 16 values
    const float *t1, *t2;     // NVFP4: per matrix
    const uint16_t* residual;
    uint16_t* out;
    int32_t* ids;
    float* weights;
    double* logits;           // [parts, T, E]: sums over parts of K
    uint16_t* h;              // [T k, f], rows in expert order; bf16: each eight values' high, then low parts
    uint16_t* xh;             // NVFP4: [T, d] fp16 (both in the order of half_slot)
    TokenScale* xs;
    Counters* count;
    int T, d, E, k, f, sigmoid, parts, max_blocks;
};

// A value that all lanes of a wave hold, as a scalar: branches on it are the wave's, not a lane's. Every loop here that
// holds a barrier ends on such a value.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// ------------------------------------------------------------------ the formats
// One step of a wave is 64 bytes of each of 16 weight rows: lane l holds 16 bytes of row l % 16, those at 16 (l / 16) of
// the step, kVals values and their products' other operand, the same K of token l % 16.
template <int FMT>
struct Fmt {
    static constexpr int kVals = FMT == kBf16 ? 8 : FMT == kInt8 ? 16 : 32;  // in 16 bytes
    static constexpr int kFrags = kVals / 8;
    static constexpr int NB = FMT == kBf16 ? 1 : 2;         // fc1: groups of 16 weight rows of a wave
    static constexpr int D1 = FMT == kBf16 ? 8 : 4;         // steps in flight in fc1
    static constexpr int kParts = FMT == kNvfp4 ? 1 : 2;    // 16-bit parts of h
    static __host__ __device__ __forceinline__ uint32_t row_bytes(int K) { return (uint32_t)(K / kVals) * 16u; }
};

struct W16 {
    u32x4 w;
    uint32_t sc;   // NVFP4: the two scale bytes
};
template <int FMT>
struct X16 {
    u32x4 v[Fmt<FMT>::kFrags];
};

// Slot of value j of eight in the fp16 operands: the pairs in which NVFP4 codes are decoded, (0 2) (4 6) (1 3) (5 7).
__host__ __device__ constexpr int half_slot(int j) { return (j & 1) * 4 + (j >> 1); }

// Eight E2M1 codes times an E4M3 scale in fp16, exact, in the order of half_slot. The upper byte of an E2M1 value's fp16
// holds all of it: a byte permute looks up four magnitudes at a time, a bit select adds the signs, four more permutes
// spread the bytes over halves. 16 full-rate operations for 8 values; four conversions and products (the converter runs
// at a quarter of the rate) would take as long as 20, fp32 conversions as 28.
__device__ __forceinline__ u32x4 decode_fp4(uint32_t w, half2v scale) {
    constexpr uint32_t kLo = 0x3E3C3800u, kHi = 0x46444240u;  // 0 .5 1 1.5, 2 3 4 6
    const uint32_t even = __builtin_amdgcn_perm(kHi, kLo, w & 0x07070707u);
    const uint32_t odd = __builtin_amdgcn_perm(kHi, kLo, (w >> 4) & 0x07070707u);
    const uint32_t e = (even & 0x7F7F7F7Fu) | ((w << 4) & 0x80808080u), o = (odd & 0x7F7F7F7Fu) | (w & 0x80808080u);
    auto put = [&](uint32_t bytes, uint32_t sel) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0u, bytes, sel)) * scale);
    };
    return (u32x4){put(e, 0x010C000Cu), put(e, 0x030C020Cu), put(o, 0x010C000Cu), put(o, 0x030C020Cu)};
}

// Fragment i (8 values) of 16 bytes of weights, in bf16 or (NVFP4) fp16.
template <int FMT>
__device__ __forceinline__ u32x4 decode(const W16& w, int i) {
    if constexpr (FMT == kBf16) {
        return w.w;
    } else if constexpr (FMT == kInt8) {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t p = w.w[2 * i + (j >> 1)] >> (16 * (j & 1));
            const float a = (float)(int8_t)(p & 0xFFu), b = (float)(int8_t)((p >> 8) & 0xFFu);
            o[j] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);  // exact: the upper halves
        }
        return o;
    } else {
        const half2v s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.sc, 1.0f, false);
        return decode_fp4(w.w[i], half2v{s[i >> 1], s[i >> 1]});
    }
}
template <int FMT>
__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 acc) {
    if constexpr (FMT == kNvfp4)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, w), __builtin_bit_cast(half8, x), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0,
                                                       0, 0);
}

// The matrices of one expert: `rows` rows of K values.
template <int FMT>
struct Matrix {
    __amdgpu_buffer_rsrc_t w, s;
    uint32_t rb;
    __device__ __forceinline__ Matrix(const void* base, const void* scales, int e, int rows, int K) {
        rb = Fmt<FMT>::row_bytes(K);
        const uint32_t bytes = (uint32_t)rows * rb;
        w = rsrc(static_cast<const uint8_t*>(base) + (int64_t)e * bytes, bytes);
        if (FMT == kNvfp4) s = rsrc(static_cast<const uint8_t*>(scales) + (int64_t)e * (bytes / 8), bytes / 8);
    }
    // 16 bytes at byte `o` of row `row` (nothing is read where !ok)
    __device__ __forceinline__ W16 load(uint32_t row, uint32_t o, bool ok) const {
        W16 r;
        const uint32_t at = ok ? row * rb + o : kNowhere;
        r.w = __builtin_amdgcn_raw_buffer_load_b128(w, at, 0, 2);  // read once: past the caches
        r.sc = FMT == kNvfp4 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(s, ok ? at / 8 : kNowhere, 0, 0) : 0;
        return r;
    }
};
template <int FMT>
__device__ __forceinline__ X16<FMT> load_x(__amdgpu_buffer_rsrc_t x, uint32_t row, int K, uint32_t o, bool ok) {
    X16<FMT> r;
#pragma unroll
    for (int i = 0; i < Fmt<FMT>::kFrags; ++i)
        r.v[i] = __builtin_amdgcn_raw_buffer_load_b128(
            x, ok ? row * (uint32_t)K * 2u + (o / 16 * Fmt<FMT>::kVals + 8 * i) * 2u : kNowhere, 0, 0);
    return r;
}

// A barrier that orders LDS only: loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------------ router logits
// One workgroup: 16 experts, 16 tokens, a part of K, shared by its four waves. The sum of 32 products that one
// instruction adds is rounded to fp32, 2^-24 of it; from there on the sums are fp64, so that of two close logits the
// larger one is chosen. K is cut so that a token's logits are some 200 workgroups: with one per 16 experts (24 of 384)
// the launch took 6.6 us.
constexpr int kRouterWaves = 4, kRouterThreads = 64 * kRouterWaves;

// x of token t in fp16 for NVFP4 weights (one workgroup).
__device__ __forceinline__ void scale_token(const Args& p, int t) {
    __shared__ uint32_t tops[kRouterWaves];
    __shared__ float sums[kRouterWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, units = p.d / 8;
    const u32x4* src = reinterpret_cast<const u32x4*>(p.x + (int64_t)t * p.d);
    u32x4* dst = reinterpret_cast<u32x4*>(p.xh + (int64_t)t * p.d);
    uint32_t m = 0;
#pragma unroll 2
    for (int u = threadIdx.x; u < units; u += kRouterThreads) {
        const u32x4 v = src[u];
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    }
    m = wave_max_u32(m);
    if (lane == 0) tops[wave] = m;
    __syncthreads();
    m = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    // a row without a largest finite value keeps its size: what it holds becomes infinities and NaN
    const int shift = m && m < 0x7F80u ? __builtin_amdgcn_frexp_expf(bf16_to_f32(m)) - 15 : 0;
    float sum = 0.0f;
#pragma unroll 2
    for (int u = threadIdx.x; u < units; u += kRouterThreads) {
        const u32x4 v = src[u];
        half8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = v[j >> 1];
            const float f = __builtin_amdgcn_ldexpf(__uint_as_float((j & 1) ? b & 0xFFFF0000u : b << 16), -shift);
            sum += fabsf(f);
            o[half_slot(j)] = (_Float16)f;
        }
        dst[u] = __builtin_bit_cast(u32x4, o);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        p.xs[t] = {shift, __builtin_amdgcn_frexp_expf(sum)};
    }
}

template <bool HALF>
__global__ __launch_bounds__(kRouterThreads) void k_decode_router(Args p) {
    __shared__ double red[kRouterWaves][16][17];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (blockIdx.x == 0 && threadIdx.x < sizeof(Counters) / 4) reinterpret_cast<uint32_t*>(p.count)[threadIdx.x] = 0;
    int b = blockIdx.x;
    if (HALF) {
        if (b < p.T) return scale_token(p, b);
        b -= p.T;
    }
    const int eb = (p.E + 15) / 16, tb = (p.T + 15) / 16;
    const int e0 = b % eb * 16, t0 = b / eb % tb * 16, z = b / (eb * tb);
    const uint32_t rb = (uint32_t)p.d * 2u;
    const auto wr = rsrc(p.wr, (uint32_t)p.E * rb), xr = rsrc(p.x, (uint32_t)p.T * rb);
    const int steps = (p.d + 31) / 32, waves = p.parts * kRouterWaves, part = (steps + waves - 1) / waves;
    const int first = (z * kRouterWaves + wave) * part, s1 = min(first + part, steps);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int s0 = first; s0 < s1; s0 += 4) {
        u32x4 w[4], x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t o = (uint32_t)(s0 + j) * 64 + q * 16;
            const bool ok = s0 + j < s1 && o < rb;
            w[j] = __builtin_amdgcn_raw_buffer_load_b128(wr, ok && e0 + r < p.E ? (e0 + r) * rb + o : kNowhere, 0, 0);
            x[j] = __builtin_amdgcn_raw_buffer_load_b128(xr, ok && t0 + r < p.T ? (t0 + r) * rb + o : kNowhere, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x4 a = mfma<kBf16>(w[j], x[j], (f32x4){0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += (double)a[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r][4 * q + i] = acc[i];
    __syncthreads();
    const int e = threadIdx.x & 15, t = threadIdx.x >> 4;
    double v = red[0][t][e];
#pragma unroll
    for (int w = 1; w < kRouterWaves; ++w) v += red[w][t][e];
    if (e0 + e < p.E && t0 + t < p.T) p.logits[((int64_t)z * p.T + t0 + t) * p.E + e0 + e] = v;
}

// ------------------------------------------------------------------ the choice
// Largest value over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    v = max(v, dpp_u32<0x140>(v));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// Logits (sigmoid: scores) of tokens t0 .. t0 + n - 1 into LDS, val[token - t0], by all threads: a thread adds the parts of
// one logit, all loaded at once.
constexpr int kMaxParts = 8;
__device__ __forceinline__ void add_parts(const Args& p, int t0, int n, double (*val)[kMaxE]) {
#pragma unroll 1
    for (int i = threadIdx.x; i < n * p.E; i += kThreads) {
        const int t = i / p.E, e = i - t * p.E;
        const double* src = p.logits + (int64_t)(t0 + t) * p.E + e;
        const int64_t step = (int64_t)p.T * p.E;
        double v[kMaxParts], l = 0.0;
#pragma unroll
        for (int z = 0; z < kMaxParts; ++z) v[z] = src[min(z, p.parts - 1) * step];
#pragma unroll
        for (int z = 0; z < kMaxParts; ++z) l += z < p.parts ? v[z] : 0.0;
        val[t][e] = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : l;
    }
}

// Ids and weights of a token by one wave, as the routers choose from val: lane j < k returns the j-th. P: expert slots per
// lane. A round compares the upper halves of the lanes' best keys; only where two lanes tie there does it compare whole
// keys. Non-finite logits order somehow; the ids stay distinct and in range.
template <int P>
__device__ __forceinline__ void choose(const Args& p, const double* val, const float* bias, int lane, int* id, float* weight) {
    uint64_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int e = lane + 64 * j;
        key[j] = 0;  // below the key of every number
        if (e < p.E) {
            const double v = val[e] + (double)bias[e];
            key[j] = order_key(v == v ? v : -__builtin_inf());
        }
    }
    uint64_t best = 0;
    int slot = 0;
    auto rank = [&]() {  // the lane's best: strictly greater, so the lowest slot among equal keys stays
        best = 0;
        slot = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const bool gt = key[j] > best;
            best = gt ? key[j] : best;
            slot = gt ? j : slot;
        }
    };
    rank();
    int mine = 0;
    for (int r = 0; r < p.k; ++r) {
        const uint32_t top = wave_max((uint32_t)(best >> 32));
        const uint64_t at = __ballot((uint32_t)(best >> 32) == top);
        int win;
        if ((at & (at - 1)) == 0) {
            const int owner = __builtin_ctzll(at);
            win = owner + 64 * __builtin_amdgcn_readlane(slot, owner);
        } else {
            uint64_t bk = best;
            win = best ? lane + 64 * slot : 0x7FFFFFFF;
            group_argmax<64>(bk, win);
            win = __builtin_amdgcn_readfirstlane(win);
        }
        const int ws = win / 64;
        const bool owner = lane == (win & 63);
#pragma unroll
        for (int j = 0; j < P; ++j) key[j] = owner && j == ws ? 0 : key[j];
        rank();
        mine = lane == r ? win : mine;
    }
    double v = lane < p.k ? val[mine] : 0.0;  // the chosen logits, or scores
    if (!p.sigmoid) {
        double m = read_lane(v, 0);
        for (int j = 1; j < p.k; ++j) m = fmax(m, read_lane(v, j));
        v = exp(v - m);
    }
    double sum = 0.0;  // in the order of the choice
    for (int j = 0; j < p.k; ++j) sum += read_lane(v, j);
    *id = mine;
    *weight = (float)(v / sum);
}

// The chosen experts and their tokens, in LDS of every workgroup: blocks of at most 16 tokens of one expert, in
// ascending expert order; row row0 + i of h, tok and wt is token i of the block.
struct Block {
    int16_t e;
    int16_t row0;
    int32_t n;
};
struct Table {
    uint64_t mask[kMaxE];  // tokens of each expert
    int32_t base[kMaxE];   // its first row
    Block blocks[kMaxV];
    float wt[kMaxA];       // routing weight; NVFP4: times w2's tensor scale
    uint8_t tok[kMaxA];
    int32_t scan[kWaves];
};
// NVFP4, per row: g and u are the sums times t1 times 2^shift; h is its fp16 value times 2^exp.
struct RowScale {
    float t1;
    int16_t shift, exp;
};
// From ids and weights (global, as another launch or `choose` of this workgroup left them). All threads take part;
// returns the number of blocks.
template <int FMT>
__device__ __forceinline__ int build(Table& tb, RowScale* rows, const Args& p, const int32_t* ids, const float* weights) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int A = p.T * p.k;
    struct Scales {
        float t1, t2;
        TokenScale x;
    };
    auto scales = [&](int a) { return Scales{p.t1[ids[a]], p.t2[ids[a]], p.xs[a / p.k]}; };
    Scales early = {};  // of row t, on their way while the table is made
    if (FMT == kNvfp4 && t < A) early = scales(t);
    for (int e = t; e < p.E; e += kThreads) tb.mask[e] = 0;
    __syncthreads();
    for (int a = t; a < A; a += kThreads)
        atomicOr(reinterpret_cast<unsigned long long*>(&tb.mask[ids[a]]), 1ull << (a / p.k));
    __syncthreads();
    // prefix sums over the experts (two neighbouring ones per thread) of rows (low half) and blocks (high half)
    int n[2], sum = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = 2 * t + j;
        n[j] = e < p.E ? __popcll(tb.mask[e]) : 0;
        sum += n[j] | ((n[j] + 15) / 16) << 16;
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(incl, off, 64);
        incl += lane >= off ? v : 0;
    }
    if (lane == 63) tb.scan[wave] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int v = tb.scan[w];
        before += w < wave ? v : 0;
        total += v;
    }
    int at = before + incl - sum;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = 2 * t + j;
        if (e < p.E) {
            const int row = at & 0xFFFF, b = at >> 16;
            tb.base[e] = row;
            for (int i = 0; i * 16 < n[j]; ++i)
                tb.blocks[b + i] = {(int16_t)e, (int16_t)(row + 16 * i), min(16, n[j] - 16 * i)};
        }
        at += n[j] | ((n[j] + 15) / 16) << 16;
    }
    __syncthreads();
    for (int a = t; a < A; a += kThreads) {
        const int e = ids[a], tk = a / p.k;
        const int row = tb.base[e] + __popcll(tb.mask[e] & ((1ull << tk) - 1));
        tb.tok[row] = (uint8_t)tk;
        tb.wt[row] = weights[a];
        if (FMT == kNvfp4) {
            const Scales s = a == t ? early : scales(a);
            tb.wt[row] *= s.t2;
            // |g|, |u| < 2^(norm + shift) times the largest weight, 2688 t1, so |h| is below the square of that: 2^exp
            // times at most 2^15
            const int b = s.x.norm + s.x.shift + __builtin_amdgcn_frexp_expf(s.t1 * 2688.0f);
            rows[row] = {s.t1, (int16_t)s.x.shift, (int16_t)(2 * b - 15)};
        }
    }
    __syncthreads();
    return (int)uniform((uint32_t)total) >> 16;
}

// ------------------------------------------------------------------ the layer
// Work is cut into tasks, and these into as many shares as there are workgroups: share i of G is tasks i, i + G, ... A
// workgroup takes the next share from a device-wide counter, and another one when it is done. It waits only for tasks that
// running workgroups hold, so a call ends however few of its workgroups are resident at a time (another call's may hold the
// rest of the chip, and wait as well); where all are, each has one share.
//
//   choice   more than 8 tokens: 8 tokens a task, one per wave (up to 8 tokens every workgroup chooses for itself,
//            which costs it less than waiting)
//   fc1      one block of tokens and 8 NB gate rows with their up rows; the waves share K
//   fc2      16 columns of out; the waves share the (block, K step) pairs of all chosen experts in contiguous runs, and
//            where a run leaves a block its wave adds weight * sum to its own token rows in LDS
//
// Which workgroup does a task does not show in its result, and every sum has a fixed order.
constexpr int kOwnChoice = kWaves;

// By one thread. (The offset that the compiler cannot see through keeps it from first adding up over the wave, which
// would wait for the result, and with it for every load in flight, on the spot.)
__device__ __forceinline__ uint32_t take(uint32_t* counter) {
    uint32_t zero = 0;
    asm volatile("" : "+v"(zero));
    counter += zero;
    return __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// All threads: everything this workgroup stored becomes visible to workgroups that see `counter` counted up by n.
__device__ __forceinline__ void publish(uint32_t* counter, uint32_t n) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        __hip_atomic_fetch_add(counter, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}
// All threads: waits until `counter` has reached n; what was published before it did is visible then.
__device__ __forceinline__ void await(uint32_t* counter, uint32_t n) {
    if (threadIdx.x == 0) {
        while (__hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < n) __builtin_amdgcn_s_sleep(1);
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    }
    __syncthreads();
}

// fc1 -> fc2. h is written through to memory (agent-scope stores), so that a workgroup has nothing to flush before it
// counts a task as finished: a release fence writes the XCD's whole L2 back, 1 to 4 us.
//
// FEW (at most kFewRows rows of h): fc2 waits block by block, so that the first experts' W2 is read while the last
// workgroups are still busy with fc1 (they end some 5 us after the median one), and reads h past the L2, so that no wave
// has to invalidate anything (2000 invalidations took 14 us). A task counts as finished a task later: the waves wait until
// no more of their memory operations are outstanding than the loads they have issued since, which costs nothing, and
// thread 0 counts after the barrier that follows. (One token on NVFP4 weights 46.7 us waiting for all of fc1, 43.8 so;
// three tokens of a small layer 26.3 and 23.1; one bf16 token the same; two bf16 tokens, 16 rows, 104 and 126.)
// Else one thread of a workgroup waits for all of fc1 and invalidates, and h is read through the L2, which serves it to 32
// CUs (64 int8 tokens: 627 us; past the L2, block by block, 800).
constexpr int kFewRows = 8;
__device__ __forceinline__ void store_through(uint16_t* p, uint32_t v) {
    __hip_atomic_store(reinterpret_cast<uint32_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void count_up(uint32_t* counter, uint32_t n) {
    __hip_atomic_fetch_add(counter, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// fc1's operands of a wave in flight: D1 steps.
template <int FMT>
struct Stage1 {
    W16 w[Fmt<FMT>::D1][Fmt<FMT>::NB];
    X16<FMT> x[Fmt<FMT>::D1];
};
struct Task1 {  // all scalars
    int block, e, n, row0, c0;
};

template <int FMT, int P, bool FEW>
__global__ __launch_bounds__(kThreads, 2) void k_decode_layer(Args p) {
    constexpr int NB = Fmt<FMT>::NB, D1 = Fmt<FMT>::D1, NF = Fmt<FMT>::kFrags, HP = Fmt<FMT>::kParts;
    constexpr int D2 = FMT == kNvfp4 && !FEW ? 6 : 8;  // steps in flight in fc2
    union Scratch {
        struct {
            float part[2][kWaves][NB][16][17];  // fc1: each wave's sums
            uint32_t told[2];                   // and a task
        };
        float rows[kWaves][kMaxT][17];      // fc2: each wave's token rows
        struct {
            int32_t ids[kOwnChoice * kMaxK];
            float weights[kOwnChoice * kMaxK];
            double val[kWaves][kMaxE];
        } c;                                // the choice
    };
    __shared__ Table tb;
    __shared__ Scratch sc;
    __shared__ uint32_t next;
    __shared__ float bias[kMaxE];
    __shared__ RowScale rows[FMT == kNvfp4 ? kMaxA : 1];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int G = gridDim.x;
    // Thread 0's shares of fc1 and fc2, asked for well before they are used: with the last task of the share before.
    uint32_t share1 = 0, share2 = 0;
    if (threadIdx.x == 0) share1 = take(&p.count->fc1);
    auto tell = [&](uint32_t share) {  // all threads: what thread 0 took (a barrier on either side)
        if (threadIdx.x == 0) next = share;
        __syncthreads();
        const uint32_t v = uniform(next);
        __syncthreads();
        return (int)v;
    };
    for (int e = threadIdx.x; e < p.E; e += kThreads) bias[e] = p.bias ? p.bias[e] : 0.0f;

    // ---- the choice
    auto choose_for = [&](int t0, int32_t* ids, float* weights) {  // tokens t0 .. t0 + 7, one per wave
        add_parts(p, t0, min(p.T - t0, kWaves), sc.c.val);
        __syncthreads();
        const int t = t0 + wave;
        if (t >= p.T) return;
        int id;
        float w;
        choose<P>(p, sc.c.val[wave], bias, lane, &id, &w);
        if (lane < p.k) {
            ids[t * p.k + lane] = id;
            weights[t * p.k + lane] = w;
        }
    };
    int V;
    if (p.T <= kOwnChoice) {
        choose_for(0, sc.c.ids, sc.c.weights);
        __syncthreads();
        if (blockIdx.x == 0)
            for (int a = threadIdx.x; a < p.T * p.k; a += kThreads) {
                p.ids[a] = sc.c.ids[a];
                p.weights[a] = sc.c.weights[a];
            }
        V = build<FMT>(tb, rows, p, sc.c.ids, sc.c.weights);
    } else {
        const uint32_t tasks = (uint32_t)(p.T + kWaves - 1) / kWaves;
        for (;;) {
            if (threadIdx.x == 0) next = take(&p.count->pick);
            __syncthreads();
            const uint32_t c = uniform(next);
            if (c >= tasks) break;
            choose_for((int)c * kWaves, p.ids, p.weights);
            publish(&p.count->picked, 1);
            // Nothing may come between thread 0's part of publish and its next take but this barrier: without it the
            // compiler makes one block of the two, and a loop around the rest that lane 0 leaves for that block while
            // the other lanes of its wave go round and wait for it there.
            __syncthreads();
        }
        await(&p.count->picked, tasks);
        V = build<FMT>(tb, rows, p, p.ids, p.weights);
    }

    // ---- fc1
    const int JB = (p.f + 8 * NB - 1) / (8 * NB), N1 = V * JB;
    const auto xr = rsrc(FMT == kNvfp4 ? p.xh : p.x, (uint32_t)p.T * (uint32_t)p.d * 2u);
    const uint32_t rb1 = Fmt<FMT>::row_bytes(p.d);
    const int steps1 = (int)(rb1 + 63) / 64, part1 = (steps1 + kWaves - 1) / kWaves;
    const int chunks = (part1 + D1 - 1) / D1, s_first = wave * part1, s_end = min(s_first + part1, steps1);
    auto set = [&](int task) {
        const int i = task / JB;
        const Block b = tb.blocks[i];
        return Task1{i, (int)uniform(b.e), (int)uniform(b.n), (int)uniform(b.row0), task % JB * 8 * NB};
    };
    auto fetch = [&](Stage1<FMT>& st, int j, const Task1& t, uint32_t xrow, int s) {
        const Matrix<FMT> m(p.w1, p.s1, t.e, 2 * p.f, p.d);
        const uint32_t o = (uint32_t)s * 64 + q * 16;
        const bool ok = s < s_end && o < rb1;
        const int col = t.c0 + (r & 7);
#pragma unroll
        for (int g = 0; g < NB; ++g)
            st.w[j][g] = m.load((r < 8 ? 0 : p.f) + col + 8 * g, o, ok && col + 8 * g < p.f);
        st.x[j] = load_x<FMT>(xr, xrow, p.d, o, ok && r < t.n);
    };
    auto token = [&](const Task1& t) { return (uint32_t)tb.tok[t.row0 + min(r, t.n - 1)]; };
    // The epilogue's thread: two columns of a token, neighbours as the operand of fc2 holds them.
    const int em = threadIdx.x / (4 * NB), eg = threadIdx.x / 4 % NB, ep = threadIdx.x & 3;
    const int ej = FMT == kNvfp4 ? (ep & 1) * 4 + (ep >> 1) : 2 * ep, ej2 = ej + (FMT == kNvfp4 ? 2 : 1);
    uint32_t finished = 0;  // tasks
    int pending = -1;       // FEW: block of the finished task that is not counted yet
    int flip = 0;
    bool asked = false;  // for a share of fc2
    // Where fc1 is long, shares are of the tasks before `tail`, whole rounds, and the rest is taken task by task, two ahead
    // of its use (64 tokens on NVFP4 weights: the last workgroup ends 6 us after the median one instead of 34).
    const int tail = N1 >= 24 * G ? (N1 / G - 4) * G : N1;
    for (int i = tell(share1); i < G; i = tell(share1)) {
        Stage1<FMT> st;
        int cur = i < tail ? i : N1, nxt = cur + G;
        if (cur >= N1) {
            if (threadIdx.x == 0) share1 = take(&p.count->fc1);
            continue;
        }
        Task1 t = set(cur);
        uint32_t xrow = token(t);
#pragma unroll
        for (int j = 0; j < D1; ++j) fetch(st, j, t, xrow, s_first + j);
        for (; cur < N1;) {
            const bool more = nxt < N1;
            // the task after the next one: of the share, or of the tail (thread 0 asks; told at this task's barrier)
            const bool ask = tail < N1 && nxt + G >= tail;
            uint32_t got = 0;
            if (threadIdx.x == 0) {
                if (ask) got = take(&p.count->tail);
                if (!more) share1 = take(&p.count->fc1);
                if (!more && !asked) share2 = take(&p.count->fc2);
            }
            asked |= !more;
            const Task1 tn = set(more ? nxt : cur);
            const uint32_t xnext = token(tn);
            float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f};  // int8: the epilogue's channel scales, ahead of the loads that follow
            if (FMT == kInt8 && wave < NB) {
                const float* s = static_cast<const float*>(p.s1) + (int64_t)t.e * 2 * p.f;
                const int c = min(t.c0 + 8 * eg + ej, p.f - 2);
                cs[0] = s[c];
                cs[1] = s[c + 1];
                cs[2] = s[p.f + c];
                cs[3] = s[p.f + c + 1];
            }
            f32x4 acc[NB];
#pragma unroll
            for (int g = 0; g < NB; ++g) acc[g] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            for (int c = 0; c < chunks; ++c) {
                const bool last = c + 1 == chunks;
                const Task1 tl = last ? tn : t;
                const uint32_t xl = last ? xnext : xrow;
                const int sl = !last ? s_first + (c + 1) * D1 : more ? s_first : s_end;
#pragma unroll
                for (int j = 0; j < D1; ++j) {
#pragma unroll
                    for (int i = 0; i < NF; ++i)
#pragma unroll
                        for (int g = 0; g < NB; ++g) acc[g] = mfma<FMT>(decode<FMT>(st.w[j][g], i), st.x[j].v[i], acc[g]);
                    fetch(st, j, tl, xl, sl + j);
                }
            }
            // lane: rows 4 q + i of the group (gate 0 .. 7, up 8 .. 15), token r
            if (r < t.n) {
#pragma unroll
                for (int g = 0; g < NB; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc.part[flip][wave][g][r][4 * q + i] = acc[g][i];
            }
            if (ask && threadIdx.x == 0) sc.told[flip] = got;
            if (FEW) wait_vm<D1 * (NB * (FMT == kNvfp4 ? 2 : 1) + NF)>();  // the loads of the next task's first steps
            lds_barrier();
            if (FEW && threadIdx.x == 0 && pending >= 0) count_up(&p.count->block[pending], 1);
            const int after = ask ? tail + (int)uniform(sc.told[flip]) : nxt + G;
            if (wave < NB) {
                const int col = t.c0 + 8 * eg + ej;
                if (em < t.n && t.c0 + 8 * eg < p.f) {
                    float g[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) {
                        const float* s = sc.part[flip][w][eg][em];
                        g[0] += s[ej];
                        g[1] += s[ej2];
                        u[0] += s[8 + ej];
                        u[1] += s[8 + ej2];
                    }
                    float h[2];
                    RowScale rs{};
                    if (FMT == kNvfp4) rs = rows[t.row0 + em];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (FMT == kInt8) {
                            g[j] *= cs[j];
                            u[j] *= cs[2 + j];
                        } else if (FMT == kNvfp4) {
                            g[j] = __builtin_amdgcn_ldexpf(g[j] * rs.t1, rs.shift);
                            u[j] = __builtin_amdgcn_ldexpf(u[j] * rs.t1, rs.shift);
                        }
                        h[j] = g[j] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[j])) * u[j];
                    }
                    uint16_t* o = p.h + ((int64_t)(t.row0 + em) * p.f + (col & ~7)) * HP + 2 * ep;
                    if (FMT == kNvfp4) {
                        const half2v v = {(_Float16)__builtin_amdgcn_ldexpf(h[0], -rs.exp),
                                          (_Float16)__builtin_amdgcn_ldexpf(h[1], -rs.exp)};
                        store_through(o, __builtin_bit_cast(uint32_t, v));
                    } else {
                        const uint32_t hi = bf16x2_rne(h[0], h[1]);
                        // (of an infinite h the first part is all)
                        const float l0 = (hi & 0x7F80u) == 0x7F80u ? 0.0f : h[0] - __uint_as_float(hi << 16);
                        const float l1 = (hi & 0x7F800000u) == 0x7F800000u ? 0.0f : h[1] - __uint_as_float(hi & 0xFFFF0000u);
                        store_through(o, hi);
                        store_through(o + 8, bf16x2_rne(l0, l1));
                    }
                }
            }
            ++finished;
            pending = t.block;
            cur = nxt;
            nxt = after;
            t = tn;
            xrow = xnext;
            flip ^= 1;  // (the next task's sums go to the other half while slow threads still read this one)
        }
    }
    wait_vm<0>();  // this wave's h is in memory
    __syncthreads();
    if (threadIdx.x == 0 && finished) {
        if (FEW) count_up(&p.count->block[pending], 1);
        else count_up(&p.count->done, finished);
    }

    // ---- fc2 + combine
    const auto hr = rsrc(p.h, (uint32_t)(p.T * p.k) * (uint32_t)p.f * (2u * HP));
    const uint32_t rb2 = Fmt<FMT>::row_bytes(p.f);
    const int S = (int)(rb2 + 63) / 64, total = V * S, part2 = (total + kWaves - 1) / kWaves;
    const int first = min(wave * part2, total), end = min(first + part2, total);
    const int N2 = (p.d + 15) / 16;
    bool waited = false;
    int upto = FEW ? first / S : V;  // blocks of this wave's run before this one have their h
    auto ready = [&](int b) {
        while (b >= upto) {
            const int at = min(b + lane, 63);
            const bool there = __hip_atomic_load(&p.count->block[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)JB;
            const uint64_t waits = ~__ballot(there);
            const int n = waits ? __builtin_ctzll(waits) : 64;
            upto = b + n;
            if (n == 0) __builtin_amdgcn_s_sleep(16);
        }
        asm volatile("" ::: "memory");
    };
    if (threadIdx.x == 0 && !asked) share2 = take(&p.count->fc2);
    for (int i = tell(share2); i < G; i = tell(share2)) {
      if (i >= N2) {
        if (threadIdx.x == 0) share2 = take(&p.count->fc2);
        continue;
      }
      for (int task = i; task < N2; task += G) {
        const int n0 = task * 16;
        const bool w_ok = n0 + r < p.d;
        for (int z = threadIdx.x; z < kWaves * kMaxT * 17; z += kThreads) (&sc.rows[0][0][0])[z] = 0.0f;
        W16 w[D2];
        u32x4 x[D2][NF][HP];
        int wv = first / S, ws = first - wv * S, xv = wv, xs = ws, cv = wv, cs = ws;  // next weights, h, products
        auto fetch_w = [&](int j, bool live) {
            const int e = __builtin_amdgcn_readfirstlane((int)tb.blocks[live ? wv : 0].e);
            const Matrix<FMT> m(p.w2, p.s2, e, p.d, p.f);
            const uint32_t o = (uint32_t)ws * 64 + q * 16;
            w[j] = m.load((uint32_t)(n0 + r), o, live && o < rb2 && w_ok);
            if (++ws == S) {
                ws = 0;
                ++wv;
            }
        };
        auto fetch_x = [&](int j, bool live) {
            if (FEW && live) ready(xv);
            const Block b = tb.blocks[live ? xv : 0];
            const int n = __builtin_amdgcn_readfirstlane(b.n), row0 = __builtin_amdgcn_readfirstlane((int)b.row0);
            const uint32_t o = (uint32_t)xs * 64 + q * 16;
            const uint32_t at = (uint32_t)(row0 + r) * (uint32_t)p.f * (2u * HP) + o / 16 * (NF * HP * 16);
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int half = 0; half < HP; ++half)
                    x[j][i][half] = __builtin_amdgcn_raw_buffer_load_b128(
                        hr, live && o < rb2 && r < n ? at + 16 * (HP * i + half) : kNowhere, 0, FEW ? kAgentScope : 0);
            if (++xs == S) {
                xs = 0;
                ++xv;
            }
        };
#pragma unroll
        for (int j = 0; j < D2; ++j) fetch_w(j, first + j < end);
        if (FEW || waited) __syncthreads();  // (sc.rows is clear)
        else await(&p.count->done, (uint32_t)N1);
        waited = true;
#pragma unroll
        for (int j = 0; j < D2; ++j) fetch_x(j, first + j < end);
        // (asked for only now, when every workgroup has had time to take its first share)
        if (threadIdx.x == 0 && task + G >= N2) share2 = take(&p.count->fc2);
        auto channel_scales = [&](int b) {  // int8: of this lane's columns in a block's expert, a block ahead of their use
            f32x4 s = {1.0f, 1.0f, 1.0f, 1.0f};
            if (FMT == kInt8 && first < end) {
                const int e = (int)uniform((uint32_t)(int)tb.blocks[min(b, V - 1)].e);
                s = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.s2) + (int64_t)e * p.d +
                                                    min(n0 + 4 * q, p.d - 4));
            }
            return s;
        };
        f32x4 cscale = channel_scales(cv);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i0 = first; i0 < end; i0 += D2) {
#pragma unroll
            for (int j = 0; j < D2; ++j) {
                if (i0 + j < end) {
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        const u32x4 v = decode<FMT>(w[j], i);
#pragma unroll
                        for (int half = 0; half < HP; ++half) acc = mfma<FMT>(v, x[j][i][half], acc);
                    }
                }
                const bool live = i0 + D2 + j < end;
                fetch_w(j, live);
                fetch_x(j, live);
                if (i0 + j < end && (++cs == S || i0 + j + 1 == end)) {
                    const Block b = tb.blocks[cv];
                    if (r < b.n) {
                        const float wt = tb.wt[b.row0 + r];
                        float* o = sc.rows[wave][tb.tok[b.row0 + r]] + 4 * q;
                        if (FMT == kInt8) acc *= cscale;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v = FMT == kNvfp4 ? __builtin_amdgcn_ldexpf(acc[i], rows[b.row0 + r].exp) : acc[i];
                            o[i] = __builtin_fmaf(wt, v, o[i]);
                        }
                    }
                    cscale = channel_scales(cv + 1);
                    acc = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
                    cs = 0;
                    ++cv;
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.T * 16; i += kThreads) {
            const int t = i >> 4, c = i & 15;
            if (n0 + c >= p.d) continue;
            float v = sc.rows[0][t][c];
#pragma unroll
            for (int w2 = 1; w2 < kWaves; ++w2) v += sc.rows[w2][t][c];
            const int64_t at = (int64_t)t * p.d + n0 + c;
            if (p.residual) v += bf16_to_f32(p.residual[at]);
            p.out[at] = (uint16_t)bf16x2_rne(v, v);
        }
        __syncthreads();
      }
    }
}

// ------------------------------------------------------------------ host side
template <int FMT>
bool dims_ok(int64_t T, int64_t d, int64_t E, int k, int64_t f) {
    constexpr int m = Fmt<FMT>::kVals;
    if (T < 0 || T > kMaxT || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E) return false;
    if (d < m || d % m != 0 || d > (1 << 22) || f < m || f % m != 0 || f > (1 << 22)) return false;
    // one expert's matrix, the router's weights and the activations are one buffer descriptor each
    return 2 * f * (int64_t)Fmt<FMT>::row_bytes((int)d) <= kMaxBytes && d * (int64_t)Fmt<FMT>::row_bytes((int)f) <= kMaxBytes &&
           E * d * 2 <= kMaxBytes && T * k * f * 4 <= kMaxBytes;
}
// Parts of K of the router's product: some 200 workgroups in all, of at least four steps a wave.
int router_parts(int64_t T, int64_t d, int64_t E) {
    const int64_t blocks = std::max<int64_t>(1, (E + 15) / 16 * ((T + 15) / 16));
    return (int)std::max<int64_t>(1, std::min({(200 + blocks - 1) / blocks, d / (32 * 4 * kRouterWaves), (int64_t)kMaxParts}));
}
size_t carve(Carver& c, int64_t T, int64_t d, int k, int64_t E, int64_t f, Args* p) {
    p->parts = router_parts(T, d, E);
    p->max_blocks = (int)std::min<int64_t>(T * k, E + T * k / 16);
    p->count = c.take<Counters>(1);
    p->logits = c.take<double>((size_t)(p->parts * T * E));
    p->h = c.take<uint16_t>((size_t)(2 * T * k * f));
    p->xh = c.take<uint16_t>((size_t)(T * d));
    p->xs = c.take<TokenScale>((size_t)T);
    return c.need;
}

template <int FMT, int P, bool FEW>
void launch_layer(const Args& p, hipStream_t s) {
    constexpr int NB = Fmt<FMT>::NB;
    // as many workgroups as have a task, at most one per CU (their registers and LDS let no more be resident)
    const int64_t tasks = std::max<int64_t>((int64_t)p.max_blocks * ((p.f + 8 * NB - 1) / (8 * NB)), (p.d + 15) / 16);
    const unsigned grid = (unsigned)std::min<int64_t>(tasks, device_cus());
    hipLaunchKernelGGL((k_decode_layer<FMT, P, FEW>), dim3(grid), dim3(kThreads), 0, s, p);
}
template <int FMT, int P>
void launch_rows(const Args& p, hipStream_t s) {
    if (p.T <= kOwnChoice && p.T * p.k <= kFewRows) launch_layer<FMT, P, true>(p, s);
    else launch_layer<FMT, P, false>(p, s);
}
template <int FMT>
int run(const Args& p, hipStream_t s) {
    const unsigned grid = (unsigned)((p.E + 15) / 16 * ((p.T + 15) / 16) * p.parts + (FMT == kNvfp4 ? p.T : 0));
    hipLaunchKernelGGL(k_decode_router<FMT == kNvfp4>, dim3(grid), dim3(kRouterThreads), 0, s, p);
    if (p.E <= 128) launch_rows<FMT, 2>(p, s);
    else if (p.E <= 384) launch_rows<FMT, 6>(p, s);
    else launch_rows<FMT, 16>(p, s);
    return launch_status();
}

template <int FMT>
int layer(const uint16_t* x, int64_t T, int64_t d, const uint16_t* w_router, const float* bias, int router, int k, int64_t E,
          int64_t f, const void* w1, const void* s1, const float* t1, const void* w2, const void* s2, const float* t2,
          const uint16_t* residual, uint16_t* out, int32_t* ids, float* weights, void* ws, size_t ws_bytes,
          nvq_stream_t stream) {
    if (router != NVQ_ROUTER_SOFTMAX && router != NVQ_ROUTER_SIGMOID) return NVQ_ERR_UNSUPPORTED;
    if (!dims_ok<FMT>(T, d, E, k, f)) return NVQ_ERR_DIM;
    if (!w_router || !w1 || !w2 || !ws || (FMT != kBf16 && (!s1 || !s2)) || (FMT == kNvfp4 && (!t1 || !t2)) ||
        (T > 0 && (!x || !out || !ids || !weights)))
        return NVQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(w_router) || !aligned16(bias) || !aligned16(w1) || !aligned16(s1) || !aligned16(t1) ||
        !aligned16(w2) || !aligned16(s2) || !aligned16(t2) || !aligned16(residual) || !aligned16(out) || !aligned16(ids) ||
        !aligned16(weights) || !aligned256(ws))
        return NVQ_ERR_ALIGN;
    Args p{};
    Carver need(nullptr);
    if (ws_bytes < carve(need, T, d, k, E, f, &p)) return NVQ_ERR_WORKSPACE;
    if (T == 0) return NVQ_OK;
    Carver cv(ws);
    carve(cv, T, d, k, E, f, &p);
    p.x = x; p.wr = w_router; p.bias = bias;
    p.w1 = w1; p.s1 = s1; p.t1 = t1;
    p.w2 = w2; p.s2 = s2; p.t2 = t2;
    p.residual = residual; p.out = out; p.ids = ids; p.weights = weights;
    p.T = (int)T; p.d = (int)d; p.E = (int)E; p.k = k; p.f = (int)f;
    p.sigmoid = router == NVQ_ROUTER_SIGMOID;
    return run<FMT>(p, as_stream(stream));
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" {

size_t moe_layer_decode_workspace_size(int64_t T, int64_t d, int k, int64_t E, int64_t d_ff) {
    if (T < 0 || T > kMaxT || d < 0 || d > (1 << 22) || k < 1 || k > kMaxK || E < 1 || E > kMaxE || d_ff < 0 || d_ff > (1 << 22)) return 0;
    Carver c(nullptr);
    Args p{};
    return carve(c, T, d, k, E, d_ff, &p);
}

int moe_layer_decode_bf16(const uint16_t* x, int64_t T, int64_t d, const uint16_t* w_router, const float* bias, int router,
                          int k, int64_t E, int64_t d_ff, const uint16_t* w1, const uint16_t* w2,
                          const uint16_t* residual, uint16_t* out, int32_t* topk_ids, float* weights, void* ws,
                          size_t ws_bytes, nvq_stream_t stream) {
    return layer<kBf16>(x, T, d, w_router, bias, router, k, E, d_ff, w1, nullptr, nullptr, w2, nullptr, nullptr, residual,
                        out, topk_ids, weights, ws, ws_bytes, stream);
}

int moe_layer_decode_int8(const uint16_t* x, int64_t T, int64_t d, const uint16_t* w_router, const float* bias, int router,
                          int k, int64_t E, int64_t d_ff, const int8_t* w1, const float* w1_scales, const int8_t* w2,
                          const float* w2_scales, const uint16_t* residual, uint16_t* out, int32_t* topk_ids,
                          float* weights, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    return layer<kInt8>(x, T, d, w_router, bias, router, k, E, d_ff, w1, w1_scales, nullptr, w2, w2_scales, nullptr,
                        residual, out, topk_ids, weights, ws, ws_bytes, stream);
}

int moe_layer_decode_nvfp4(const uint16_t* x, int64_t T, int64_t d, const uint16_t* w_router, const float* bias, int router,
                           int k, int64_t E, int64_t d_ff, const uint8_t* w1_codes, const uint8_t* w1_scales,
                           const float* w1_tscale, const uint8_t* w2_codes, const uint8_t* w2_scales,
                           const float* w2_tscale, const uint16_t* residual, uint16_t* out, int32_t* topk_ids,
                           float* weights, void* ws, size_t ws_bytes, nvq_stream_t stream) {
    return layer<kNvfp4>(x, T, d, w_router, bias, router, k, E, d_ff, w1_codes, w1_scales, w1_tscale, w2_codes, w2_scales,
                         w2_tscale, residual, out, topk_ids, weights, ws, ws_bytes, stream);
}

}  // extern "C"
