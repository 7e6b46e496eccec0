// nvq_decode.hip -- a whole mixture-of-experts layer for a few tokens (up to
// 64, single tokens being decoded): router, chosen experts and weighted combine
// on bf16, int8 or NVFP4 weights.
//
//   k_decode_router   logits = x Wr^T
//   k_decode_fc1      ids, weights = top-k of the logits (k_decode_choice where
//                     tokens are more than eight);
//                     h = silu(g) * u of every (expert, token) pair
//   k_decode_fc2      out = residual + sum_s weight * (W2 h)
//
// All of it after the router in one kernel, whose workgroups took tasks from
// device counters, handed h over through memory and had their first W2 in
// flight while they waited, was built and measured too. For 8 of 384 experts,
// d 4096, f 1024 (us, that kernel and these): one bf16 token 65 and 56, four
// int8 tokens 113 and 102, one NVFP4 token 43 and 38, 64 of them 515 and 497 (before WIDE).
// Noticing that the last workgroup is done and reading h past the caches costs
// more than a launch.
//
// Bound by reading the chosen experts' weights, once per 16 tokens of an expert
// (NVFP4's fc2: eight). The activations are not quantized: they are a few rows,
// and it would save nothing. A weight reaches the matrix pipe as the bf16 value
// that holds it exactly (int8 codes have 8 significant bits, e2m1 * e4m3 has 6);
// the channel's or tensor's fp32 scale is applied to the fp32 sum.
//
// The other operand is x as it is, and h as two bf16 parts, its rounding and the
// rounding of what that left (2^-16 of it in all; one part would be 2^-8, as much
// as out's own rounding). bf16's exponents hold whatever fp32's do, so nothing has
// to be known of h's size beforehand: fp16 needs a power of two per row, and the
// only one at hand before h is computed, from the 1-norm of x and the largest
// weight that the tensor scale allows, can lie any number of bits above h.
#include "nvq_argmax.hpp"
#include "nvq_device.hpp"
#include "nvq_host.hpp"

#include <algorithm>

namespace nvq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

enum { kBf16 = 0, kInt8 = 1, kNvfp4 = 2 };

constexpr int kMaxT = 64;       // tokens: an expert's are one 64-bit mask
constexpr int kMaxE = 1024;
constexpr int kMaxK = 64;
constexpr int kMaxA = kMaxT * kMaxK;
constexpr int kMaxV = kMaxE + kMaxA / 16;  // blocks of at most 16 tokens of one expert
constexpr int kMaxV8 = kMaxE + kMaxA / 8;  // of at most eight
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int64_t kMaxBytes = 0xFFFFFE00ll;     // of a buffer
constexpr uint32_t kNowhere = (uint32_t)kMaxBytes;  // an offset behind any buffer's end, also with 511 added: reads zeros

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
    uint16_t* h;              // [T k, f], rows in expert order: each eight values' high, then low parts
    uint16_t* xp;             // NVFP4: x (both in the order of decoded codes)
    uint32_t* tail;           // tasks taken of fc1's tail (k_decode_router clears it)
    struct Plan* plan;        // fc1's table, for fc2
    int T, d, E, k, f, sigmoid, parts, max_blocks;  // max_blocks: of fc2
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
    static constexpr int kRows = FMT == kNvfp4 ? 8 : 16;    // tokens of a block in fc2
    static __host__ __device__ __forceinline__ uint32_t row_bytes(int K) { return (uint32_t)(K / kVals) * 16u; }
};

struct W16 {
    u32x4 w;
    uint32_t sc;   // NVFP4: the two scale bytes, in the lower or (decode's HI) upper half
};
template <int FMT>
struct X16 {
    u32x4 v[Fmt<FMT>::kFrags];
};

// NVFP4's codes are decoded in the pairs (0 2) (4 6) (1 3) (5 7) of eight, and the other operands are held in that order.
//
// The eight magnitudes of E2M1 times the E4M3 scale `byte`, as bf16 (6 significant bits at most: exact; all NaN for a NaN):
// the lower bytes of codes 0 .. 3 and 4 .. 7, then the upper ones.
__device__ __forceinline__ u32x4 fp4_products(uint32_t byte) {
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
    constexpr float kMag[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
    u32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t b = __float_as_uint(kMag[c] * s);
        o[c >> 2] |= (b >> 16 & 0xFFu) << 8 * (c & 3);
        o[2 + (c >> 2)] |= (b >> 24) << 8 * (c & 3);
    }
    return o;
}
// fp4_products of every scale byte, in LDS, by all threads.
__device__ __forceinline__ void fill_products(u32x4 (&table)[256]) {
    if (threadIdx.x < 256) table[threadIdx.x] = fp4_products(threadIdx.x);
}

// fc2, WIDE (d_ff a multiple of kWideF): place of a row's group u of eight h. A lane takes four neighbouring groups of a step's
// 16, one with each load; the groups that the lanes of one load take are neighbours here, whole lines of both parts (64
// tokens of 384 experts 397 us without, 394 with; of 8, all chosen, 154 and 146).
constexpr int kWideF = 512;  // blocks of whole groups of four steps
__device__ __forceinline__ int wide_group(int u) { return (u & ~15) | (u & 3) << 2 | (u >> 2 & 3); }

// Eight E2M1 codes times the scale of products `t`. Byte permutes look up lower and upper bytes four
// codes at a time, the codes' signs flip the upper ones, four more permutes join them: 14 full-rate operations for 8 values, and
// one LDS read for 16 of them. (Multiplying by the scale would be done in fp32, 28 operations.)
__device__ __forceinline__ u32x4 decode_fp4(uint32_t w, u32x4 t) {
    const uint32_t even = w & 0x07070707u, odd = (w >> 4) & 0x07070707u;
    const uint32_t el = __builtin_amdgcn_perm(t[1], t[0], even), ol = __builtin_amdgcn_perm(t[1], t[0], odd);
    const uint32_t eh = __builtin_amdgcn_perm(t[3], t[2], even) ^ ((w << 4) & 0x80808080u);
    const uint32_t oh = __builtin_amdgcn_perm(t[3], t[2], odd) ^ (w & 0x80808080u);
    return (u32x4){__builtin_amdgcn_perm(eh, el, 0x05010400u), __builtin_amdgcn_perm(eh, el, 0x07030602u),
                   __builtin_amdgcn_perm(oh, ol, 0x05010400u), __builtin_amdgcn_perm(oh, ol, 0x07030602u)};
}

// Fragment i (8 values) of 16 bytes of weights, in bf16. `table`: NVFP4's fill_products.
template <int FMT, bool HI = false, typename Table>
__device__ __forceinline__ u32x4 decode(const W16& w, int i, const Table& table) {
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
        return decode_fp4(w.w[i], table[w.sc >> (16 * HI + 8 * (i >> 1)) & 0xFFu]);
    }
}
__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
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
    // 16 bytes at byte `o` of row `row` (nothing is read where !ok) and, unless WIDE, NVFP4's scales
    template <bool WIDE>
    __device__ __forceinline__ W16 load(uint32_t row, uint32_t o, bool ok) const {
        W16 r;
        const uint32_t at = ok ? row * rb + o : kNowhere;
        r.w = __builtin_amdgcn_raw_buffer_load_b128(w, at, 0, 2);  // read once: past the caches
        r.sc = FMT == kNvfp4 && !WIDE ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(s, ok ? at / 8 : kNowhere, 0, 0) : 0;
        return r;
    }
    // The eight scale bytes of a row's step (whole steps only).
    __device__ __forceinline__ u32x2 scales(uint32_t row, int step, bool ok) const {
        return __builtin_amdgcn_raw_buffer_load_b64(s, ok ? row * (rb / 8) + step * 8 : kNowhere, 0, 0);
    }
};
// NVFP4, WIDE: four steps' scales as one load, lane l taking the eight bytes of step l / 16, of which lane 16 j + r wants
// bytes 2 j, 2 j + 1 of each: a 4 x 4 transposition between the lanes of a row. sc[0]: steps 0, 1; sc[1]: 2, 3. Two bytes
// per lane and step, as `load` takes them, are a memory instruction for each weight instruction: the 384-expert layer's 64
// tokens took 497 us with those, 377 so, eight 143 and 113, one 38 and 34 (with h in one part).
__device__ __forceinline__ void spread(u32x2 v, int lane, uint32_t (&sc)[2]) {
    const uint32_t half = lane & 16 ? 0x07060302u : 0x05040100u;
    const auto ab = __builtin_amdgcn_permlane32_swap(v[0], v[1], false, false);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto eo = __builtin_amdgcn_permlane16_swap(ab[i], ab[i], false, false);
        sc[i] = __builtin_amdgcn_perm(eo[1], eo[0], half);
    }
}
template <int FMT>
__device__ __forceinline__ X16<FMT> load_x(__amdgpu_buffer_rsrc_t x, uint32_t row, int K, uint32_t o, bool ok) {
    X16<FMT> r;
    const uint32_t at = ok ? row * (uint32_t)K * 2u + o / 16 * (2u * Fmt<FMT>::kVals) : kNowhere;
#pragma unroll
    for (int i = 0; i < Fmt<FMT>::kFrags; ++i) r.v[i] = __builtin_amdgcn_raw_buffer_load_b128(x, at + 16 * i, 0, 0);
    return r;
}

// A barrier that orders LDS only: loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------------ router logits
// One workgroup: 16 experts, 16 tokens, a part of K, shared by its four waves. Products and sums are fp64, so that of two
// close logits the larger one is chosen: the bf16 instruction's sum of 32 products is off by up to 2^-21 of their magnitudes
// (1 and 31 products of 2^-28 give 1), which chooses wrongly where x has a few large values. Its launch took 3.7 us for one
// token of 384 experts and 7.7 for 64, this one takes 4.5 and 7.5. K is cut so that a token's logits are some 800 workgroups,
// or eight parts: the fp64 products are the most of its time, and 64 tokens in three parts, 288 workgroups on 256 CUs, take
// 11.4 us, in five 8.7.
constexpr int kRouterWaves = 4, kRouterThreads = 64 * kRouterWaves;

// x of token t in the order of decoded codes for NVFP4 weights (one workgroup).
__device__ __forceinline__ void order_token(const Args& p, int t) {
    const u32x4* src = reinterpret_cast<const u32x4*>(p.x + (int64_t)t * p.d);
    u32x4* dst = reinterpret_cast<u32x4*>(p.xp + (int64_t)t * p.d);
#pragma unroll 2
    for (int u = threadIdx.x; u < p.d / 8; u += kRouterThreads) {
        const u32x4 v = src[u];
        auto even = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); };
        auto odd = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); };
        dst[u] = (u32x4){even(v[0], v[1]), even(v[2], v[3]), odd(v[0], v[1]), odd(v[2], v[3])};
    }
}

template <bool ORDER>
__global__ __launch_bounds__(kRouterThreads) void k_decode_router(Args p) {
    __shared__ double red[kRouterWaves][16][17];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.tail = 0;
    int b = blockIdx.x;
    if (ORDER) {
        if (b < p.T) return order_token(p, b);
        b -= p.T;
    }
    const int eb = (p.E + 15) / 16, tb = (p.T + 15) / 16;
    const int e0 = b % eb * 16, t0 = b / eb % tb * 16, z = b / (eb * tb);
    const uint32_t rb = (uint32_t)p.d * 2u;
    const auto wr = rsrc(p.wr, (uint32_t)p.E * rb), xr = rsrc(p.x, (uint32_t)p.T * rb);
    const int steps = (p.d + 31) / 32, waves = p.parts * kRouterWaves, part = (steps + waves - 1) / waves;
    const int first = (z * kRouterWaves + wave) * part, s1 = min(first + part, steps);
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
    auto value = [](u32x4 u, int v) {
        return (double)__uint_as_float(v & 1 ? u[v >> 1] & 0xFFFF0000u : u[v >> 1] << 16);
    };
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
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 8; ++v)  // lane: value v of its eight of K
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(value(w[j], v), value(x[j], v), acc, 0, 0, 0);
    }
    // lane: experts q + 4 i of token r
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r][q + 4 * i] = acc[i];
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

// The chosen experts and their tokens: blocks of at most 16 tokens of one expert (NVFP4's fc2: eight), in ascending expert
// order; row row0 + i of h and of rows is token i of the block.
struct Block {
    int16_t e;
    int16_t row0;
    int32_t n;
};
struct Row {
    float wt;       // routing weight; NVFP4: times w2's tensor scale
    int32_t token;
};
struct Plan {       // fc2's
    int32_t blocks_n;
    int32_t pad[3];
    Block blocks[kMaxV8];
    Row rows[kMaxA];
};
struct Table {
    uint64_t mask[kMaxE];  // tokens of each expert
    int32_t base[kMaxE];   // its first row
    Block blocks[kMaxV];
    Row rows[kMaxA];
    uint32_t scan[kWaves];
};
// From ids and weights (of another launch, or of this workgroup). All threads take part; returns the number of blocks. t1:
// NVFP4's w1 tensor scale per row. `plan`: where not null, fc2's blocks go there.
template <int FMT>
__device__ __forceinline__ int build(Table& tb, float* t1, Plan* plan, const Args& p, const int32_t* ids,
                                     const float* weights) {
    constexpr int kRows = Fmt<FMT>::kRows;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int A = p.T * p.k;
    struct Scales {
        float t1, t2;
    };
    auto scales = [&](int a) { return Scales{p.t1[ids[a]], p.t2[ids[a]]}; };
    Scales early = {};  // of row t, on their way while the table is made
    if (FMT == kNvfp4 && t < A) early = scales(t);
    for (int e = t; e < p.E; e += kThreads) tb.mask[e] = 0;
    __syncthreads();
    for (int a = t; a < A; a += kThreads)
        atomicOr(reinterpret_cast<unsigned long long*>(&tb.mask[ids[a]]), 1ull << (a / p.k));
    __syncthreads();
    // prefix sums over the experts (two neighbouring ones per thread) of blocks (the lowest 11 bits: at most kMaxV), of what
    // blocks of eight are more (9 bits: at most kMaxA / 9) and of rows (12 bits, modulo kMaxA: an expert with rows starts below)
    static_assert(kMaxV < 1 << 11 && kMaxA / 9 < 1 << 9 && kMaxA == 1 << 12, "packed sums");
    auto counts = [](uint32_t n) { return (n + 15) / 16 | (n + 7) / 16 << 11 | n << 20; };
    uint32_t n[2], sum = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = 2 * t + j;
        n[j] = e < p.E ? __popcll(tb.mask[e]) : 0;
        sum += counts(n[j]);
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t v = (uint32_t)__shfl_up((int)incl, off, 64);
        incl += lane >= off ? v : 0;
    }
    if (lane == 63) tb.scan[wave] = incl;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t v = tb.scan[w];
        before += w < wave ? v : 0;
        total += v;
    }
    uint32_t at = before + incl - sum;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = 2 * t + j;
        if (e < p.E) {
            const int row = at >> 20, b = at & 0x7FF, more = at >> 11 & 0x1FF, m = (int)n[j];
            auto put = [&](Block* to, int rows) {
                for (int i = 0; i * rows < m; ++i) to[i] = {(int16_t)e, (int16_t)(row + rows * i), min(rows, m - rows * i)};
            };
            tb.base[e] = row;
            put(tb.blocks + b, 16);
            if (plan) put(plan->blocks + b + (kRows == 8 ? more : 0), kRows);
        }
        at += counts(n[j]);
    }
    const uint32_t blocks = total & 0x7FF, more = total >> 11 & 0x1FF;
    if (plan && t == 0) plan->blocks_n = blocks + (kRows == 8 ? more : 0);
    __syncthreads();
    for (int a = t; a < A; a += kThreads) {
        const int e = ids[a], tk = a / p.k;
        const int row = tb.base[e] + __popcll(tb.mask[e] & ((1ull << tk) - 1));
        Row v = {weights[a], tk};
        if (FMT == kNvfp4) {
            const Scales s = a == t ? early : scales(a);
            v.wt *= s.t2;
            t1[row] = s.t1;
        }
        tb.rows[row] = v;
    }
    __syncthreads();
    return (int)uniform(blocks);
}

// Up to this many tokens every workgroup of fc1 chooses for itself: a launch of its own costs as much as adding eight tokens'
// logits (three tokens of 8 experts 22.4 us against 25.2 with the launch, eight of 64 32.7 and 34.3, eight of 384 on int8
// weights 169 and 167.5).
constexpr int kOwnChoice = kWaves;
// Tokens t0 .. t0 + N - 1 (those below T), one per wave, by all threads.
template <int P, int N>
__device__ __forceinline__ void choose_for(const Args& p, int t0, double (*val)[kMaxE], const float* bias, int32_t* ids,
                                           float* weights) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), t = t0 + wave;
    add_parts(p, t0, min(p.T - t0, N), val);
    __syncthreads();
    if (wave >= N || t >= p.T) return;
    int id;
    float w;
    choose<P>(p, val[wave], bias, lane, &id, &w);
    if (lane < p.k) {
        ids[t * p.k + lane] = id;
        weights[t * p.k + lane] = w;
    }
}
__device__ __forceinline__ void load_bias(const Args& p, float* bias) {
    for (int e = threadIdx.x; e < p.E; e += kThreads) bias[e] = p.bias ? p.bias[e] : 0.0f;
}
// A token per workgroup: its threads add the logits' parts, one wave chooses. (Eight tokens per workgroup, 64 tokens of 384
// experts: 10.4 us instead of 7.)
template <int P>
__global__ __launch_bounds__(kThreads) void k_decode_choice(Args p) {
    __shared__ double val[1][kMaxE];
    __shared__ float bias[kMaxE];
    load_bias(p, bias);
    choose_for<P, 1>(p, (int)blockIdx.x, val, bias, p.ids, p.weights);
}

// ------------------------------------------------------------------ fc1 + SwiGLU
// One persistent workgroup per CU. A task is one block of tokens and 8 NB gate rows with their up rows; the waves share K
// and their sums meet in LDS, added in order. A wave's loads run ahead across the tasks' ends: D1 steps, 8 KiB of weights,
// are in flight all the time, 64 KiB per CU (twice as many were no faster): 64 tokens read the w1 of the 210 of 384 experts
// that they hit at 4.8 TB/s (bf16, 731 us), 4.7 (int8, 375) and 4.0 (NVFP4, 246: a wave has four loads of x for two of
// weights), one bf16 token that of its eight at 4.1.
template <int FMT>
struct Stage1 {  // operands of a wave in flight
    u32x2 raw[Fmt<FMT>::NB];  // WIDE: scales of the steps
    W16 w[Fmt<FMT>::D1][Fmt<FMT>::NB];
    X16<FMT> x[Fmt<FMT>::D1];
};
struct Task1 {  // all scalars
    int e, n, row0, c0;
};

// Next of the tail's tasks, by one thread. (The offset that the compiler cannot see through keeps it from first adding up
// over the wave, which would wait for the result, and with it for every load in flight, on the spot.)
__device__ __forceinline__ uint32_t take(uint32_t* counter) {
    uint32_t zero = 0;
    asm volatile("" : "+v"(zero));
    return __hip_atomic_fetch_add(counter + zero, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int FMT, int P, bool WIDE>
__global__ __launch_bounds__(kThreads, 2) void k_decode_fc1(Args p) {
    static_assert(!WIDE || (FMT == kNvfp4 && Fmt<FMT>::D1 == 4), "four steps' scales");
    constexpr int NB = Fmt<FMT>::NB, D1 = Fmt<FMT>::D1, NF = Fmt<FMT>::kFrags;
    union Scratch {
        struct {
            float part[2][kWaves][NB][16][17];  // each wave's sums
            uint32_t told[2];                   // a task
        };
        struct {
            int32_t ids[kOwnChoice * kMaxK];
            float weights[kOwnChoice * kMaxK];
            double val[kWaves][kMaxE];
        } c;                                    // the choice
    };
    __shared__ Table tb;
    __shared__ Scratch sc;
    __shared__ float bias[kMaxE];
    __shared__ float t1[FMT == kNvfp4 ? kMaxA : 1];
    __shared__ u32x4 products[FMT == kNvfp4 ? 256 : 1];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int G = gridDim.x;
    if constexpr (FMT == kNvfp4) fill_products(products);
    Plan* plan = (int)blockIdx.x == G - 1 ? p.plan : nullptr;  // (by the workgroup with the fewest tasks)
    int V;
    if (p.T <= kOwnChoice) {
        load_bias(p, bias);
        choose_for<P, kOwnChoice>(p, 0, sc.c.val, bias, sc.c.ids, sc.c.weights);
        __syncthreads();
        V = build<FMT>(tb, t1, plan, p, sc.c.ids, sc.c.weights);
    } else {
        V = build<FMT>(tb, t1, plan, p, p.ids, p.weights);
    }
    if (plan) {  // the rest of it, and what the caller gets
        const int A = p.T * p.k;
        for (int i = threadIdx.x; i < A; i += kThreads) {
            plan->rows[i] = tb.rows[i];
            if (p.T <= kOwnChoice) {
                p.ids[i] = sc.c.ids[i];
                p.weights[i] = sc.c.weights[i];
            }
        }
        __syncthreads();
    }

    const int JB = (p.f + 8 * NB - 1) / (8 * NB), N1 = V * JB;
    const auto xr = rsrc(FMT == kNvfp4 ? p.xp : p.x, (uint32_t)p.T * (uint32_t)p.d * 2u);
    const uint32_t rb = Fmt<FMT>::row_bytes(p.d);
    const int steps = (int)(rb + 63) / 64, part = (steps + kWaves - 1) / kWaves;
    const int chunks = (part + D1 - 1) / D1, s_first = wave * part, s_end = min(s_first + part, steps);
    auto set = [&](int task) {
        const Block b = tb.blocks[task / JB];
        return Task1{(int)uniform(b.e), (int)uniform(b.n), (int)uniform(b.row0), task % JB * 8 * NB};
    };
    auto fetch = [&](Stage1<FMT>& st, int j, const Task1& t, uint32_t xrow, int s) {
        const Matrix<FMT> m(p.w1, p.s1, t.e, 2 * p.f, p.d);
        const uint32_t o = (uint32_t)s * 64 + q * 16;
        const bool ok = s < s_end && o < rb;
        const int col = t.c0 + (r & 7);
#pragma unroll
        for (int g = 0; g < NB; ++g) {
            const uint32_t row = (r < 8 ? 0 : p.f) + col + 8 * g;
            if (WIDE && j == 0) st.raw[g] = m.scales(row, s + q, s + q < s_end && col + 8 * g < p.f);
            st.w[j][g] = m.template load<WIDE>(row, o, ok && col + 8 * g < p.f);
        }
        st.x[j] = load_x<FMT>(xr, xrow, p.d, o, ok && r < t.n);
    };
    auto token = [&](const Task1& t) { return (uint32_t)tb.rows[t.row0 + min(r, t.n - 1)].token; };
    // The epilogue's thread: two columns of a token, neighbours as the operand of fc2 holds them.
    const int em = threadIdx.x / (4 * NB), eg = threadIdx.x / 4 % NB, ep = threadIdx.x & 3;
    const int ej = FMT == kNvfp4 ? (ep & 1) * 4 + (ep >> 1) : 2 * ep, ej2 = ej + (FMT == kNvfp4 ? 2 : 1);
    // A workgroup's tasks are blockIdx.x, + G, ...; where there are many, only those before `tail`, whole rounds, and the
    // rest is taken from a counter, two tasks ahead of its use (64 tokens of 384 experts without
    // and with, before WIDE: NVFP4 504 and 497 us, int8 607 and 599, bf16 1013 and 995; the last workgroup ends 6 us after
    // the median one instead of 34). Which workgroup does a task does not show in its result.
    const int tail = N1 >= 24 * G ? (N1 / G - 4) * G : N1;
    int cur = blockIdx.x, nxt = cur + G, flip = 0;
    if (cur >= N1) return;
    Stage1<FMT> st;
    Task1 t = set(cur);
    uint32_t xrow = token(t);
#pragma unroll
    for (int j = 0; j < D1; ++j) fetch(st, j, t, xrow, s_first + j);
    while (cur < N1) {
        const bool more = nxt < N1;
        // the task after the next one (a taken one is told at this task's barrier)
        const bool ask = tail < N1 && nxt + G >= tail;
        uint32_t got = 0;
        if (ask && threadIdx.x == 0) got = take(p.tail);
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
            uint32_t sc2[NB][2];
            if (WIDE) {
#pragma unroll
                for (int g = 0; g < NB; ++g) spread(st.raw[g], lane, sc2[g]);
            }
#pragma unroll
            for (int j = 0; j < D1; ++j) {
#pragma unroll
                for (int i = 0; i < NF; ++i)
#pragma unroll
                    for (int g = 0; g < NB; ++g) {
                        W16 w = st.w[j][g];
                        if (WIDE) w.sc = sc2[g][j >> 1 & 1];
                        acc[g] = mfma(WIDE && (j & 1) ? decode<FMT, true>(w, i, products) : decode<FMT>(w, i, products),
                                      st.x[j].v[i], acc[g]);
                    }
                fetch(st, j, tl, xl, sl + j);
                __builtin_amdgcn_sched_barrier(0);  // (steps run into each other take 80 registers more and are slower)
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
        lds_barrier();
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
                const float ts = FMT == kNvfp4 ? t1[t.row0 + em] : 1.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (FMT == kInt8) {
                        g[j] *= cs[j];
                        u[j] *= cs[2 + j];
                    } else if (FMT == kNvfp4) {
                        g[j] *= ts;
                        u[j] *= ts;
                    }
                    h[j] = g[j] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[j])) * u[j];
                }
                const int at = FMT == kNvfp4 && p.f % kWideF == 0 ? wide_group(col >> 3) : col >> 3;
                uint16_t* o = p.h + (int64_t)(t.row0 + em) * p.f * 2 + at * 16 + 2 * ep;
                const uint32_t hi = bf16x2_rne(h[0], h[1]);
                // (of an infinite h the first part is all)
                const float l0 = (hi & 0x7F80u) == 0x7F80u ? 0.0f : h[0] - __uint_as_float(hi << 16);
                const float l1 = (hi & 0x7F800000u) == 0x7F800000u ? 0.0f : h[1] - __uint_as_float(hi & 0xFFFF0000u);
                *reinterpret_cast<uint32_t*>(o) = hi;
                *reinterpret_cast<uint32_t*>(o + 8) = bf16x2_rne(l0, l1);
            }
        }
        cur = nxt;
        nxt = after;
        t = tn;
        xrow = xnext;
        flip ^= 1;  // (the next task's sums go to the other half while slow threads still read this one)
    }
}

// ------------------------------------------------------------------ fc2 + combine
// A workgroup owns 16 columns of out: d = 4096 is one per CU, fewer columns leave CUs without work (64 tokens of 384
// experts read w2 at 4.3, 3.3 and 3.0 TB/s in bf16, int8 and NVFP4 with d = 4096, at 2.6, 1.9 and 1.7 with 2048). Its waves
// share the (block, K step) pairs of all chosen experts in equal contiguous runs, D2 steps in flight; where a run leaves a
// block, the wave adds weight * sum to its own token rows in LDS. The waves' rows are added in order at the end. Nothing
// but the operands is loaded inside the loop, so that no wait empties the pipeline (int8 with the channel scales loaded
// there: four tokens 118 us instead of 102, 64 713 instead of 602). D2 of 6, 10 or (bf16) 12, 16 is within 2 % of 8, the
// deeper ones on the slow side.
//
// The two parts of h are two products with one weight fragment. NVFP4's 16 bytes are four fragments, and both parts of them
// would be 256 registers for D2 steps: there a block is at most eight tokens, columns 0 .. 7 of one product their upper and
// 8 .. 15 their lower parts, and the two sums are added at the block's end. Blocks of 16 with both products and four steps in
// flight: 64 tokens of 384 experts 442 us, 394 so; eight 129 and 115; only where most blocks are full are they a little
// faster (64 tokens, all of 8 experts 137 and 146). What the lower part costs is its way through the L2: that last case
// takes 113 us with one part, and its fc2 half as long without any h.
template <int FMT, bool WIDE>
__global__ __launch_bounds__(kThreads, 2) void k_decode_fc2(Args p) {
    constexpr bool SPLIT = Fmt<FMT>::kRows == 8;
    constexpr int D2 = 8, kOuts = kMaxT * 16 / kThreads, NF = Fmt<FMT>::kFrags, HP = SPLIT ? 1 : 2;
    __shared__ Block blocks[SPLIT ? kMaxV8 : kMaxV];
    __shared__ Row rows[kMaxA];
    __shared__ float sums[kWaves][kMaxT][17];
    __shared__ f32x4 channel[FMT == kInt8 ? kMaxV : 1][4];  // s2 of the 16 columns, per block
    __shared__ u32x4 products[FMT == kNvfp4 ? 256 : 1];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int hrow = SPLIT ? r & 7 : r, low = SPLIT ? r >> 3 : 0;  // row of the block, and part, in this lane's column
    if constexpr (FMT == kNvfp4) fill_products(products);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int A = p.T * p.k, V = (int)uniform((uint32_t)p.plan->blocks_n);
    for (int i = threadIdx.x; i < p.max_blocks; i += kThreads) blocks[i] = p.plan->blocks[i];
    for (int i = threadIdx.x; i < A; i += kThreads) rows[i] = p.plan->rows[i];
    const auto hr = rsrc(p.h, (uint32_t)A * (uint32_t)p.f * 4u);
    const uint32_t rb = Fmt<FMT>::row_bytes(p.f);
    const int S = (int)(rb + 63) / 64, total = V * S;
    constexpr int kUnit = WIDE ? 4 : 1;  // steps whose scales are one load; a block is whole units of them
    const int part = (total + kWaves * kUnit - 1) / (kWaves * kUnit) * kUnit;
    const int first = min(wave * part, total), end = min(first + part, total);
    const int n0 = blockIdx.x * 16;
    const bool w_ok = n0 + r < p.d;
#pragma unroll 1
    for (int z = lane; z < p.T * 17; z += 64) (&sums[wave][0][0])[z] = 0.0f;
    uint16_t old[kOuts] = {};  // the residual of this thread's outputs, ahead of all other loads
#pragma unroll
    for (int u = 0; u < kOuts; ++u) {
        const int i = threadIdx.x + u * kThreads, c = i & 15;
        if (p.residual && i < p.T * 16 && n0 + c < p.d) old[u] = p.residual[(int64_t)(i >> 4) * p.d + n0 + c];
    }
    __syncthreads();
    W16 w[D2];
    u32x4 x[D2][NF][HP];
    u32x2 raw[D2 / 4];
    int cv = first / S, cs = first - cv * S;  // the next step's block and step in it, of the products
    int lv = cv, ls = cs;                     // and of the loads
    Matrix<FMT> m(p.w2, p.s2, 0, p.d, p.f);
    uint32_t at = 0;                          // of this lane's row of h in block lv
    bool x_ok = false;
    auto enter = [&](int v) {
        const Block b = blocks[min(v, V - 1)];
        m = Matrix<FMT>(p.w2, p.s2, (int)uniform((uint32_t)(int)b.e), p.d, p.f);
        at = ((uint32_t)(int)uniform((uint32_t)(int)b.row0) + hrow) * (uint32_t)p.f * 4u + 16 * low;
        x_ok = hrow < (int)uniform((uint32_t)b.n);
    };
    auto fetch = [&](int j, bool live) {
        const uint32_t o = (uint32_t)ls * 64 + q * 16;
        const bool ok = live & (o < rb);
        if (WIDE && (j & 3) == 0) raw[j >> 2] = m.scales((uint32_t)(n0 + r), ls + q, live & w_ok);
        w[j] = m.template load<WIDE>((uint32_t)(n0 + r), o, ok & w_ok);
        const uint32_t from = (ok & x_ok) ? at + (WIDE ? (uint32_t)ls * 512u + q * 32 : o / 16 * (NF * 32)) : kNowhere;
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int half = 0; half < HP; ++half)
                x[j][i][half] = __builtin_amdgcn_raw_buffer_load_b128(hr, from + (WIDE ? 128 : 32) * i + 16 * half, 0, 0);
        if (++ls == S) {
            ls = 0;
            enter(++lv);
        }
    };
    enter(lv);
#pragma unroll
    for (int j = 0; j < D2; ++j) fetch(j, first + j < end);
    if (FMT == kInt8) {  // through LDS: a wait for a load of its own would wait for all that run ahead
        for (int i = threadIdx.x; i < 4 * V; i += kThreads)
            channel[i >> 2][i & 3] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.s2) +
                                                                     (int64_t)blocks[i >> 2].e * p.d + min(n0 + 4 * (i & 3), p.d - 4));
        lds_barrier();
    }
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t sc2[2];
    for (int i0 = first; i0 < end; i0 += D2) {
#pragma unroll
        for (int j = 0; j < D2; ++j) {
            if (WIDE && (j & 3) == 0) spread(raw[j >> 2], lane, sc2);
            if (i0 + j < end) {
                W16 wj = w[j];
                if (WIDE) wj.sc = sc2[j >> 1 & 1];
#pragma unroll
                for (int i = 0; i < NF; ++i) {
                    const u32x4 v = WIDE && (j & 1) ? decode<FMT, true>(wj, i, products) : decode<FMT>(wj, i, products);
#pragma unroll
                    for (int half = 0; half < HP; ++half) acc = mfma(v, x[j][i][half], acc);
                }
            }
            fetch(j, i0 + D2 + j < end);
            __builtin_amdgcn_sched_barrier(0);  // (four int8 tokens 102.5 us without, 100 with)
            if (i0 + j < end && (++cs == S || i0 + j + 1 == end)) {
                const Block b = blocks[cv];
                if (SPLIT) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // of lane r + 8
                        acc[i] += __uint_as_float(dpp_u32<0x128>(__float_as_uint(acc[i])));
                }
                if (r < b.n) {
                    const Row row = rows[b.row0 + r];
                    float* o = sums[wave][row.token] + 4 * q;
                    if (FMT == kInt8) acc *= channel[cv][q];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = __builtin_fmaf(row.wt, acc[i], o[i]);
                }
                acc = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
                cs = 0;
                ++cv;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kOuts; ++u) {
        const int i = threadIdx.x + u * kThreads, t = i >> 4, c = i & 15;
        if (i >= p.T * 16 || n0 + c >= p.d) continue;
        float v = sums[0][t][c];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) v += sums[k][t][c];
        if (p.residual) v += bf16_to_f32(old[u]);
        p.out[(int64_t)t * p.d + n0 + c] = (uint16_t)bf16x2_rne(v, v);
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
// Parts of K of the router's product: some 800 workgroups in all, of at least four steps a wave.
int router_parts(int64_t T, int64_t d, int64_t E) {
    const int64_t blocks = std::max<int64_t>(1, (E + 15) / 16 * ((T + 15) / 16));
    return (int)std::max<int64_t>(1, std::min({(800 + blocks - 1) / blocks, d / (32 * 4 * kRouterWaves), (int64_t)kMaxParts}));
}
// `rows`: tokens of a block in fc2.
size_t carve(Carver& c, int64_t T, int64_t d, int k, int64_t E, int64_t f, int rows, Args* p) {
    p->parts = router_parts(T, d, E);
    p->max_blocks = (int)std::min<int64_t>(T * k, E + T * k / rows);
    p->tail = c.take<uint32_t>(1);
    p->plan = c.take<Plan>(1);
    p->logits = c.take<double>((size_t)(p->parts * T * E));
    p->h = c.take<uint16_t>((size_t)(2 * T * k * f));
    p->xp = c.take<uint16_t>((size_t)(T * d));
    return c.need;
}

template <int FMT, int P>
void launch_fc1(const Args& p, hipStream_t s) {
    constexpr int NB = Fmt<FMT>::NB;
    if (p.T > kOwnChoice)
        hipLaunchKernelGGL(k_decode_choice<P>, dim3((unsigned)p.T), dim3(kThreads), 0, s, p);
    const int64_t blocks = std::min<int64_t>(p.T * p.k, p.E + p.T * p.k / 16), tasks = blocks * ((p.f + 8 * NB - 1) / (8 * NB));
    const dim3 grid((unsigned)std::min<int64_t>(tasks, device_cus()));
    if constexpr (FMT == kNvfp4) {
        if (p.d % 128 == 0) {  // whole steps
            hipLaunchKernelGGL((k_decode_fc1<FMT, P, true>), grid, dim3(kThreads), 0, s, p);
            return;
        }
    }
    hipLaunchKernelGGL((k_decode_fc1<FMT, P, false>), grid, dim3(kThreads), 0, s, p);
}
template <int FMT>
void launch_fc2(const Args& p, hipStream_t s) {
    const dim3 grid((unsigned)(p.d + 15) / 16);
    if constexpr (FMT == kNvfp4) {
        if (p.f % kWideF == 0) {
            hipLaunchKernelGGL((k_decode_fc2<FMT, true>), grid, dim3(kThreads), 0, s, p);
            return;
        }
    }
    hipLaunchKernelGGL((k_decode_fc2<FMT, false>), grid, dim3(kThreads), 0, s, p);
}
template <int FMT>
int run(const Args& p, hipStream_t s) {
    const unsigned grid = (unsigned)((p.E + 15) / 16 * ((p.T + 15) / 16) * p.parts + (FMT == kNvfp4 ? p.T : 0));
    hipLaunchKernelGGL(k_decode_router<FMT == kNvfp4>, dim3(grid), dim3(kRouterThreads), 0, s, p);
    if (p.E <= 128) launch_fc1<FMT, 2>(p, s);
    else if (p.E <= 384) launch_fc1<FMT, 6>(p, s);
    else launch_fc1<FMT, 16>(p, s);
    launch_fc2<FMT>(p, s);
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
    if (ws_bytes < carve(need, T, d, k, E, f, Fmt<FMT>::kRows, &p)) return NVQ_ERR_WORKSPACE;
    if (T == 0) return NVQ_OK;
    Carver cv(ws);
    carve(cv, T, d, k, E, f, Fmt<FMT>::kRows, &p);
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
    return carve(c, T, d, k, E, d_ff, 8, &p);
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
