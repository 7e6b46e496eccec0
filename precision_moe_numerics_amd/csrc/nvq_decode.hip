// nvq_decode.hip -- a whole mixture-of-experts layer for a few tokens (up to
// 64, single tokens being decoded): router, chosen experts and weighted combine
// on bf16, int8 or NVFP4 weights.
//
//   logits = x Wr^T                       k_decode_router
//   ids, weights = top-k of the logits;
//   h = silu(g) * u of every (expert, token) pair   k_decode_fc1
//   out = residual + sum_s weight * (W2 h)          k_decode_fc2
//
// Bound by reading the chosen experts' weights once. The activations stay bf16
// in all three formats: they are a few rows, and quantizing them would save
// nothing. A weight reaches the matrix pipe as a bf16 value that holds it
// exactly (int8 codes have 8 significant bits, e2m1 * e4m3 has 6); the channel's
// or tensor's fp32 scale is applied to the fp32 sum. h is rounded to bf16, the
// matrix pipe's type, once.
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
constexpr int64_t kMaxBytes = 0xFFFFFE00ll;

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
    double* logits;           // [T, E]
    uint16_t* h;              // [T k, f], rows in expert order
    int T, d, E, k, f, sigmoid;
};

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

// Fragment i (8 values) of 16 bytes of weights, in bf16.
template <int FMT>
__device__ __forceinline__ bf16x8 decode(const W16& w, int i) {
    if constexpr (FMT == kBf16) {
        return __builtin_bit_cast(bf16x8, w.w);
    } else if constexpr (FMT == kInt8) {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t p = w.w[2 * i + (j >> 1)] >> (16 * (j & 1));
            const float a = (float)(int8_t)(p & 0xFFu), b = (float)(int8_t)((p >> 8) & 0xFFu);
            o[j] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);  // exact: the upper halves
        }
        return __builtin_bit_cast(bf16x8, o);
    } else {
        const auto s2 = e4m3_pair_to_f32(w.sc);
        const float s = s2[i >> 1];
        u32x4 o;
        auto put = [&](int j, nvq_f32x2 v) {
            o[j] = __builtin_amdgcn_perm(__float_as_uint(v[1] * s), __float_as_uint(v[0] * s), 0x07060302u);
        };
        put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.w[i], 1.0f, 0));
        put(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.w[i], 1.0f, 1));
        put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.w[i], 1.0f, 2));
        put(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.w[i], 1.0f, 3));
        return __builtin_bit_cast(bf16x8, o);
    }
}

template <int FMT>
__device__ __forceinline__ f32x4 product(const W16& w, const X16<FMT>& x, f32x4 acc) {
#pragma unroll
    for (int i = 0; i < Fmt<FMT>::kFrags; ++i)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode<FMT>(w, i), __builtin_bit_cast(bf16x8, x.v[i]), acc, 0, 0, 0);
    return acc;
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

// ------------------------------------------------------------------ router logits
// One workgroup: 16 experts, 16 tokens, K over the waves. The sum of 32 products that one instruction adds is rounded
// to fp32, 2^-24 of it; from there on the sums are fp64, so that of two close logits the larger one is chosen.
__global__ __launch_bounds__(kThreads, 2) void k_decode_router(Args p) {
    __shared__ double red[kWaves][16][17];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    const uint32_t rb = (uint32_t)p.d * 2u;
    const auto wr = rsrc(p.wr, (uint32_t)p.E * rb), xr = rsrc(p.x, (uint32_t)p.T * rb);
    const int steps = (p.d + 31) / 32, part = (steps + kWaves - 1) / kWaves;
    const int s1 = min((wave + 1) * part, steps);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int s0 = wave * part; s0 < s1; s0 += 8) {
        u32x4 w[8], x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t o = (uint32_t)(s0 + j) * 64 + q * 16;
            const bool ok = s0 + j < s1 && o < rb;
            w[j] = __builtin_amdgcn_raw_buffer_load_b128(wr, ok && e0 + r < p.E ? (e0 + r) * rb + o : kNowhere, 0, 0);
            x[j] = __builtin_amdgcn_raw_buffer_load_b128(xr, ok && t0 + r < p.T ? (t0 + r) * rb + o : kNowhere, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
            const f32x4 a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[j]),
                                                                    __builtin_bit_cast(bf16x8, x[j]), z, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += (double)a[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r][4 * q + i] = acc[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int e = threadIdx.x & 15, t = threadIdx.x >> 4;
        double v = red[0][t][e];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][t][e];
        if (e0 + e < p.E && t0 + t < p.T) p.logits[(int64_t)(t0 + t) * p.E + e0 + e] = v;
    }
}

// ------------------------------------------------------------------ the choice
// Ids and weights of token t by one wave, as the routers choose (logits in fp64): lane j < k returns the j-th.
// P: expert slots per lane. Non-finite logits order somehow; the ids stay distinct and in range.
template <int P>
__device__ __forceinline__ void choose(const Args& p, int t, int lane, int* id, float* weight) {
    const double* lt = p.logits + (int64_t)t * p.E;
    auto score = [&](double l) { return p.sigmoid ? 1.0 / (1.0 + exp(-l)) : l; };
    uint64_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int e = lane + 64 * j;
        key[j] = 0;  // below the key of every number
        if (e < p.E) {
            const double v = score(lt[e]) + (p.bias ? (double)p.bias[e] : 0.0);
            key[j] = order_key(v == v ? v : -__builtin_inf());
        }
    }
    int mine = 0;
    for (int r = 0; r < p.k; ++r) {
        uint64_t bk = 0;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const bool gt = key[j] > bk;  // strict: the lowest slot among equal keys stays
            bk = gt ? key[j] : bk;
            bj = gt ? j : bj;
        }
        int be = bk ? lane + 64 * bj : 0x7FFFFFFF;
        group_argmax<64>(bk, be);
        if ((be & 63) == lane) {
#pragma unroll
            for (int j = 0; j < P; ++j) key[j] = j == be / 64 ? 0 : key[j];
        }
        mine = lane == r ? be : mine;
    }
    const bool chosen = lane < p.k;
    const double l = chosen ? lt[mine] : -__builtin_inf();
    double v;
    if (p.sigmoid) {
        v = chosen ? score(l) : 0.0;
    } else {
        double m = l;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) m = fmax(m, __shfl_xor(m, off, 64));
        v = chosen ? exp(l - m) : 0.0;
    }
    double sum = 0.0;
    for (int j = 0; j < p.k; ++j) sum += __shfl(v, j, 64);
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
    float wt[kMaxA];
    uint8_t tok[kMaxA];
    int32_t scan[2][kWaves];
};
// From ids and weights (global, as another launch or `choose` of this workgroup left them). All threads take part;
// returns the number of blocks.
__device__ __forceinline__ int build(Table& tb, const Args& p, const int32_t* ids, const float* weights) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int A = p.T * p.k;
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
    if (lane == 63) tb.scan[0][wave] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int v = tb.scan[0][w];
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
    }
    __syncthreads();
    return total >> 16;
}

// ------------------------------------------------------------------ fc1 + SwiGLU
// A task is one block of tokens and NB groups of 8 gate rows and their 8 up rows; KS waves share a group's K. Every
// workgroup walks tasks blockIdx.x, + gridDim.x, ...; the sums of the KS parts meet in LDS and are added in order.
template <int FMT, int P>
__global__ __launch_bounds__(kThreads, 2) void k_decode_fc1(Args p) {
    constexpr int NB = FMT == kBf16 ? 1 : FMT == kInt8 ? 2 : 4, KS = kWaves / NB, D = FMT == kNvfp4 ? 4 : 8;
    __shared__ Table tb;
    __shared__ float red[2][kWaves][16][17];
    __shared__ int32_t ids_lds[kMaxA];
    __shared__ float w_lds[kMaxA];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    for (int t = wave; t < p.T; t += kWaves) {
        int id;
        float w;
        choose<P>(p, t, lane, &id, &w);
        if (lane < p.k) {
            ids_lds[t * p.k + lane] = id;
            w_lds[t * p.k + lane] = w;
            if (blockIdx.x == 0) {
                p.ids[t * p.k + lane] = id;
                p.weights[t * p.k + lane] = w;
            }
        }
    }
    __syncthreads();
    const int V = build(tb, p, ids_lds, w_lds);
    const int JB = (p.f + 8 * NB - 1) / (8 * NB);
    const auto xr = rsrc(p.x, (uint32_t)p.T * (uint32_t)p.d * 2u);
    const uint32_t rb = Fmt<FMT>::row_bytes(p.d);
    const int steps = (int)(rb + 63) / 64, part = (steps + KS - 1) / KS;
    const int s_first = wave % KS * part, s_end = min(s_first + part, steps);
    int flip = 0;
    for (int task = blockIdx.x; task < V * JB; task += gridDim.x) {
        const Block b = tb.blocks[task / JB];
        const int e = __builtin_amdgcn_readfirstlane((int)b.e), n = __builtin_amdgcn_readfirstlane(b.n);
        const int row0 = __builtin_amdgcn_readfirstlane((int)b.row0), c0 = task % JB * 8 * NB;
        const Matrix<FMT> m(p.w1, p.s1, e, 2 * p.f, p.d);
        const int col = c0 + wave / KS * 8 + (r & 7);
        const uint32_t wrow = r < 8 ? col : p.f + col;
        const bool w_ok = col < p.f, x_ok = r < n;
        const uint32_t xrow = x_ok ? tb.tok[row0 + r] : 0;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = s_first; s0 < s_end; s0 += D) {
            W16 w[D];
            X16<FMT> x[D];
#pragma unroll
            for (int j = 0; j < D; ++j) {
                const uint32_t o = (uint32_t)(s0 + j) * 64 + q * 16;
                const bool ok = s0 + j < s_end && o < rb;
                w[j] = m.load(wrow, o, ok && w_ok);
                x[j] = load_x<FMT>(xr, xrow, p.d, o, ok && x_ok);
            }
#pragma unroll
            for (int j = 0; j < D; ++j) acc = product<FMT>(w[j], x[j], acc);
        }
        // lane: rows 4 q + i of the group (gate 0 .. 7, up 8 .. 15), token r
#pragma unroll
        for (int i = 0; i < 4; ++i) red[flip][wave][r][4 * q + i] = acc[i];
        __syncthreads();
        if (threadIdx.x < 16 * 8 * NB) {
            const int cc = threadIdx.x % (8 * NB), i = threadIdx.x / (8 * NB), g8 = cc / 8, j = cc % 8;
            if (i < n && c0 + cc < p.f) {
                float g = red[flip][g8 * KS][i][j], u = red[flip][g8 * KS][i][8 + j];
#pragma unroll
                for (int w = 1; w < KS; ++w) {
                    g += red[flip][g8 * KS + w][i][j];
                    u += red[flip][g8 * KS + w][i][8 + j];
                }
                if (FMT == kInt8) {
                    const float* s = static_cast<const float*>(p.s1) + (int64_t)e * 2 * p.f + c0 + cc;
                    g *= s[0];
                    u *= s[p.f];
                } else if (FMT == kNvfp4) {
                    g *= p.t1[e];
                    u *= p.t1[e];
                }
                const float h = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
                p.h[(int64_t)(row0 + i) * p.f + c0 + cc] = (uint16_t)bf16x2_rne(h, h);
            }
        }
        flip ^= 1;  // (the next task's sums go to the other half while slow threads still read this one)
    }
}

// ------------------------------------------------------------------ fc2 + combine
// A workgroup owns 16 columns of out. Its waves share the (block, K step) pairs of all chosen experts in equal
// contiguous runs; where a run leaves a block, the wave adds weight * sum to its own token rows in LDS. The waves' rows
// are added in order at the end.
template <int FMT>
__global__ __launch_bounds__(kThreads, 2) void k_decode_fc2(Args p) {
    constexpr int D = FMT == kNvfp4 ? 4 : 8;
    __shared__ Table tb;
    __shared__ float red[kWaves][kMaxT][17];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    for (int i = threadIdx.x; i < kWaves * kMaxT * 17; i += kThreads) (&red[0][0][0])[i] = 0.0f;
    const int V = build(tb, p, p.ids, p.weights);
    const int n0 = blockIdx.x * 16;
    const auto hr = rsrc(p.h, (uint32_t)(p.T * p.k) * (uint32_t)p.f * 2u);
    const uint32_t rb = Fmt<FMT>::row_bytes(p.f);
    const int S = (int)(rb + 63) / 64;
    const int total = V * S, part = (total + kWaves - 1) / kWaves;
    const int first = min(wave * part, total), end = min(first + part, total);
    const bool w_ok = n0 + r < p.d;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    int lv = first / S, ls = first - lv * S;  // load position
    int cv = lv, cs = ls;                     // product position
    for (int i0 = first; i0 < end; i0 += D) {
        W16 w[D];
        X16<FMT> x[D];
#pragma unroll
        for (int j = 0; j < D; ++j) {
            const bool live = i0 + j < end;
            const Block b = tb.blocks[live ? lv : 0];
            const int e = __builtin_amdgcn_readfirstlane((int)b.e), n = __builtin_amdgcn_readfirstlane(b.n);
            const int row0 = __builtin_amdgcn_readfirstlane((int)b.row0);
            const Matrix<FMT> m(p.w2, p.s2, e, p.d, p.f);
            const uint32_t o = (uint32_t)ls * 64 + q * 16;
            const bool ok = live && o < rb;
            w[j] = m.load((uint32_t)(n0 + r), o, ok && w_ok);
            x[j] = load_x<FMT>(hr, (uint32_t)(row0 + r), p.f, o, ok && r < n);
            if (++ls == S) {
                ls = 0;
                ++lv;
            }
        }
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i0 + j >= end) break;
            acc = product<FMT>(w[j], x[j], acc);
            if (++cs == S || i0 + j + 1 == end) {
                const Block b = tb.blocks[cv];
                if (r < b.n) {
                    const float wt = tb.wt[b.row0 + r];
                    float* o = red[wave][tb.tok[b.row0 + r]] + 4 * q;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = acc[i];
                        if (FMT == kInt8) {
                            const int c = min(n0 + 4 * q + i, p.d - 1);
                            v *= static_cast<const float*>(p.s2)[(int64_t)b.e * p.d + c];
                        } else if (FMT == kNvfp4) {
                            v *= p.t2[b.e];
                        }
                        o[i] = __builtin_fmaf(wt, v, o[i]);
                    }
                }
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
        float v = red[0][t][c];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][t][c];
        const int64_t at = (int64_t)t * p.d + n0 + c;
        if (p.residual) v += bf16_to_f32(p.residual[at]);
        p.out[at] = (uint16_t)bf16x2_rne(v, v);
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
           E * d * 2 <= kMaxBytes && T * k * f * 2 <= kMaxBytes;
}
size_t carve(Carver& c, int64_t T, int k, int64_t E, int64_t f, Args* p) {
    p->logits = c.take<double>((size_t)(T * E));
    p->h = c.take<uint16_t>((size_t)(T * k * f));
    return c.need;
}

template <int FMT, int P>
void launch_fc1(const Args& p, hipStream_t s) {
    constexpr int NB = FMT == kBf16 ? 1 : FMT == kInt8 ? 2 : 4;
    const int64_t tasks = (int64_t)std::min(p.T * p.k, p.E + p.T * p.k / 16) * ((p.f + 8 * NB - 1) / (8 * NB));
    const unsigned grid = (unsigned)std::min<int64_t>(tasks, device_cus());
    hipLaunchKernelGGL((k_decode_fc1<FMT, P>), dim3(grid), dim3(kThreads), 0, s, p);
}
template <int FMT>
int run(const Args& p, hipStream_t s) {
    hipLaunchKernelGGL(k_decode_router, dim3((unsigned)(p.E + 15) / 16, (unsigned)(p.T + 15) / 16), dim3(kThreads), 0, s, p);
    if (p.E <= 128) launch_fc1<FMT, 2>(p, s);
    else if (p.E <= 512) launch_fc1<FMT, 8>(p, s);
    else launch_fc1<FMT, 16>(p, s);
    hipLaunchKernelGGL(k_decode_fc2<FMT>, dim3((unsigned)(p.d + 15) / 16), dim3(kThreads), 0, s, p);
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
    if (ws_bytes < carve(need, T, k, E, f, &p)) return NVQ_ERR_WORKSPACE;
    if (T == 0) return NVQ_OK;
    Carver cv(ws);
    carve(cv, T, k, E, f, &p);
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
    (void)d;
    if (T < 0 || T > kMaxT || k < 1 || k > kMaxK || E < 1 || E > kMaxE || d_ff < 0 || d_ff > (1 << 22)) return 0;
    Carver c(nullptr);
    Args p{};
    return carve(c, T, k, E, d_ff, &p);
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
