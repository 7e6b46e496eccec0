// nvq_gemm16.hpp -- BF16 matrix products on the gfx950 matrix pipe, shared by
// the grouped products of the unquantized expert layer (nvq_moe16.hip) and the
// dense product with its epilogue (nvq_linear.hip).
//
// Three kernels compute out[m][n] = sum_k A(m, k) B(n, k) with bf16 operands and
// fp32 accumulation; launch_gemm16 chooses one by the sizes:
//   k_gemm16         128 x 128 tiles, two workgroups per CU (here);
//   k_gemm16_big     256 x 256 tiles in one persistent stream per CU
//                    (nvq_gemm16_big.hpp);
//   k_gemm16_skinny  FWD of a few rows per expert (nvq_gemm16_skinny.hpp).
// Operand arrangements:
//   FWD    A rows and B rows hold k contiguously (x W^T);
//   DGRAD  A as above, B holds n contiguously (g W, W as the forward keeps it);
//   WGRAD  A and B hold m and n contiguously, k runs over token rows (g^T x).
// Rows come in expert segments (or one dense block), may be gathered on the
// way in and scattered on the way out. Here too: what the kernels share, the
// loads into LDS, the fragments, the activations and the epilogues.
#pragma once

#include <type_traits>

#include "nvq_device.hpp"
#include "nvq_host.hpp"

namespace nvq {
namespace g16 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };   // operand arrangement
enum { kEpiOut = 0, kEpiAct = 1, kEpiGlu = 2 };

constexpr int kBK = 64;          // K per LDS stage

// One m-tile of the row-segmented arrangements, written by k_tile_table.
struct Tile {
    int32_t e, row0, row_end, pad;
};

struct Args {
    const uint16_t* a;
    const uint16_t* b;
    const int32_t* a_gather;  // source row of logical row r: a_gather[r] / a_div (NULL: r)
    const int32_t* b_gather;  // WGRAD only
    const int32_t* seg;       // [E + 1] (NULL: one segment [0, rows))
    const Tile* tiles;        // FWD, DGRAD with segments: [count], count at tile_count
    const int32_t* tile_count;
    const int32_t* scatter;   // destination of logical row r (NULL: r)
    void* out;
    const float* bias;
    const uint16_t* residual;
    uint16_t* z;              // saved pre-activation
    int64_t a_bytes, b_bytes; // gathered operands: bytes of the whole source (bounds the loads)
    uint32_t a_div, b_div;
    uint32_t a_mul, b_mul;    // source row of gather entry v < 2^31: div_by(v, mul, shift)
    int32_t a_shift, b_shift;
    uint32_t group_mul;       // the same for the 256 x 256 kernel's tile groups
    int32_t group_shift;
    int32_t lda, ldb;         // row strides in elements
    int32_t E, rows;          // experts; logical token rows
    int32_t M, N, K;          // WGRAD: M x N outputs; FWD, DGRAD: N columns (GLU: N outputs), K
    int32_t m_tiles, n_tiles, total;  // tiles: of an expert's rows (WGRAD), of columns, in all (segments: at most)
    int32_t out_f32, accumulate, act;
};

// ------------------------------------------------------------------ LDS staging
// 16 bytes per lane from a buffer straight into LDS at lds_addr + 16 * lane.
// A lane whose offset lies at or past the descriptor's byte count gets zeros
// (kNowhere always does): ragged rows, columns and K tails need no branch and
// contribute nothing. The instruction has no destination register; the caller
// waits with wait_vm before the barrier that publishes the stage. It is
// written out because a builtin load into LDS makes the compiler drain every
// load in flight before the next LDS read of any stage.
constexpr uint32_t kNowhere = 0xFFFFFFE0u;
constexpr int64_t kMaxBytes = 0xFFFFFE00ll;  // largest descriptor: every real offset below kNowhere

__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t off, uint32_t lds_addr) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(__builtin_amdgcn_readfirstlane((int)lds_addr)), "v"(off), "s"(rsrc)
        : "memory");
}

// The same with 4 bytes per lane.
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t off, uint32_t lds_addr) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, 0 offen lds"
        :
        : "s"(__builtin_amdgcn_readfirstlane((int)lds_addr)), "v"(off), "s"(rsrc)
        : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Buffer descriptor over [p, p + bytes), bytes clamped to [0, kMaxBytes].
__device__ __forceinline__ i32x4 make_rsrc(const void* p, int64_t bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const int64_t n = bytes < 0 ? 0 : bytes > kMaxBytes ? kMaxBytes : bytes;
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
    r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(u >> 32) & 0xFFFFu));
    r[2] = __builtin_amdgcn_readfirstlane((int)(uint32_t)n);
    r[3] = 0x00020000;
    return r;
}

typedef const __attribute__((address_space(3))) s16x8 lds_s16x8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ uint32_t lds_off(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Swizzle of a stage that holds n (or m) contiguously, R columns per k row:
// 16-byte chunk c of k row k sits at slot c ^ rkey(k). The four k rows that one
// transposing read touches per 16 lanes, and the next 16 lanes' four, then lie
// in different 32-byte bank groups.
__device__ __forceinline__ uint32_t rkey(uint32_t k) { return 2u * ((k & 3u) | ((k >> 1) & 4u)); }

// MFMA operand of 16 rows starting at row `r0` of a stage that holds k
// contiguously (128-byte rows, chunk c of row r at slot c ^ (r & 7)):
// lane l gets row l % 16, k = 32 ks + 8 (l / 16) .. + 7.
__device__ __forceinline__ bf16x8 frag_k(const uint8_t* st, int r0, int ks, int lane) {
    const int r = r0 + (lane & 15);
    const int c = ks * 4 + (lane >> 4);
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const s16x8*>(st + r * 128 + ((c ^ (r & 7)) << 4)));
}

// The same operand from a stage of R columns per k row: two transposing reads
// of four k each. Lane i of a 16-lane group passes the address of k row i / 4,
// columns 4 (i % 4) .. + 3 and receives column i of the four rows.
template <int R>
__device__ __forceinline__ bf16x8 frag_r(const uint8_t* st, int r0, int ks, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const uint32_t k = ks * 32 + 8 * g + (i >> 2);
    const uint32_t c = (uint32_t)(r0 >> 3) + ((i >> 1) & 1);
    // k + 4 has the same key
    const uint8_t* q = st + k * (R * 2) + ((c ^ rkey(k)) << 4) + ((i & 1) << 3);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)q);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(q + 4 * R * 2));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ------------------------------------------------------------------ activations
// In fp32. exp overflow gives inf and a reciprocal of 0, the limits wanted.
__device__ __forceinline__ float sigmoidf(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
// GELU's Phi by its tail: 1 - Phi(x) = exp(-x^2 / 2) R(x) for x = |v|, R = t q(t), t = 1 / (1 + 0.305 x), with q the
// polynomial of degree 7 whose largest relative error over 0 <= x <= 14.5 is least (1.0e-7; past that exp gives 0). The
// error has to be relative, since gelu(v) for v < 0 is v times this tail: in fp32 as evaluated here it is (v^2 / 2 + 16)
// 2^-23, the rounding of the exponent (4e-8 of the 2-norm on N(0, 1), as an erff). A form with an absolute error of
// 3e-7, a few operations shorter, is off by 5 % at v = -5; 8192 x 8192 x 4096 with GELU takes 470 us with it, 474 so.
struct NormTail {
    float e;     // exp(-v^2 / 2)
    float tail;  // 1 - Phi(|v|)
    __device__ __forceinline__ explicit NormTail(float v) {
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(v), 0.305f, 1.0f));
        float q = __builtin_fmaf(0.036638804f, t, -0.15274584f);
        q = __builtin_fmaf(q, t, 0.18531451f);
        q = __builtin_fmaf(q, t, -0.037620325f);
        q = __builtin_fmaf(q, t, 0.12084021f);
        q = __builtin_fmaf(q, t, 0.10347375f);
        q = __builtin_fmaf(q, t, 0.12245867f);
        q = __builtin_fmaf(q, t, 0.12164024f);
        e = __builtin_amdgcn_exp2f(-0.72134752f * (v * v));
        tail = q * t * e;
    }
    // Phi(v). For v > 0 the tail is taken from 1 here, before a product with v: v - v (1 - Phi(v)) would be inf - inf * 0.
    __device__ __forceinline__ float phi(float v) const { return v > 0.0f ? 1.0f - tail : tail; }
};
__device__ __forceinline__ float gelu_erf(float v) { return v * NormTail(v).phi(v); }
// 0.5 (1 + tanh(t)) = sigmoid(2 t)
__device__ __forceinline__ float gelu_tanh(float v) {
    return v * sigmoidf(1.5957691216057308f * (v + 0.044715f * v * v * v));
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float v) {
    if (ACT == NVQ_ACT_RELU) return v > 0.0f ? v : (v != v ? v : 0.0f);
    if (ACT == NVQ_ACT_GELU) return gelu_erf(v);
    if (ACT == NVQ_ACT_GELU_TANH) return gelu_tanh(v);
    if (ACT == NVQ_ACT_SILU) return v * sigmoidf(v);
    return v;
}

// ------------------------------------------------------------------ epilogue
__device__ __forceinline__ f32x4 load4_bf16(const uint16_t* p) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    return (f32x4){__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                   __uint_as_float(w[1] & 0xFFFF0000u)};
}
// Output position of a wave: lane l holds, of its 16 x 16 block (i, j), row
// row(i) + l % 16 and columns col(j) + 4 (l / 16) .. + 3 (the operands are
// passed to the MFMA as B, A, so a lane's four values are neighbours along n).
// Blocks come in groups of four along m, 128 rows apart, and in pairs of
// adjacent ones along n, pair_step apart (GLU: of the outputs, whose gate and
// up blocks alternate).
struct Pos {
    int64_t out_base;  // WGRAD: first element of the expert's matrix
    int row0, row_end, col0, pair_step;
    __device__ __forceinline__ int row(int i) const { return row0 + 16 * (i & 3) + 128 * (i >> 2); }
    __device__ __forceinline__ int col(int pair) const { return col0 + pair_step * pair; }
};

// Stores one row's values of an adjacent pair of blocks (columns n .. n + 31 of
// the wave; v0, v1 this lane's four of each). bf16: lanes of neighbouring
// 16-lane rows trade halves, so that each holds eight neighbouring columns: one
// 16-byte store per lane, whole 64-byte pieces per row and instruction.
// base: the row's first element. Must be called by all lanes of the four
// 16-lane rows that share an output row.
__device__ __forceinline__ void store_pair(void* out, int64_t base, int n, int N, f32x4 v0, f32x4 v1, bool f32,
                                           int lane) {
    const int g = lane >> 4;
    if (f32) {
        float* o = static_cast<float*>(out) + base;
        if (n + 4 * g < N) *reinterpret_cast<f32x4*>(o + n + 4 * g) = v0;
        if (n + 16 + 4 * g < N) *reinterpret_cast<f32x4*>(o + n + 16 + 4 * g) = v1;
        return;
    }
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const auto lo = __builtin_amdgcn_permlane16_swap(bf16x2_rne(v0[0], v0[1]), bf16x2_rne(v1[0], v1[1]), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(bf16x2_rne(v0[2], v0[3]), bf16x2_rne(v1[2], v1[3]), false, false);
    const int c = n + ((g & 1) ? 16 + 4 * (g - 1) : 4 * g);
    if (c < N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + base + c) = (u32x4){lo[0], hi[0], lo[1], hi[1]};
}

// Epilogue of a weight gradient. Every output is stored (empty experts too) and a tile's K is short, so the stores are
// half the work: 2 KiB at a time go through the wave's own LDS (16 rows of 64 bf16 or 32 fp32, 16-byte chunk c of row r
// at slot c ^ (r & 7)) so that eight neighbouring lanes hold 128 bytes of one row, bf16: twice 64. Neighbouring lanes in
// neighbouring rows, as the accumulators lie, take the CU's store path a cycle per lane (384 experts of 4096 x 1024 in
// fp32, 341 rows on average: 2.29 ms against 2.48; the products alone 1.50). A piece is read back before the one ahead of it is stored.
// `full`: all rows and columns lie inside the output.
constexpr int kRowBuf = 2048;
template <bool F32, int MF, int NF>
__device__ __forceinline__ void epilogue_wgrad(const Args& p, const f32x4 (&acc)[MF][NF], const Pos& o, uint8_t* buf,
                                               bool full, int lane) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    static_assert(NF == 4, "two pairs of blocks");
    constexpr int kPieces = F32 ? 2 * MF : MF;
    const int N = p.N, r = lane & 15, g = lane >> 4;
    const int rr = lane >> 3, c = lane & 7;  // read back: rows rr and rr + 8
    const int cc = F32 ? 4 * c : (c >> 2) * o.pair_step + 8 * (c & 3);
    const uint32_t off = (uint32_t)rr * N + cc;  // of this lane's first value from the piece's
    u32x4 w[2][2];
    auto turn = [&](int t, u32x4 (&v)[2]) {
        if constexpr (F32) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
                *reinterpret_cast<f32x4*>(buf + r * 128 + (((g + 4 * b) ^ (r & 7)) << 4)) = acc[t >> 1][2 * (t & 1) + b];
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                f32x4 a = acc[t][b];
                const int m = o.row(t) + r, n = o.col(b >> 1) + 16 * (b & 1) + 4 * g;
                if (p.accumulate && m < o.row_end && n < N)
                    a += load4_bf16(static_cast<const uint16_t*>(p.out) + o.out_base + (int64_t)m * N + n);
                *reinterpret_cast<u32x2*>(buf + r * 128 + (((2 * b + (g >> 1)) ^ (r & 7)) << 4) + (g & 1) * 8) =
                    (u32x2){bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3])};
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // one wave's LDS accesses complete in order
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = *reinterpret_cast<const u32x4*>(buf + (rr + 8 * h) * 128 + ((c ^ rr) << 4));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    turn(0, w[0]);
#pragma unroll
    for (int t = 0; t < kPieces; ++t) {
        if (t + 1 < kPieces) turn(t + 1, w[(t + 1) & 1]);
        const int i = F32 ? t >> 1 : t, n = F32 ? o.col(t & 1) : o.col0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t first = o.out_base + (int64_t)(o.row(i) + 8 * h) * N + n;
            if (full || (o.row(i) + 8 * h + rr < o.row_end && n + cc < N)) {
                if constexpr (F32) {
                    f32x4 v = __builtin_bit_cast(f32x4, w[t & 1][h]);
                    float* d = static_cast<float*>(p.out) + first + off;
                    if (p.accumulate) v += *reinterpret_cast<const f32x4*>(d);
                    *reinterpret_cast<f32x4*>(d) = v;
                } else {
                    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + first + off) = w[t & 1][h];
                }
            }
        }
    }
}

template <int EPI, int ACT, int MF, int NF>
__device__ __forceinline__ void epilogue_act(const Args& p, const f32x4 (&acc)[MF][NF], const Pos& o, int lane) {
    const int N = p.N;
    const int c4 = (lane >> 4) * 4;
    constexpr int NP = EPI == kEpiGlu ? NF / 4 : NF / 2;  // pairs of output blocks
    constexpr int CH = MF < 4 ? MF : 4;                   // rows whose residual is loaded together
#pragma unroll
    for (int i0 = 0; i0 < MF; i0 += CH) {
        u32x2 res[CH][NP][2];
        if (EPI != kEpiOut && p.residual) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int m = min(o.row(i0 + i) + (lane & 15), o.row_end - 1);
#pragma unroll
                for (int q = 0; q < NP; ++q)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        res[i][q][t] = *reinterpret_cast<const u32x2*>(p.residual + (int64_t)m * N +
                                                                       min(o.col(q) + 16 * t + c4, N - 4));
            }
        }
#pragma unroll
        for (int ii = 0; ii < CH; ++ii) {
            const int i = i0 + ii;
            const int m = o.row(i) + (lane & 15);
            if (m >= o.row_end) continue;
            const int64_t r = EPI == kEpiOut && p.scatter ? p.scatter[m] : m;
            const int64_t base = o.out_base + r * N;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const int n = o.col(q);
                f32x4 v[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int nn = n + 16 * t + c4;
                    if (EPI == kEpiOut) {
                        v[t] = acc[i][2 * q + t];
                    } else if (EPI == kEpiAct) {
                        v[t] = acc[i][2 * q + t];
                        if (p.bias) v[t] += *reinterpret_cast<const f32x4*>(p.bias + min(nn, N - 4));
                    } else {
                        f32x4 g = acc[i][4 * q + 2 * t], u = acc[i][4 * q + 2 * t + 1];
                        if (p.bias) {
                            g += *reinterpret_cast<const f32x4*>(p.bias + min(nn, N - 4));
                            u += *reinterpret_cast<const f32x4*>(p.bias + N + min(nn, N - 4));
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[t][e] = g[e] * sigmoidf(g[e]) * u[e];
                    }
                }
                if (EPI == kEpiAct) {
                    if (p.z) store_pair(p.z, base, n, N, v[0], v[1], false, lane);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[t][e] = act_fwd<ACT>(v[t][e]);
                }
                if (EPI == kEpiGlu && p.z) {
                    f32x4 g[2], u[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        g[t] = acc[i][4 * q + 2 * t];
                        u[t] = acc[i][4 * q + 2 * t + 1];
                        if (p.bias) {
                            const int nn = min(n + 16 * t + c4, N - 4);
                            g[t] += *reinterpret_cast<const f32x4*>(p.bias + nn);
                            u[t] += *reinterpret_cast<const f32x4*>(p.bias + N + nn);
                        }
                    }
                    store_pair(p.z, 2 * base, n, N, g[0], g[1], false, lane);
                    store_pair(p.z, 2 * base + N, n, N, u[0], u[1], false, lane);
                }
                if (EPI != kEpiOut && p.residual) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const u32x2 w = res[ii][q][t];
                        v[t] += (f32x4){__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
                                        __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
                    }
                }
                store_pair(p.out, base, n, N, v[0], v[1], p.out_f32, lane);
            }
        }
    }
}

// One scalar branch on the activation, outside the unrolled stores.
template <int EPI, int MF, int NF>
__device__ __forceinline__ void epilogue(const Args& p, const f32x4 (&acc)[MF][NF], const Pos& o, int lane) {
    if constexpr (EPI != kEpiAct) {
        epilogue_act<EPI, NVQ_ACT_NONE>(p, acc, o, lane);
    } else {
        switch (p.act) {
            case NVQ_ACT_RELU: epilogue_act<EPI, NVQ_ACT_RELU>(p, acc, o, lane); break;
            case NVQ_ACT_GELU: epilogue_act<EPI, NVQ_ACT_GELU>(p, acc, o, lane); break;
            case NVQ_ACT_GELU_TANH: epilogue_act<EPI, NVQ_ACT_GELU_TANH>(p, acc, o, lane); break;
            case NVQ_ACT_SILU: epilogue_act<EPI, NVQ_ACT_SILU>(p, acc, o, lane); break;
            default: epilogue_act<EPI, NVQ_ACT_NONE>(p, acc, o, lane); break;
        }
    }
}

// Scalar load of a table entry at a wave-uniform index.
template <typename T>
__device__ __forceinline__ T sload(const T* base, int64_t i) {
    typedef const __attribute__((address_space(4))) T ct;
    return ((ct*)base)[i];
}

// v / d for 0 <= v < 2^31: with 2^(s-1) < d <= 2^s and mul = floor(2^(31+s) / d) + 1 < 2^32 (host), exactly
// (v * mul) >> (31 + s); d = 1 is shift -1. (A hardware division is some twenty instructions.)
__device__ __forceinline__ uint32_t div_by(uint32_t v, uint32_t mul, int shift) {
    return shift < 0 ? v : __umulhi(v, mul) >> shift;
}

// Virtual id of a workgroup: consecutive ids on one XCD (workgroups are dealt to
// the 8 XCDs round robin), ids 0 .. n - 1 spread over all of them. -1 where the
// grid has more workgroups than ids.
__device__ __forceinline__ int xcd_id(int n) {
    const int per = (n + 7) / 8, i = (int)(blockIdx.x / 8);
    const int v = (int)(blockIdx.x % 8) * per + i;
    return i < per && v < n ? v : -1;
}

// ------------------------------------------------------------------ the kernel
// Tile TM x TN, WM x WN waves; every wave holds (TM / WM) x (TN / WN) outputs
// as 16 x 16 blocks. Two LDS stages of kBK. A step reads its whole stage into
// registers first; after a barrier the stage two steps on is fetched into its
// place, under the products of this step and all of the next. Two workgroups
// of the 128 x 128 tile share a CU and cover each other's waits. AHEAD: a step
// reads the stage after its own into a second set of registers under the first
// half of its products, and fetches the one three steps on.
template <int MODE, int EPI, int TM, int TN, int WM, int WN, bool AHEAD>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_gemm16(Args p) {
    constexpr int NW = WM * WN;
    constexpr int MF = TM / WM / 16, NF = TN / WN / 16;
    constexpr bool A_R = MODE == kWgrad, B_R = MODE != kFwd;
    constexpr int CA = TM * 8 / (64 * NW), CB = TN * 8 / (64 * NW);  // 16-byte loads per lane and stage
    constexpr int kStage = (TM + TN) * 128;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2][kStage];
    __shared__ __attribute__((aligned(16))) uint8_t rows_lds[MODE == kWgrad ? WM * WN : 1][kRowBuf];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t lds0 = lds_off(&lds[0][0]);

    const int t = xcd_id(MODE != kWgrad && p.tiles ? sload(p.tile_count, 0) * p.n_tiles : p.total);
    if (t < 0) return;
    const int nt = t % p.n_tiles, mt = t / p.n_tiles;
    int e = 0, row0, row_end;  // FWD, DGRAD: token rows; WGRAD: output rows
    int k0 = 0, klen = p.K;    // WGRAD: token rows
    if (MODE == kWgrad) {
        e = mt / p.m_tiles;
        row0 = (mt % p.m_tiles) * TM;
        row_end = p.M;
        klen = p.rows;
        if (p.seg) {
            k0 = min(max(sload(p.seg, e), 0), p.rows);
            klen = max(min(max(sload(p.seg, e + 1), 0), p.rows) - k0, 0);
        }
    } else if (p.tiles) {
        e = sload(&p.tiles[mt].e, 0);
        row0 = sload(&p.tiles[mt].row0, 0);
        row_end = sload(&p.tiles[mt].row_end, 0);
    } else {
        row0 = mt * TM;
        row_end = p.rows;
    }
    constexpr int TNO = EPI == kEpiGlu ? TN / 2 : TN;  // output columns of a tile
    const int col0 = nt * TNO;

    // ---- operand addressing: lane offsets (bytes) within a descriptor whose
    // base advances along K. Rows and columns past the tile's edge are loaded as
    // they come or as zeros: they only reach outputs that are not stored.
    const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
    uint32_t ao[A_R ? 1 : CA], bo;
    const uint16_t *abase, *bbase;
    int64_t a_lim, b_lim;       // bytes of the descriptor at k = 0
    const int kc = ((lane & 7) ^ (lane >> 3)) * 8;  // k of this lane's chunk in K-contiguous stages
    const bool ga = p.a_gather != nullptr, gb = MODE == kWgrad && p.b_gather != nullptr;
    // K-strided stage of R columns: piece i of a wave is 512 / R k rows of R / 8 chunks
    auto row_r = [&](int R, int i) { return (i * NW + wave) * (512 / R) + lane / (R / 8); };
    auto col_r = [&](int R) { return (int)((uint32_t)(lane % (R / 8)) ^ rkey(row_r(R, 0))) * 8; };
    if constexpr (!A_R) {
        abase = ga ? p.a : p.a + (int64_t)row0 * p.lda;
        a_lim = ga ? p.a_bytes : (int64_t)(row_end - row0) * lda2;
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int rl = (i * NW + wave) * 8 + (lane >> 3);
            uint32_t src = rl;
            if (ga) src = div_by((uint32_t)p.a_gather[min(row0 + rl, row_end - 1)], p.a_mul, p.a_shift);
            ao[i] = src * lda2 + kc * 2;
        }
    } else {
        abase = ga ? p.a : p.a + (int64_t)k0 * p.lda;
        a_lim = ga ? p.a_bytes : (int64_t)klen * lda2;
        ao[0] = (row0 + col_r(TM)) * 2 + (ga ? 0 : row_r(TM, 0) * lda2);
    }
    if constexpr (!B_R) {
        constexpr int rows_per = EPI == kEpiGlu ? 2 : 1;
        bbase = p.b + ((int64_t)e * rows_per * p.N + col0) * p.ldb;
        b_lim = ((int64_t)rows_per * p.N - col0) * ldb2;
        const int r = wave * 8 + (lane >> 3);
        // GLU: blocks of 16: gate, up, gate, up, ...
        bo = (uint32_t)(EPI == kEpiGlu ? ((r >> 4) & 1) * p.N + (r >> 5) * 16 + (r & 15) : r) * ldb2 + kc * 2;
    } else {
        bbase = gb ? p.b : p.b + (MODE == kDgrad ? (int64_t)e * p.K : (int64_t)k0) * p.ldb;
        b_lim = gb ? p.b_bytes : (int64_t)klen * ldb2;
        bo = (col0 + col_r(TN)) * 2 + (gb ? 0 : row_r(TN, 0) * ldb2);
    }
    if (MODE == kWgrad && p.accumulate && klen == 0) return;  // old + 0 would turn -0 into +0
    const int nk = (klen + kBK - 1) / kBK;
    // K-strided pieces: by row number, or through a gather (its entries by scalar loads)
    auto issue_r = [&](auto R_tag, const uint16_t* base, int64_t lim, uint32_t o, int ld, bool gat,
                       const int32_t* gather, uint32_t mul, int shift, int k, uint32_t dst) {
        constexpr int R = decltype(R_tag)::value, n = R * 8 / (64 * NW), per = 512 / R;
        const uint32_t ld2 = (uint32_t)ld * 2u;
        const i32x4 r = gat ? make_rsrc(base, lim) : make_rsrc(base + (int64_t)k * ld, lim - (int64_t)k * ld2);
        const int q = lane / (R / 8);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            uint32_t off = o + i * NW * per * ld2;
            if (gat) {
                const int kl = k + (i * NW + wave) * per;
                uint32_t v = (uint32_t)sload(gather, k0 + min(kl, klen - 1));
#pragma unroll
                for (int u = 1; u < per; ++u) {
                    const uint32_t w = (uint32_t)sload(gather, k0 + min(kl + u, klen - 1));
                    v = q == u ? w : v;
                }
                off = kl + q < klen ? div_by(v, mul, shift) * ld2 + o : kNowhere;
            }
            dma16(r, off, dst + (i * NW + wave) * 1024);
        }
    };
    auto issue = [&](int s) {
        const uint32_t la = lds0 + (s & 1) * kStage, lb = la + TM * 128;
        const int k = s * kBK;
        const bool in_k = k + kc < klen;
        if constexpr (!A_R) {
            const i32x4 r = make_rsrc(abase + k, a_lim - (int64_t)k * 2);
#pragma unroll
            for (int i = 0; i < CA; ++i) dma16(r, in_k ? ao[i] : kNowhere, la + (i * NW + wave) * 1024);
        } else {
            issue_r(std::integral_constant<int, TM>{}, abase, a_lim, ao[0], p.lda, ga, p.a_gather, p.a_mul, p.a_shift, k,
                    la);
        }
        if constexpr (!B_R) {
            const i32x4 r = make_rsrc(bbase + k, b_lim - (int64_t)k * 2);
            constexpr int step = EPI == kEpiGlu ? NW * 4 : NW * 8;  // rows of w between pieces
#pragma unroll
            for (int i = 0; i < CB; ++i) dma16(r, in_k ? bo + i * step * ldb2 : kNowhere, lb + (i * NW + wave) * 1024);
        } else {
            issue_r(std::integral_constant<int, TN>{}, bbase, b_lim, bo, p.ldb, gb, p.b_gather, p.b_mul, p.b_shift, k, lb);
        }
    };

    f32x4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

    if (nk > 0) issue(0);
    if (nk > 1) issue(1);
    struct Frags {
        bf16x8 a[2][MF], b[2][NF];
    };
    auto read = [&](Frags& f, int s) {
        const uint8_t* sa = lds[s & 1];
        const uint8_t* sb = sa + TM * 128;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const int r0 = wn * (TN / WN) + 16 * j;
                if constexpr (B_R) f.b[ks][j] = frag_r<TN>(sb, r0, ks, lane);
                else f.b[ks][j] = frag_k(sb, r0, ks, lane);
            }
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const int r0 = wm * (TM / WM) + 16 * i;
                if constexpr (A_R) f.a[ks][i] = frag_r<TM>(sa, r0, ks, lane);
                else f.a[ks][i] = frag_k(sa, r0, ks, lane);
            }
        }
    };
    auto mul = [&](const Frags& f, int ks) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[ks][j], f.a[ks][i], acc[i][j], 0, 0, 0);
    };
    // this wave's loads of stage s have landed, those of stage s + 1 may be under way
    auto landed = [&](int s) {
        if (s + 1 < nk) wait_vm<CA + CB>();
        else wait_vm<0>();
        stage_barrier();
    };
    constexpr int kReads = (A_R ? 4 : 2) * MF + (B_R ? 4 : 2) * NF, kMuls = MF * NF;
    auto step = [&](int s, const Frags& f, Frags& next) {
        landed(s + 1);
        read(next, s + 1);
        mul(f, 0);
#pragma unroll
        for (int r = 0; r < kMuls; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x100, kReads / kMuls, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (s + 3 < nk) {
            stage_barrier();
            issue(s + 3);
        }
        __builtin_amdgcn_sched_barrier(0);
        mul(f, 1);
    };
    if constexpr (!AHEAD) {
        for (int s = 0; s < nk; ++s) {
            Frags f;
            landed(s);
            read(f, s);
            if (s + 2 < nk) {
                stage_barrier();
                issue(s + 2);
            }
            mul(f, 0);
            mul(f, 1);
        }
    } else if (nk > 0) {
        Frags x, y;
        landed(0);
        read(x, 0);
        if (nk > 2) {
            stage_barrier();
            issue(2);
        }
        for (int s = 0; s + 1 < nk; s += 2) {
            step(s, x, y);
            if (s + 2 < nk) step(s + 1, y, x);
            else x = y;
        }
        mul(x, 0);
        mul(x, 1);
    }
    Pos o;
    o.out_base = MODE == kWgrad ? (int64_t)e * p.M * p.N : 0;
    o.row0 = row0 + wm * (TM / WM);
    o.row_end = row_end;
    o.col0 = col0 + wn * (TNO / WN);
    o.pair_step = 32;
    if constexpr (MODE == kWgrad) {
        const bool full = o.row0 + TM / WM <= o.row_end && o.col0 + TN / WN <= p.N;
        if (p.out_f32) epilogue_wgrad<true>(p, acc, o, rows_lds[wave], full, lane);
        else epilogue_wgrad<false>(p, acc, o, rows_lds[wave], full, lane);
    } else {
        epilogue<EPI>(p, acc, o, lane);
    }
}

}  // namespace g16

// Launches the product described by `p` (operands, sizes, epilogue; tiles and
// tile counts are filled in here). `ws` holds gemm16_ws_bytes for segmented
// FWD and DGRAD. mode is g16::kFwd, kDgrad or kWgrad.
void launch_gemm16(int mode, int epi, g16::Args p, void* ws, hipStream_t s);
size_t gemm16_ws_bytes(int64_t rows, int64_t E);
// Whether every tile count and lane offset of the product fits (see the limits in nvq.h).
bool gemm16_dims_ok(int mode, bool glu, int64_t rows, int64_t E, int64_t M, int64_t N, int64_t K);

}  // namespace nvq
