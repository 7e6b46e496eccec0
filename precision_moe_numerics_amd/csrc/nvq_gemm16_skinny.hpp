// nvq_gemm16_skinny.hpp -- the BF16 forward products for a few rows per expert
// (single tokens being served), which are bound by reading the weights once.
#pragma once

#include "nvq_gemm16.hpp"

namespace nvq {
namespace g16 {

constexpr int kSkWaves = 8;   // waves of a workgroup: KS parts of K x 8 / KS blocks of weight rows
constexpr int kSkBatch = 8;   // 32-deep steps whose loads are in flight together

// Expert and first row of m-tile `t` of the segments (tm rows each), by one
// wave: lane l counts the tiles of its ceil(E / 64) neighbouring experts, a
// prefix sum over the lanes finds the lane, then its experts are walked. Offsets
// are clamped as in k_tile_table. False past the last tile.
__device__ __forceinline__ bool find_tile(const int32_t* seg, int E, int rows, int tm, int t, int lane, int* e_out,
                                          int* row0, int* row_end) {
    const int per = (E + 63) / 64, e0 = lane * per;
    auto off = [&](int e) { return min(max(seg[min(e, E)], 0), rows); };
    int n = 0, prev = off(e0);
    for (int j = 1; j <= per; ++j) {
        const int cur = off(e0 + j);
        n += (max(cur - prev, 0) + tm - 1) / tm;
        prev = cur;
    }
    int sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d, 64);
        sum += lane >= d ? v : 0;
    }
    const uint64_t past = __ballot(sum > t);
    if (past == 0) return false;
    const int src = __builtin_ctzll(past);
    int left = t - __shfl(sum - n, src, 64);
    int e = src * per;
    for (;;) {
        const int lo = off(e), hi = max(off(e + 1), lo);
        const int tiles = (hi - lo + tm - 1) / tm;
        if (left < tiles) {
            *e_out = __builtin_amdgcn_readfirstlane(e);
            *row0 = __builtin_amdgcn_readfirstlane(lo + left * tm);
            *row_end = __builtin_amdgcn_readfirstlane(hi);
            return true;
        }
        left -= tiles;
        ++e;
    }
}

// One workgroup: 8 / KS blocks of 16 rows of the weights (GLU: of 8 gate rows
// and their 8 up rows) times up to 16 MB rows of one expert. Each wave takes one
// block and a contiguous part of K and loads both operands as MFMA fragments
// straight into registers, a batch of steps at once, the weights past the
// caches (they are read once); rows of x that do not exist cost no traffic. The
// sums of the KS parts meet in LDS and are added in order.
template <int EPI, int MB, int KS, bool I8>
__global__ __launch_bounds__(64 * kSkWaves) void k_gemm16_skinny(Args p) {
    using Sum = std::conditional_t<I8, int, float>;
    __shared__ Sum red[kSkWaves][MB][16][17];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int nt = blockIdx.x % p.n_tiles, mt = blockIdx.x / p.n_tiles;
    int e = 0, row0 = mt * 16 * MB, row_end = p.rows;
    if (p.seg && !find_tile(p.seg, p.E, p.rows, 16 * MB, mt, lane, &e, &row0, &row_end)) return;
    constexpr int TNO = EPI == kEpiGlu ? 8 : 16, NB = kSkWaves / KS;
    const int part_k = wave % KS;
    const int n_first = nt * TNO * NB;
    const int n0 = n_first + wave / KS * TNO;
    const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
    const int r = lane & 15, kc = (lane >> 4) * 8;
    constexpr int rows_per = EPI == kEpiGlu ? 2 : 1;
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p.b + (int64_t)e * rows_per * p.N * p.ldb), 0, (int)((uint32_t)(rows_per * p.N) * ldb2),
        0x00020000);
    const int brow = EPI == kEpiGlu ? (r < 8 ? n0 + r : p.N + n0 + r - 8) : n0 + r;
    const bool b_ok = n0 + (EPI == kEpiGlu ? 0 : r) < p.N;
    const uint32_t bo = (uint32_t)brow * ldb2 + kc * 2;
    const bool gat = p.a_gather != nullptr;
    const uint16_t* abase = gat ? p.a : p.a + (int64_t)row0 * p.lda;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(abase), 0, gat ? (int)(uint32_t)p.a_bytes : (int)((uint32_t)min(row_end - row0, 16 * MB) * lda2),
        0x00020000);
    uint32_t ao[MB];
    bool a_ok[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int m = row0 + 16 * i + r;
        a_ok[i] = m < row_end;
        uint32_t src = 16 * i + r;
        if (gat) src = div_by((uint32_t)p.a_gather[min(m, row_end - 1)], p.a_mul, p.a_shift);
        ao[i] = src * lda2 + kc * 2;
    }
    const int steps = (p.K + 31) / 32;
    const int part = ((steps + KS - 1) / KS + 1) & ~1;  // even: whole 128-byte lines
    const int s_end = min((part_k + 1) * part, steps);
    Acc<I8> acc[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[i] = (Acc<I8>){0, 0, 0, 0};
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    for (int s0 = part_k * part; s0 < s_end; s0 += kSkBatch) {
        u32x4 bv[kSkBatch], av[kSkBatch][MB];
#pragma unroll
        for (int j = 0; j < kSkBatch; ++j) {
            const int k = (s0 + j) * 32;
            const bool ok = s0 + j < s_end && k + kc < p.K;
            bv[j] = __builtin_amdgcn_raw_buffer_load_b128(rb, ok && b_ok ? bo + k * 2 : kNowhere, 0, 2);
#pragma unroll
            for (int i = 0; i < MB; ++i)
                av[j][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, ok && a_ok[i] ? ao[i] + k * 2 : kNowhere, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kSkBatch; ++j)
#pragma unroll
            for (int i = 0; i < MB; ++i)
                acc[i] = mfma64<I8>(__builtin_bit_cast(bf16x8, bv[j]), __builtin_bit_cast(bf16x8, av[j][i]), acc[i]);
    }
    // lane: columns 4 (lane / 16) + t of row lane % 16
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) red[wave][i][4 * (lane >> 4) + t][r] = acc[i][t];
    __syncthreads();
    auto total = [&](int b, int i, int n, int m) {
        Sum s = red[b * KS][i][n][m];
#pragma unroll
        for (int w = 1; w < KS; ++w) s += red[b * KS + w][i][n][m];
        return (float)s;
    };
    auto put = [&](void* out, int64_t idx, float v, bool f32) {
        if (f32) static_cast<float*>(out)[idx] = v;
        else static_cast<uint16_t*>(out)[idx] = (uint16_t)bf16x2_rne(v, v);
    };
    for (int u = threadIdx.x; u < MB * 16 * TNO * NB; u += 64 * kSkWaves) {
        const int nn = u % (TNO * NB), b = nn / TNO, n = nn % TNO;
        const int m16 = u / (TNO * NB), i = m16 >> 4, mr = m16 & 15;
        const int m = row0 + m16, col = n_first + nn;
        if (m >= row_end || col >= p.N) continue;
        const int64_t base = (EPI == kEpiOut && p.scatter ? (int64_t)p.scatter[m] : m) * p.N;
        float v = total(b, i, n, mr);
        const float* bs = I8 ? p.b_scale + (int64_t)e * rows_per * p.N + col : nullptr;
        const float xs = I8 ? row_scale(p, m) : 1.0f;
        if (I8) v = v * xs * bs[0];
        if (EPI == kEpiAct) {
            if (p.bias) v += p.bias[col];
            if (p.z) put(p.z, base + col, v, false);
            switch (p.act) {
                case NVQ_ACT_RELU: v = act_fwd<NVQ_ACT_RELU>(v); break;
                case NVQ_ACT_GELU: v = act_fwd<NVQ_ACT_GELU>(v); break;
                case NVQ_ACT_GELU_TANH: v = act_fwd<NVQ_ACT_GELU_TANH>(v); break;
                case NVQ_ACT_SILU: v = act_fwd<NVQ_ACT_SILU>(v); break;
                default: break;
            }
        } else if (EPI == kEpiGlu) {
            float g = v, up = total(b, i, n + 8, mr);
            if (I8) up = up * xs * bs[p.N];
            if (p.bias) {
                g += p.bias[col];
                up += p.bias[p.N + col];
            }
            if (p.z) {
                put(p.z, 2 * base + col, g, false);
                put(p.z, 2 * base + p.N + col, up, false);
            }
            v = g * sigmoidf(g) * up;
        }
        if (EPI != kEpiOut && p.residual) v += bf16_to_f32(p.residual[base + col]);
        put(p.out, base + col, v, p.out_f32);
    }
}

}  // namespace g16
}  // namespace nvq
