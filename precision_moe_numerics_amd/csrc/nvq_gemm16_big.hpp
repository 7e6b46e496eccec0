// nvq_gemm16_big.hpp -- the persistent 256 x 256 form of the BF16 products.
#pragma once

#include "nvq_gemm16.hpp"

#include <type_traits>

namespace nvq {
namespace g16 {

constexpr int kBigT = 256;                    // output tile: 256 x 256
constexpr int kBigK = 32;                     // K of one LDS stage
constexpr int kBigStages = 4;
constexpr int kBigOp = kBigT * kBigK * 2;     // 16 KiB per operand and stage
constexpr int kBigStage = 2 * kBigOp;
constexpr int kBigWaves = 8;                  // 2 (m) x 4 (n), each 128 x 64

// Operand of 16 rows from a stage that holds k contiguously: 64-byte rows, chunk
// c of row r at slot c ^ ((r >> 1) & 3). One read covers 16 whole rows; the
// eight lanes served together touch eight different 16-byte bank groups.
__device__ __forceinline__ uint32_t bkey(uint32_t r) { return (r >> 1) & 3u; }
__device__ __forceinline__ bf16x8 big_frag_k(const uint8_t* st, int r0, int lane) {
    const uint32_t r = lane & 15, c = lane >> 4;
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const s16x8*>(st + r0 * 64 + r * 64 + ((c ^ bkey(r)) << 4)));
}

// A tile of the stream (wave-uniform).
struct BigTile {
    int e, row0, row_end, col0, k0, klen;
};

template <int MODE, int EPI>
__device__ __forceinline__ BigTile big_tile(const Args& p, int t) {
    constexpr int TNO = EPI == kEpiGlu ? kBigT / 2 : kBigT;
    BigTile T;
    const int mt = t / p.n_tiles;
    T.col0 = (t % p.n_tiles) * TNO;
    T.k0 = 0;
    T.klen = p.K;
    T.e = 0;
    if (MODE == kWgrad) {
        T.e = mt / p.m_tiles;
        T.row0 = (mt % p.m_tiles) * kBigT;
        T.row_end = p.M;
        T.klen = p.rows;
        if (p.seg) {
            T.k0 = min(max(sload(p.seg, T.e), 0), p.rows);
            T.klen = max(min(max(sload(p.seg, T.e + 1), 0), p.rows) - T.k0, 0);
        }
    } else if (p.tiles) {
        T.e = sload(&p.tiles[mt].e, 0);
        T.row0 = sload(&p.tiles[mt].row0, 0);
        T.row_end = sload(&p.tiles[mt].row_end, 0);
    } else {
        T.row0 = mt * kBigT;
        T.row_end = p.rows;
    }
    return T;
}

// The loader's view of the tile it is fetching: descriptor bases at k = 0 and
// this lane's offsets for its two 16-byte pieces of each operand and stage.
template <int MODE, int EPI>
struct BigLoad {
    const uint16_t *abase, *bbase;
    int64_t a_lim, b_lim;
    uint32_t ao[2], bo[2];
    int klen, k0;

    __device__ __forceinline__ void set(const Args& p, const BigTile& T, int wave, int lane) {
        constexpr bool A_R = MODE == kWgrad, B_R = MODE != kFwd;
        const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
        const int kc = (int)((lane & 3) ^ bkey(lane >> 2)) * 16;  // bytes of this lane's chunk within a 64-byte row
        klen = T.klen;
        k0 = T.k0;
        if constexpr (!A_R) {
            const bool gat = p.a_gather != nullptr;
            abase = gat ? p.a : p.a + (int64_t)T.row0 * p.lda;
            a_lim = gat ? p.a_bytes : (int64_t)(T.row_end - T.row0) * lda2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rl = (i * kBigWaves + wave) * 16 + (lane >> 2);
                const bool ok = T.row0 + rl < T.row_end;
                uint32_t src = rl;
                if (gat) src = (uint32_t)p.a_gather[ok ? T.row0 + rl : T.row0] / p.a_div;
                ao[i] = ok ? src * lda2 + kc : kNowhere;
            }
        } else {
            abase = p.a_gather ? p.a : p.a + (int64_t)T.k0 * p.lda;
            a_lim = p.a_gather ? p.a_bytes : (int64_t)T.klen * lda2;
            set_r(ao, T.row0, T.row_end, wave, lane);
        }
        if constexpr (!B_R) {
            constexpr int rows_per = EPI == kEpiGlu ? 2 : 1;
            bbase = p.b + (int64_t)T.e * rows_per * p.N * p.ldb;
            b_lim = (int64_t)rows_per * p.N * ldb2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (i * kBigWaves + wave) * 16 + (lane >> 2);
                int n, src;
                if (EPI == kEpiGlu) {  // blocks of 16: gate, up, gate, up, ...
                    n = T.col0 + (r >> 5) * 16 + (r & 15);
                    src = ((r >> 4) & 1) * p.N + n;
                } else {
                    n = src = T.col0 + r;
                }
                bo[i] = n < p.N ? (uint32_t)src * ldb2 + kc : kNowhere;
            }
        } else if constexpr (MODE == kDgrad) {
            bbase = p.b + (int64_t)T.e * p.K * p.ldb;
            b_lim = (int64_t)p.K * ldb2;
            set_r(bo, T.col0, p.N, wave, lane);
        } else {
            bbase = p.b_gather ? p.b : p.b + (int64_t)T.k0 * p.ldb;
            b_lim = p.b_gather ? p.b_bytes : (int64_t)T.klen * ldb2;
            set_r(bo, T.col0, p.N, wave, lane);
        }
    }
    // column part of the offsets of a K-strided operand: piece i is half of k
    // row (i * 8 + wave) * 2 + lane / 32
    __device__ __forceinline__ void set_r(uint32_t (&o)[2], int c0, int lim, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t k = (i * kBigWaves + wave) * 2 + (lane >> 5);
            const int c = c0 + (int)((lane & 31) ^ rkey(k)) * 8;
            o[i] = c < lim ? (uint32_t)c * 2u : kNowhere;
        }
    }
    __device__ __forceinline__ void issue_k(const uint16_t* base, int64_t lim, const uint32_t (&o)[2], int k, int kend,
                                            uint32_t dst, int wave, int lane) const {
        const i32x4 r = make_rsrc(base + k, lim - (int64_t)k * 2);
        const int kc = (int)((lane & 3) ^ bkey(lane >> 2)) * 8;
        const bool ok = k + kc < kend;
#pragma unroll
        for (int i = 0; i < 2; ++i) dma16(r, ok ? o[i] : kNowhere, dst + (i * kBigWaves + wave) * 1024);
    }
    __device__ __forceinline__ void issue_r(const uint16_t* base, int64_t lim, const uint32_t (&o)[2], int k, int ld,
                                            const int32_t* gather, uint32_t div, uint32_t dst, int wave,
                                            int lane) const {
        const uint32_t ld2 = (uint32_t)ld * 2u;
        const i32x4 r = gather ? make_rsrc(base, lim) : make_rsrc(base + (int64_t)k * ld, lim - (int64_t)k * ld2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int kl = (i * kBigWaves + wave) * 2;  // of lanes 0-31; lanes 32-63 the next row
            uint32_t row = kl + (lane >> 5);
            const bool ok = k + (int)row < klen && o[i] != kNowhere;
            if (gather && klen > 0) {
                const int last = klen - 1;
                const uint32_t s0 = (uint32_t)sload(gather, k0 + min(k + kl, last)) / div;
                const uint32_t s1 = (uint32_t)sload(gather, k0 + min(k + kl + 1, last)) / div;
                row = lane < 32 ? s0 : s1;
            }
            dma16(r, ok ? row * ld2 + o[i] : kNowhere, dst + (i * kBigWaves + wave) * 1024);
        }
    }
    // stage at K offset k (a kBigK multiple below klen) into LDS at dst
    __device__ __forceinline__ void issue(const Args& p, int k, uint32_t dst, int wave, int lane) const {
        if constexpr (MODE == kWgrad) issue_r(abase, a_lim, ao, k, p.lda, p.a_gather, p.a_div, dst, wave, lane);
        else issue_k(abase, a_lim, ao, k, klen, dst, wave, lane);
        if constexpr (MODE == kFwd) issue_k(bbase, b_lim, bo, k, klen, dst + kBigOp, wave, lane);
        else
            issue_r(bbase, b_lim, bo, k, p.ldb, MODE == kWgrad ? p.b_gather : nullptr, p.b_div, dst + kBigOp, wave,
                    lane);
    }
};

// Fragments of one stage for a wave: 8 blocks of 16 rows of A, 4 of B.
struct BigFrags {
    bf16x8 a[8], b[4];
};

template <int MODE, int NA>
__device__ __forceinline__ void big_read(BigFrags& f, const uint8_t* st, int wm, int wn, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (MODE != kFwd) f.b[j] = frag_r<kBigT>(st + kBigOp, wn * 64 + 16 * j, 0, lane);
        else f.b[j] = big_frag_k(st + kBigOp, wn * 64 + 16 * j, lane);
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        if constexpr (MODE == kWgrad) f.a[i] = frag_r<kBigT>(st, wm * 128 + 16 * i, 0, lane);
        else f.a[i] = big_frag_k(st, wm * 128 + 16 * i, lane);
    }
}

template <int NA>
__device__ __forceinline__ void big_mfma(f32x4 (&acc)[NA][4], const BigFrags& f) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
}

template <int MODE, int EPI>
__global__ __launch_bounds__(64 * kBigWaves, 2) void k_gemm16_big(Args p, int total_cap) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kBigStages][kBigStage];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 2, wn = wave & 3;
    const uint32_t lds0 = lds_off(&lds[0][0]);
    const int G = gridDim.x;
    const int v = (G % 8 == 0) ? (int)((blockIdx.x % 8) * (G / 8) + blockIdx.x / 8) : (int)blockIdx.x;
    const int total = MODE != kWgrad && p.tiles ? min(sload(p.tile_count, 0) * p.n_tiles, total_cap) : total_cap;
    if (v >= total) return;

    // loader: tile lt, next stage at lk, next LDS slot ls
    BigLoad<MODE, EPI> L;
    int lt = v, lk = 0, ls = 0;
    {
        const BigTile T = big_tile<MODE, EPI>(p, lt);
        L.set(p, T, wave, lane);
    }
    auto issue_next = [&]() {
        // next tile with a stage left; past the last tile the same number of
        // loads goes out with every lane past its descriptor
        while (lk >= L.klen && lt < total) {
            lt += G;
            lk = 0;
            if (lt < total) {
                const BigTile T = big_tile<MODE, EPI>(p, lt);
                L.set(p, T, wave, lane);
            } else {
                L.klen = 0;
            }
        }
        L.issue(p, lk, lds0 + ls * kBigStage, wave, lane);
        lk += kBigK;
        ls = (ls + 1) & (kBigStages - 1);
    };

#pragma unroll
    for (int s = 0; s < kBigStages - 1; ++s) issue_next();
    wait_vm<0>();
    int fresh = kBigStages - 1;  // stages ahead of the compute cursor known to have landed
    int cs = 0;                  // LDS slot of the compute cursor
    // One tile of a wave with NA active blocks of 16 rows (0, 4 or 8): separate
    // loops rather than a branch inside one, so that the accumulators never
    // cross a join of paths that write different parts of them.
    auto tile = [&](const BigTile& T, auto na_tag) {
        constexpr int NA = decltype(na_tag)::value;
        const int nk = (T.klen + kBigK - 1) / kBigK;
        f32x4 acc[NA ? NA : 1][4];
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < nk; ++s) {
            if (fresh > 0) --fresh;
            else wait_vm<4 * (kBigStages - 2)>();
            stage_barrier();
            issue_next();
            if constexpr (NA > 0) {
                BigFrags f;
                big_read<MODE, NA>(f, lds[cs], wm, wn, lane);
                big_mfma<NA>(acc, f);
            }
            cs = (cs + 1) & (kBigStages - 1);
        }
        wait_vm<0>();
        fresh = kBigStages - 1;
        if constexpr (NA > 0) {
            Pos o;
            o.out_base = MODE == kWgrad ? (int64_t)T.e * p.M * p.N : 0;
            o.row0 = T.row0 + wm * 128;
            o.row_end = T.row_end;
            o.col0 = T.col0 + wn * (EPI == kEpiGlu ? 32 : 64);
            epilogue<EPI>(p, acc, o, lane);
        }
    };
    for (int t = v; t < total; t += G) {
        const BigTile T = big_tile<MODE, EPI>(p, t);
        const int rows = T.row_end - (T.row0 + wm * 128);
        if (rows > 64) tile(T, std::integral_constant<int, 8>{});
        else if (rows > 0) tile(T, std::integral_constant<int, 4>{});
        else tile(T, std::integral_constant<int, 0>{});
    }
}

}  // namespace g16
}  // namespace nvq
