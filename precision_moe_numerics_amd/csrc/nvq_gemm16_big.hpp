// nvq_gemm16_big.hpp -- the persistent 256 x 256 form of the BF16 products.
#pragma once

#include "nvq_gemm16.hpp"

#include <type_traits>

namespace nvq {
namespace g16 {

constexpr int kBigT = 256;                 // output tile: 256 x 256
constexpr int kBigK = 64;                  // K of a stage: whole 128-byte lines of K-contiguous rows
constexpr int kBigWaves = 8;               // 2 (m) x 4 (n)
constexpr int kHalf = 128 * kBigK * 2;     // half an operand's stage (128 rows or columns): 16 KiB
constexpr int kBigStage = 4 * kHalf;       // A0, A1, B0, B1
constexpr int kGroupM = 4;                 // m-tiles that run side by side

// A tile of the stream (wave-uniform).
struct BigTile {
    int e, row0, row_end, col0, k0, klen;
};

// Tile t. Tiles go in groups of kGroupM m-tiles, n outside m within a group:
// the 32 workgroups of an XCD then hold 4 m-tiles x 8 n-tiles at a time, 12
// operand panels instead of 33 for the same 32 tiles along a row.
template <int MODE, int EPI>
__device__ __forceinline__ BigTile big_tile(const Args& p, int t, int m_count) {
    constexpr int TNO = EPI == kEpiGlu ? kBigT / 2 : kBigT;
    BigTile T;
    T.e = 0;
    if (MODE == kWgrad) {
        const int per = p.m_tiles * p.n_tiles;
        T.e = t / per;
        t -= T.e * per;
        m_count = p.m_tiles;
    }
    const int g = t / (kGroupM * p.n_tiles);
    const int rem = t - g * (kGroupM * p.n_tiles);
    const int gm = min(kGroupM, m_count - g * kGroupM);
    const int nt = rem / gm;
    const int mt = g * kGroupM + (rem - nt * gm);
    T.col0 = nt * TNO;
    T.k0 = 0;
    T.klen = p.K;
    if (MODE == kWgrad) {
        T.row0 = mt * kBigT;
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

// The loader: the stage being fetched, as descriptor bases and byte counts at
// its K offset and this lane's offsets within them. A stage is fetched in
// halves of 128 rows (columns), each in two pieces of 16 bytes per lane. Rows
// and columns past the tile's edge are loaded as they come (another row, or
// zeros past the descriptor): they only reach outputs that are not stored. What
// is past the end of K must be zero in both operands, whatever lies there:
// K-strided operands end their descriptor at the last row, K-contiguous ones
// send the lane nowhere. Registers are short here (128 accumulators, 96 of
// fragments): all that is kept per lane is one offset per operand (four where
// rows are gathered), the rest is formed when a piece goes out.
template <int MODE, int EPI>
struct BigLoad {
    static constexpr bool A_R = MODE == kWgrad, B_R = MODE != kFwd;
    const uint16_t *abase, *bbase;
    uint32_t alim, blim;  // K-contiguous operands: descriptor bytes
    uint32_t ao[A_R ? 1 : 4], bo;
    int klen, k0, k;      // K extent and start of the tile, K offset of the stage

    // K-contiguous: a piece is 16 bytes of row 128 half + 64 i + 8 wave + lane / 8; rows of 128 bytes
    // in LDS, chunk c of row r at slot c ^ (r & 7)
    static __device__ __forceinline__ int row_k(int wave, int lane) { return wave * 8 + (lane >> 3); }
    static __device__ __forceinline__ int chunk_k(int lane) { return (lane & 7) ^ (lane >> 3); }
    // K-strided: 16 bytes of k row 32 i + 4 wave + lane / 16; rows of 256 bytes in LDS, see rkey
    static __device__ __forceinline__ int row_r(int wave, int lane) { return wave * 4 + (lane >> 4); }
    static __device__ __forceinline__ int col_r(int wave, int lane) {
        return (int)((lane & 15) ^ rkey(row_r(wave, lane))) * 8;
    }

    __device__ __forceinline__ void set(const Args& p, const BigTile& T, int wave, int lane) {
        const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
        klen = T.klen;
        k0 = T.k0;
        k = 0;
        const bool ga = p.a_gather != nullptr;
        if constexpr (!A_R) {
            const int r = row_k(wave, lane);
            abase = ga ? p.a : p.a + (int64_t)T.row0 * p.lda;
            alim = ga ? (uint32_t)p.a_bytes : (uint32_t)min(T.row_end - T.row0, kBigT) * lda2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t src = r + 64 * i;
                if (ga) src = (uint32_t)p.a_gather[min(T.row0 + r + 64 * i, T.row_end - 1)] / p.a_div;
                ao[i] = src * lda2 + chunk_k(lane) * 16;
            }
        } else {
            abase = ga ? p.a : p.a + (int64_t)T.k0 * p.lda;
            ao[0] = (T.row0 + col_r(wave, lane)) * 2 + (ga ? 0 : row_r(wave, lane) * lda2);
        }
        if constexpr (!B_R) {
            bbase = p.b + ((int64_t)T.e * (EPI == kEpiGlu ? 2 : 1) * p.N + T.col0) * p.ldb;
            blim = (uint32_t)(EPI == kEpiGlu ? 2 * p.N - T.col0 : min(p.N - T.col0, kBigT)) * ldb2;
            const int r = row_k(wave, lane);
            // GLU: blocks of 16 rows: gate, up, gate, up, ...
            const int src = EPI == kEpiGlu ? ((r >> 4) & 1) * p.N + (r >> 5) * 16 + (r & 15) : r;
            bo = (uint32_t)src * ldb2 + chunk_k(lane) * 16;
        } else {
            const bool gb = MODE == kWgrad && p.b_gather != nullptr;
            bbase = gb ? p.b : p.b + (MODE == kDgrad ? (int64_t)T.e * p.K : (int64_t)T.k0) * p.ldb;
            bo = (T.col0 + col_r(wave, lane)) * 2 + (gb ? 0 : row_r(wave, lane) * ldb2);
        }
    }
    __device__ __forceinline__ void advance(const Args& p) {
        k += kBigK;
        if constexpr (!A_R) {
            abase += kBigK;
            alim -= kBigK * 2;
        } else if (!p.a_gather) {
            abase += (int64_t)kBigK * p.lda;
        }
        if constexpr (!B_R) {
            bbase += kBigK;
            blim -= kBigK * 2;
        } else if (MODE == kDgrad || !p.b_gather) {
            bbase += (int64_t)kBigK * p.ldb;
        }
    }
    static __device__ __forceinline__ i32x4 rsrc(const uint16_t* base, uint32_t bytes) {
        const uint64_t u = reinterpret_cast<uint64_t>(base);
        i32x4 r;
        r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
        r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(u >> 32) & 0xFFFFu));
        r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
        r[3] = 0x00020000;
        return r;
    }
    // K-contiguous piece at lane offset o (klen <= 0: nothing left to fetch)
    __device__ __forceinline__ void piece_k(const uint16_t* base, uint32_t lim, uint32_t o, uint32_t dst,
                                            int lane) const {
        dma16(rsrc(base, klen > 0 ? lim : 0), k + chunk_k(lane) * 8 < klen ? o : kNowhere, dst);
    }
    // K-strided piece i of half h
    __device__ __forceinline__ void piece_r(const uint16_t* base, int64_t bytes, uint32_t o, const int32_t* gather,
                                            uint32_t div, int ld, int h, int i, uint32_t dst, int wave,
                                            int lane) const {
        const uint32_t ld2 = (uint32_t)ld * 2u;
        if (!gather) {
            dma16(rsrc(base, (uint32_t)min(max(klen - k, 0), kBigK) * ld2), o + i * 32 * ld2 + h * 256, dst);
            return;
        }
        uint32_t src = 0;
        const int kl = k + 32 * i + 4 * wave;  // of lanes 0 .. 15; then the next rows
        if (klen > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t s = (uint32_t)sload(gather, k0 + min(kl + q, klen - 1)) / div;
                src = (lane >> 4) == q ? s : src;
            }
        }
        dma16(rsrc(base, (uint32_t)bytes), kl + (lane >> 4) < klen ? src * ld2 + o + h * 256 : kNowhere, dst);
    }
    // half (A0, A1, B0, B1), piece i of the stage, into the LDS stage at dst
    __device__ __forceinline__ void piece(const Args& p, int half, int i, uint32_t dst, int wave, int lane) const {
        const int h = half & 1;
        dst += half * kHalf + (i * kBigWaves + wave) * 1024;
        if (half < 2) {
            if constexpr (A_R) piece_r(abase, p.a_bytes, ao[0], p.a_gather, p.a_div, p.lda, h, i, dst, wave, lane);
            else piece_k(abase, alim, ao[2 * h + i], dst, lane);
        } else {
            constexpr int step = EPI == kEpiGlu ? 32 : 64;  // rows of w between pieces
            if constexpr (B_R)
                piece_r(bbase, p.b_bytes, bo, MODE == kWgrad ? p.b_gather : nullptr, p.b_div, p.ldb, h, i, dst, wave,
                        lane);
            else piece_k(bbase, blim, bo + (2 * h + i) * step * ((uint32_t)p.ldb * 2u), dst, lane);
        }
    }
};

enum { kA0 = 0, kA1 = 1, kB0 = 2, kB1 = 3 };

// Fragments of a wave: four blocks of 16 rows of an A half, two of a B half,
// both halves of K.
struct FragA {
    bf16x8 v[4][2];
};
struct FragB {
    bf16x8 v[2][2];
};

template <bool R>
__device__ __forceinline__ bf16x8 big_frag(const uint8_t* half, int r0, int ks, int lane) {
    if constexpr (R) return frag_r<128>(half, r0, ks, lane);
    else return frag_k(half, r0, ks, lane);
}
template <bool R>
__device__ __forceinline__ void big_read_a(FragA& f, const uint8_t* half, int ks, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i][ks] = big_frag<R>(half, (wave >> 2) * 64 + 16 * i, ks, lane);
}
template <bool R>
__device__ __forceinline__ void big_read_b(FragB& f, const uint8_t* half, int wave, int lane) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) f.v[j][ks] = big_frag<R>(half, (wave & 3) * 32 + 16 * j, ks, lane);
}

// The eight products of an A half (blocks i0 ..) and a B half (blocks j0 ..)
// in K half ks, with READS LDS reads (already written, into registers these
// products do not use) spread between them.
template <bool MUL, int READS>
__device__ __forceinline__ void big_mul(f32x4 (*acc)[4], int i0, int j0, const FragA& a, const FragB& b, int ks) {
    if (MUL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i0 + i][j0 + j] =
                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[j][ks], a.v[i][ks], acc[i0 + i][j0 + j], 0, 0, 0);
#pragma unroll
        for (int r = 0; r < READS; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Persistent kernel over the tiles v, v + G, ...: the K stages of a workgroup's
// tiles form one stream through two LDS stages of four halves, so a tile's
// first stages arrive while the tile before it is finished and stored.
//
// A K step of stage q has four quarters of 16 products a wave: A0 B0, A0 B1,
// A1 B1, A1 B0, each in two halves of K. Fragments are read while earlier
// products run, into registers whose last use has been issued: A's K halves
// alternate, B0 and B1 swap places from step to step. As soon as a half has
// been read by every wave (barrier) the same half two stages on is fetched into
// its place: B0 in quarter 0, A0 in 1, B1 in 2, A1 in 3. It is first read six or
// seven quarters later, so at the barriers before quarters 3, 0 and 1, the ones
// whose reads need a new half, everything but the newest five halves (10 loads
// of the wave) has landed; five quarters are 2560 matrix cycles of the SIMD.
template <int MODE, int EPI>
__global__ __launch_bounds__(64 * kBigWaves, 2) void k_gemm16_big(Args p, int total_cap) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2][kBigStage];
    using Load = BigLoad<MODE, EPI>;
    constexpr int kNew = 10;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 2, wn = wave & 3;
    const uint32_t lds0 = lds_off(&lds[0][0]);
    const int G = gridDim.x;
    const int v = (G % 8 == 0) ? (int)((blockIdx.x % 8) * (G / 8) + blockIdx.x / 8) : (int)blockIdx.x;
    const int m_count = MODE == kWgrad ? p.m_tiles : p.tiles ? sload(p.tile_count, 0) : (p.rows + kBigT - 1) / kBigT;
    const int total = MODE == kWgrad ? total_cap : min(m_count * p.n_tiles, total_cap);
    if (v >= total) return;

    Load ld;
    int lt = v;  // the loader's tile
    ld.set(p, big_tile<MODE, EPI>(p, lt, m_count), wave, lane);
    // past the last tile the same number of loads goes out, none with anything to read
    auto settle = [&]() {
        while (ld.k >= ld.klen && lt < total) {
            lt += G;
            if (lt < total) ld.set(p, big_tile<MODE, EPI>(p, lt, m_count), wave, lane);
            else ld.klen = 0;
        }
    };
    settle();
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) ld.piece(p, h, i, lds0 + s * kBigStage, wave, lane);
        ld.advance(p);
        settle();
    }
    wait_vm<0>();
    stage_barrier();
    int slot = 0;  // LDS stage of the step
    FragA a;
    FragB bx, by;
    big_read_a<Load::A_R>(a, lds[0] + kA0 * kHalf, 0, wave, lane);
    big_read_b<Load::B_R>(bx, lds[0] + kB0 * kHalf, wave, lane);

    // One tile of a wave with NA active A halves (0, 1 or 2): separate loops
    // rather than a branch inside one, so that the accumulators never cross a
    // join of paths that write different parts of them. On entry a and bx hold
    // the first stage's A0 (first K half) and B0, and every load issued so far
    // has landed in this wave's view: until loads of the tile itself are needed
    // no wait is made, so that none waits for the stores of the tile before.
    auto tile = [&](const BigTile& T, auto na_tag) {
        constexpr int NA = decltype(na_tag)::value;
        constexpr int RA = Load::A_R ? 8 : 4, RB = Load::B_R ? 8 : 4;  // LDS reads of half the A, all the B fragments
        const int nk = (T.klen + kBigK - 1) / kBigK;
        f32x4 acc[NA ? 4 * NA : 1][4];
#pragma unroll
        for (int i = 0; i < 4 * NA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        auto step = [&](int s, FragB& b0, FragB& b1) {
            const uint8_t* cur = lds[slot];
            const uint8_t* nxt = lds[slot ^ 1];
            const uint32_t dst = lds0 + slot * kBigStage;
            // quarter 0
            if (s > 1) wait_vm<kNew>();
            stage_barrier();
            ld.piece(p, kB0, 0, dst, wave, lane);
            if (NA > 0) big_read_a<Load::A_R>(a, cur + kA0 * kHalf, 1, wave, lane);
            big_mul<(NA > 0), RA>(acc, 0, 0, a, b0, 0);
            ld.piece(p, kB0, 1, dst, wave, lane);
            if (NA > 0) big_read_b<Load::B_R>(b1, cur + kB1 * kHalf, wave, lane);
            big_mul<(NA > 0), RB>(acc, 0, 0, a, b0, 1);
            // quarter 1
            if (s > 1) wait_vm<kNew>();
            stage_barrier();
            ld.piece(p, kA0, 0, dst, wave, lane);
            big_mul<(NA > 0), 0>(acc, 0, 2, a, b1, 0);
            ld.piece(p, kA0, 1, dst, wave, lane);
            if (NA > 1) big_read_a<Load::A_R>(a, cur + kA1 * kHalf, 0, wave, lane);
            big_mul<(NA > 0), (NA > 1 ? RA : 0)>(acc, 0, 2, a, b1, 1);
            // quarter 2 (nothing new is needed and B1 was read before the last barrier)
            ld.piece(p, kB1, 0, dst, wave, lane);
            if (NA > 1) big_read_a<Load::A_R>(a, cur + kA1 * kHalf, 1, wave, lane);
            big_mul<(NA > 1), RA>(acc, 4, 2, a, b1, 0);
            ld.piece(p, kB1, 1, dst, wave, lane);
            big_mul<(NA > 1), 0>(acc, 4, 2, a, b1, 1);
            // quarter 3
            if (s > 0) wait_vm<kNew>();
            stage_barrier();
            ld.piece(p, kA1, 0, dst, wave, lane);
            big_read_b<Load::B_R>(b1, nxt + kB0 * kHalf, wave, lane);
            big_mul<(NA > 1), RB>(acc, 4, 0, a, b0, 0);
            ld.piece(p, kA1, 1, dst, wave, lane);
            big_read_a<Load::A_R>(a, nxt + kA0 * kHalf, 0, wave, lane);
            big_mul<(NA > 1), RA>(acc, 4, 0, a, b0, 1);
            ld.advance(p);
            settle();
            slot ^= 1;
        };
#pragma unroll 1
        for (int s = 0; s < nk; s += 2) {
            step(s, bx, by);
            if (s + 1 < nk) step(s + 1, by, bx);
            else bx = by;
        }
        if (nk > 0) wait_vm<0>();
        if constexpr (NA > 0) {
            Pos o;
            o.out_base = MODE == kWgrad ? (int64_t)T.e * p.M * p.N : 0;
            o.row0 = T.row0 + wm * 64;
            o.row_end = T.row_end;
            o.col0 = T.col0 + wn * (EPI == kEpiGlu ? 16 : 32);
            o.col_step = EPI == kEpiGlu ? 64 : 128;
            epilogue<EPI>(p, acc, o, lane);
        }
    };
    for (int t = v; t < total; t += G) {
        const BigTile T = big_tile<MODE, EPI>(p, t, m_count);
        const int rows = T.row_end - (T.row0 + wm * 64);
        if (rows > 128) tile(T, std::integral_constant<int, 2>{});
        else if (rows > 0) tile(T, std::integral_constant<int, 1>{});
        else tile(T, std::integral_constant<int, 0>{});
    }
}

}  // namespace g16
}  // namespace nvq
