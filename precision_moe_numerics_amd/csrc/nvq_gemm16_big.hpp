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
constexpr int kSlots = 8;                  // halves in LDS
constexpr int kGroupM = 4;                 // m-tiles that run side by side

// A tile of the stream (wave-uniform).
struct BigTile {
    int e, row0, row_end, col0, k0, klen;
};

// Walks a workgroup's tiles v, v + G, ... and holds the next one's table entries
// as they come from scalar loads issued a tile earlier: a tile of a weight
// gradient lasts a few microseconds, and a chain of dependent loads and integer
// divisions at its head would cost as much again.
//
// Tiles go in groups of kGroupM m-tiles, n outside m within a group: the 32
// workgroups of an XCD then hold 4 m-tiles x 8 n-tiles at a time, 12 operand
// panels instead of 33 for the same 32 tiles along a row.
template <int MODE, int EPI>
struct BigWalk {
    int t;            // the tile
    int e, r;         // WGRAD: its expert and number within the expert
    int mt, nt;
    int32_t q0, q1, q2;  // table entries

    __device__ __forceinline__ void start(const Args& p, int t0, int total, int m_count) {
        t = t0;
        e = MODE == kWgrad ? t / (p.m_tiles * p.n_tiles) : 0;
        r = t - e * (p.m_tiles * p.n_tiles);
        load(p, total, m_count);
    }
    __device__ __forceinline__ void next(const Args& p, int G, int total, int m_count) {
        t += G;
        if (MODE == kWgrad) {
            r += G;
            const int per = p.m_tiles * p.n_tiles;
            while (r >= per) {
                r -= per;
                ++e;
            }
        }
        load(p, total, m_count);
    }
    __device__ __forceinline__ void load(const Args& p, int total, int m_count) {
        if (t >= total) return;
        const int u = MODE == kWgrad ? r : t;
        const int g = (int)div_by((uint32_t)u, p.group_mul, p.group_shift);  // kGroupM * n_tiles per group
        const int rem = u - g * (kGroupM * p.n_tiles);
        const int gm = min(kGroupM, (MODE == kWgrad ? p.m_tiles : m_count) - g * kGroupM);
        nt = gm == 4 ? rem >> 2 : gm == 2 ? rem >> 1 : gm == 1 ? rem : (int)__umulhi((uint32_t)rem, 0x55555556u);
        mt = g * kGroupM + (rem - nt * gm);
        if (MODE == kWgrad) {
            if (p.seg) {
                q0 = sload(p.seg, e);
                q1 = sload(p.seg, e + 1);
            }
        } else if (p.tiles) {
            q0 = sload(&p.tiles[mt].e, 0);
            q1 = sload(&p.tiles[mt].row0, 0);
            q2 = sload(&p.tiles[mt].row_end, 0);
        }
    }
    __device__ __forceinline__ BigTile get(const Args& p) const {
        BigTile T;
        T.e = e;
        T.col0 = nt * (EPI == kEpiGlu ? kBigT / 2 : kBigT);
        T.k0 = 0;
        T.klen = p.K;
        T.row0 = mt * kBigT;
        if (MODE == kWgrad) {
            T.row_end = p.M;
            T.klen = p.rows;
            if (p.seg) {
                T.k0 = min(max(q0, 0), p.rows);
                T.klen = max(min(max(q1, 0), p.rows) - T.k0, 0);
            }
        } else if (p.tiles) {
            T.e = q0;
            T.row0 = q1;
            T.row_end = q2;
        } else {
            T.row_end = p.rows;
        }
        return T;
    }
};

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
    uint32_t ra[2], rb[2]; // WGRAD with gathers: byte offsets of this lane's source rows of the stage (A, B)

    // K-contiguous: a piece is 16 bytes of row 128 half + 64 i + 8 wave + lane / 8; rows of 128 bytes
    // in LDS, chunk c of row r at slot c ^ (r & 7)
    static __device__ __forceinline__ int row_k(int wave, int lane) { return wave * 8 + (lane >> 3); }
    static __device__ __forceinline__ int chunk_k(int lane) { return (lane & 7) ^ (lane >> 3); }
    // K-strided: 16 bytes of k row 32 i + 4 wave + lane / 16; rows of 256 bytes in LDS, see rkey
    static __device__ __forceinline__ int row_r(int wave, int lane) { return wave * 4 + (lane >> 4); }
    static __device__ __forceinline__ int col_r(int wave, int lane) {
        return (int)((lane & 15) ^ rkey(row_r(wave, lane))) * 8;
    }

    // Gather entries of a tile's rows (this wave's 32: row 64 i + 8 wave + j at 8 i + j) into LDS at dst, a tile before
    // set() reads them there: a load into registers would wait for every stage in flight.
    static __device__ __forceinline__ void fetch_rows(const Args& p, const BigTile& T, uint32_t dst, int wave,
                                                      int lane) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // set()'s reads of the tile before
        const int r = T.row0 + 64 * (lane >> 3) + 8 * wave + (lane & 7);
        dma4(rsrc(reinterpret_cast<const uint16_t*>(p.a_gather + T.row0), (uint32_t)min(T.row_end - T.row0, kBigT) * 4u),
             lane < 32 && r < T.row_end ? (uint32_t)(r - T.row0) * 4u : kNowhere, dst);
    }
    __device__ __forceinline__ void set(const Args& p, const BigTile& T, const int32_t* idx, int wave, int lane) {
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
                if (ga) src = div_by((uint32_t)idx[8 * i + (lane >> 3)], p.a_mul, p.a_shift);
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
            // GLU: blocks of 16 rows: gate, up, gate, up, ..., each wave's pairs of both halves adjacent:
            // rows 32 w .. 32 w + 31 of half h are gate and up of outputs 32 w + 16 h .. + 15
            const int src = EPI == kEpiGlu ? ((r >> 4) & 1) * p.N + (r >> 5) * 32 + (r & 15) : r;
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
    // Gather entries of the wave's k rows (32 i + 4 wave + q) of the stage at K offset kk, as scalar loads, issued
    // well before rows() waits for them and picks this lane's.
    typedef int32_t Entries __attribute__((ext_vector_type(8)));
    __device__ __forceinline__ Entries entries(const int32_t* gather, int kk, int wave) const {
        Entries r = {0, 0, 0, 0, 0, 0, 0, 0};
        if (klen > 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    r[4 * i + q] = sload(gather, k0 + min(kk + 32 * i + 4 * wave + q, klen - 1));
        }
        return r;
    }
    static __device__ __forceinline__ void rows(uint32_t (&o)[2], Entries r, uint32_t mul, int shift, int ld,
                                                int lane) {
        const int q = lane >> 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t v = (uint32_t)r[4 * i];
#pragma unroll
            for (int t = 1; t < 4; ++t) v = q == t ? (uint32_t)r[4 * i + t] : v;
            o[i] = div_by(v, mul, shift) * ((uint32_t)ld * 2u);
        }
    }
    // K-strided piece i of half h
    __device__ __forceinline__ void piece_r(const uint16_t* base, uint32_t o, int ld, int h, int i, uint32_t dst) const {
        const uint32_t ld2 = (uint32_t)ld * 2u;
        dma16(rsrc(base, (uint32_t)min(max(klen - k, 0), kBigK) * ld2), o + i * 32 * ld2 + h * 256, dst);
    }
    __device__ __forceinline__ void piece_g(const uint16_t* base, int64_t bytes, uint32_t o, const uint32_t (&row)[2],
                                            int h, int i, uint32_t dst, int wave, int lane) const {
        const bool ok = k + 32 * i + 4 * wave + (lane >> 4) < klen;
        dma16(rsrc(base, (uint32_t)bytes), ok ? row[i] + o + h * 256 : kNowhere, dst);
    }
    // half (A0, A1, B0, B1), piece i of the stage, into the LDS slot at dst
    __device__ __forceinline__ void piece(const Args& p, int half, int i, uint32_t dst, int wave, int lane) const {
        const int h = half & 1;
        dst += (i * kBigWaves + wave) * 1024;
        if (half < 2) {
            if constexpr (A_R) {
                if (p.a_gather)
                    piece_g(abase, p.a_bytes, ao[0], ra, h, i, dst, wave, lane);
                else piece_r(abase, ao[0], p.lda, h, i, dst);
            } else {
                piece_k(abase, alim, ao[2 * h + i], dst, lane);
            }
        } else {
            const int rows = EPI == kEpiGlu ? 64 * i + 16 * h : 64 * i + 128 * h;  // of w, from piece 0 of half 0
            if constexpr (B_R) {
                if (MODE == kWgrad && p.b_gather)
                    piece_g(bbase, p.b_bytes, bo, rb, h, i, dst, wave, lane);
                else piece_r(bbase, bo, p.ldb, h, i, dst);
            } else piece_k(bbase, blim, bo + rows * ((uint32_t)p.ldb * 2u), dst, lane);
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
template <bool MUL, int READS, bool I8>
__device__ __forceinline__ void big_mul(Acc<I8> (*acc)[4], int i0, int j0, const FragA& a, const FragB& b, int ks) {
    if (MUL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i0 + i][j0 + j] = mfma64<I8>(b.v[j][ks], a.v[i][ks], acc[i0 + i][j0 + j]);
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
// tiles form one stream through LDS, so a tile's first stages arrive while the
// tile before it is finished and stored.
//
// A K step of stage q has four quarters of 16 products a wave: A0 B0, A0 B1,
// A1 B1, A1 B0, each in two halves of K. Fragments are read while earlier
// products run, into registers whose last use has been issued: A's K halves
// alternate, B0 and B1 swap places from step to step. The operand halves B0,
// A0, B1, A1 of stage 0, 1, .. are one sequence that goes round eight LDS slots:
// half n is read in quarters n - 2 to n - 1 (of quarters counted through), so at
// the barrier that opens quarter n its slot is free and half n + 8 is fetched
// into it. At the barriers before quarters 3, 0 and 1, whose reads need a new
// half, everything but the newest five halves (10 loads of the wave) has
// landed; a half has six quarters of some 512 matrix cycles to arrive.
// (Ten slots, the whole LDS and eight quarters, measured no faster.)
template <int MODE, int EPI, bool I8>
__global__ __launch_bounds__(64 * kBigWaves, 2) void k_gemm16_big(Args p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSlots * kHalf];
    __shared__ int32_t rows_lds[kBigWaves][64];
    __shared__ __attribute__((aligned(16))) int32_t ring[kBigWaves][4][4];
    __shared__ __attribute__((aligned(16))) uint8_t row_buf[MODE == kWgrad ? kBigWaves : 1][kRowBuf];
    __shared__ __attribute__((aligned(16))) std::conditional_t<I8, Side<128>, int> side[I8 ? kBigWaves : 1];
    using Load = BigLoad<MODE, EPI>;
    constexpr int kNew = 2 * (kSlots - 3);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 2, wn = wave & 3;
    const uint32_t lds0 = lds_off(&lds[0]);
    const int G = gridDim.x;
    const int m_count = MODE == kWgrad ? p.m_tiles : p.tiles ? sload(p.tile_count, 0) : (p.rows + kBigT - 1) / kBigT;
    const int total = MODE == kWgrad ? p.total : m_count * p.n_tiles;
    const int v = xcd_id(min(total, G));
    if (v < 0) return;

    Load ld;
    BigWalk<MODE, EPI> lw;  // the tile after the one fetched
    lw.start(p, v, total, m_count);
    // The tiles between the loader and the products. A weight gradient's loader
    // may pass any number of empty segments at once and the products follow
    // with a walk of their own; otherwise every tile has a stage, the loader is
    // at most three tiles ahead, and it leaves them in a ring.
    BigWalk<MODE, EPI> cw;
    if (MODE == kWgrad) cw = lw;
    int pushed = 0, popped = 0;
    const bool gat_r = MODE != kWgrad && p.a_gather;
    const int32_t* idx = &rows_lds[wave][0];
    const uint32_t idx0 = lds_off(idx);
    if (gat_r) {
        Load::fetch_rows(p, lw.get(p), idx0, wave, lane);
        wait_vm<0>();
    }
    // moves the loader to its next tile; past the last one the same number of
    // loads goes out, none with anything to read
    auto next_tile = [&]() {
        if (lw.t >= total) {
            ld.klen = 0;
            return;
        }
        const BigTile T = lw.get(p);
        ld.set(p, T, idx, wave, lane);
        if (MODE != kWgrad) {
            int32_t* q = ring[wave][pushed++ & 3];
            if (lane == 0) {
                q[0] = T.row0;
                q[1] = T.row_end;
                q[2] = T.col0;
                if (I8) q[3] = T.e;
            }
        }
        lw.next(p, G, total, m_count);
        if (gat_r && lw.t < total) Load::fetch_rows(p, lw.get(p), idx0, wave, lane);
    };
    bool done = false;
    auto settle = [&]() {
        bool moved = false;
        while (ld.k >= ld.klen && !done) {
            done = lw.t >= total;
            next_tile();
            moved = true;
        }
        return moved;
    };
    const bool gat_a = MODE == kWgrad && p.a_gather, gat_b = MODE == kWgrad && p.b_gather;
    auto rows_a = [&](typename Load::Entries e) { Load::rows(ld.ra, e, p.a_mul, p.a_shift, p.lda, lane); };
    auto rows_b = [&](typename Load::Entries e) { Load::rows(ld.rb, e, p.b_mul, p.b_shift, p.ldb, lane); };
    next_tile();
    auto start_stage = [&]() {
        settle();
        if (gat_r) wait_vm<0>();  // (before the loop several tiles may start with no wait between them)
        if (gat_a) rows_a(ld.entries(p.a_gather, ld.k, wave));
        if (gat_b) rows_b(ld.entries(p.b_gather, ld.k, wave));
    };
    start_stage();
    // the halves of a stage in the order they are used
    auto fetch = [&](int half, int slot, int i) { ld.piece(p, half, i, lds0 + slot * kHalf, wave, lane); };
    constexpr int kOrder[4] = {kB0, kA0, kB1, kA1};
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
        fetch(kOrder[n & 3], n, 0);
        fetch(kOrder[n & 3], n, 1);
        if ((n & 3) == 3) {
            ld.advance(p);
            start_stage();
        }
    }
    wait_vm<0>();
    stage_barrier();
    int base = 0;  // slot of the step's B0
    auto slot_of = [&](int j) {
        const int x = base + j;
        return x >= kSlots ? x - kSlots : x;
    };
    FragA a;
    FragB bx, by;
    big_read_a<Load::A_R>(a, lds + kHalf, 0, wave, lane);
    big_read_b<Load::B_R>(bx, lds, wave, lane);

    int behind = 0;  // stores of the last tile that its loads in flight are older than (see tile)

    // One tile of a wave with NA active A halves (0, 1 or 2): separate loops
    // rather than a branch inside one, so that the accumulators never cross a
    // join of paths that write different parts of them. On entry a and bx hold
    // the first stage's A0 (first K half) and B0, and every load issued so far
    // has landed in this wave's view: until loads of the tile itself are needed
    // no wait is made, so that none waits for the stores of the tile before.
    // A weight gradient's whole tile is 16 (fp32: 32) stores of each wave: the
    // tile after it counts them in (`behind`) instead, and the loads of its
    // first stages, whose latency would be a tenth of a tile, stay in flight.
    auto tile = [&](const BigTile& T, auto na_tag) {
        constexpr int NA = decltype(na_tag)::value;
        constexpr int RA = Load::A_R ? 8 : 4, RB = Load::B_R ? 8 : 4;  // LDS reads of half the A, all the B fragments
        const int nk = (T.klen + kBigK - 1) / kBigK;
        Acc<I8> acc[NA ? 4 * NA : 1][4];
#pragma unroll
        for (int i = 0; i < 4 * NA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = (Acc<I8>){0, 0, 0, 0};
        // loads older than the newest five halves, where stores of the tile before may lie between
        auto settled = [&](bool steady) {
            if (steady) wait_vm<kNew>();
            else if (MODE == kWgrad && behind == 16) wait_vm<kNew + 16>();
            else if (MODE == kWgrad && behind == 32) wait_vm<kNew + 32>();
        };
        auto step = [&](int s, FragB& b0, FragB& b1) {
            const uint8_t* A0 = lds + slot_of(1) * kHalf;
            const uint8_t* B1 = lds + slot_of(2) * kHalf;
            const uint8_t* A1 = lds + slot_of(3) * kHalf;
            const uint8_t* nB0 = lds + slot_of(4) * kHalf;
            const uint8_t* nA0 = lds + slot_of(5) * kHalf;
            // quarter 0
            settled(s > 1);
            stage_barrier();
            fetch(kB0, base, 0);
            if (NA > 0) big_read_a<Load::A_R>(a, A0, 1, wave, lane);
            big_mul<(NA > 0), RA, I8>(acc, 0, 0, a, b0, 0);
            fetch(kB0, base, 1);
            if (NA > 0) big_read_b<Load::B_R>(b1, B1, wave, lane);
            big_mul<(NA > 0), RB, I8>(acc, 0, 0, a, b0, 1);
            // quarter 1
            settled(s > 1);
            stage_barrier();
            fetch(kA0, slot_of(1), 0);
            big_mul<(NA > 0), 0, I8>(acc, 0, 2, a, b1, 0);
            fetch(kA0, slot_of(1), 1);
            if (NA > 1) big_read_a<Load::A_R>(a, A1, 0, wave, lane);
            big_mul<(NA > 0), (NA > 1 ? RA : 0), I8>(acc, 0, 2, a, b1, 1);
            // quarter 2 (nothing new is needed, and B1 was read before the last barrier)
            typename Load::Entries ea = {0, 0, 0, 0, 0, 0, 0, 0}, eb = ea;
            if (gat_a) ea = ld.entries(p.a_gather, ld.k + kBigK, wave);  // for the next stage
            fetch(kB1, slot_of(2), 0);
            if (NA > 1) big_read_a<Load::A_R>(a, A1, 1, wave, lane);
            big_mul<(NA > 1), RA, I8>(acc, 4, 2, a, b1, 0);
            fetch(kB1, slot_of(2), 1);
            big_mul<(NA > 1), 0, I8>(acc, 4, 2, a, b1, 1);
            // quarter 3
            settled(s > 0);
            stage_barrier();
            if (gat_b) eb = ld.entries(p.b_gather, ld.k + kBigK, wave);
            fetch(kA1, slot_of(3), 0);
            big_read_b<Load::B_R>(b1, nB0, wave, lane);
            big_mul<(NA > 1), RB, I8>(acc, 4, 0, a, b0, 0);
            fetch(kA1, slot_of(3), 1);
            big_read_a<Load::A_R>(a, nA0, 0, wave, lane);
            big_mul<(NA > 1), RA, I8>(acc, 4, 0, a, b0, 1);
            ld.advance(p);
            if (settle()) {
                if (gat_a) ea = ld.entries(p.a_gather, ld.k, wave);
                if (gat_b) eb = ld.entries(p.b_gather, ld.k, wave);
            }
            if (gat_a) rows_a(ea);
            if (gat_b) rows_b(eb);
            base = slot_of(4);
        };
#pragma unroll 1
        for (int s = 0; s < nk; s += 2) {
            step(s, bx, by);
            if (s + 1 < nk) step(s + 1, by, bx);
            else bx = by;
        }
        const bool full = T.row_end - T.row0 >= kBigT && p.N - T.col0 >= kBigT;
        const int stays = MODE == kWgrad && full && !p.accumulate ? p.out_f32 ? 32 : 16 : 0;
        if (!stays && (nk > 0 || behind)) wait_vm<0>();
        behind = stays;
        if constexpr (NA > 0) {
            Pos o;
            o.out_base = MODE == kWgrad ? (int64_t)T.e * p.M * p.N : 0;
            o.row0 = T.row0 + wm * 64;
            o.row_end = T.row_end;
            o.col0 = T.col0 + wn * 32;
            o.pair_step = 128;
            o.e = T.e;
            if constexpr (MODE == kWgrad) {
                if (p.out_f32) epilogue_wgrad<true>(p, acc, o, row_buf[wave], full, lane);
                else epilogue_wgrad<false>(p, acc, o, row_buf[wave], full, lane);
            } else {
                epilogue<EPI>(p, acc, o, side[I8 ? wave : 0], lane);
            }
        }
    };
    for (int t = v; t < total; t += G) {
        BigTile T;
        if (MODE == kWgrad) {
            T = cw.get(p);
            cw.next(p, G, total, m_count);
            if (p.accumulate && T.klen == 0) continue;  // old + 0 would turn -0 into +0
        } else {
            const int32_t* q = ring[wave][popped++ & 3];
            T.row0 = __builtin_amdgcn_readfirstlane(q[0]);
            T.row_end = __builtin_amdgcn_readfirstlane(q[1]);
            T.col0 = __builtin_amdgcn_readfirstlane(q[2]);
            T.klen = p.K;
            T.e = I8 ? __builtin_amdgcn_readfirstlane(q[3]) : 0;
            T.k0 = 0;
        }
        const int rows = T.row_end - (T.row0 + wm * 64);
        if (rows > 128) tile(T, std::integral_constant<int, 2>{});
        else if (rows > 0) tile(T, std::integral_constant<int, 1>{});
        else tile(T, std::integral_constant<int, 0>{});
    }
}

}  // namespace g16
}  // namespace nvq
