// nvq_gemm16.hip -- tile tables and launches of the BF16 matrix products.
#include "nvq_gemm16_big.hpp"
#include "nvq_gemm16_skinny.hpp"

#include <algorithm>
#include <cmath>

namespace nvq {
namespace g16 {

constexpr int kTabThreads = 1024;
constexpr int kMaxE = 4096;

// The m-tiles of E expert segments, one entry each: expert, first row, end of
// the expert's rows. One workgroup: prefix sums of the experts' tile counts in
// LDS (four experts per thread), then every thread fills entries t, t + 1024,
// ... by binary search. Offsets are clamped to [0, rows] and a decreasing one
// counts as an empty segment, so no entry points outside the rows and none is
// written past `cap`. Offsets that fall and rise again can make sums past 2^31,
// which wrap: the entries found then still lie in their segments (a search ends
// at first[lo] <= i < first[lo + 1], which no wrap lies between), and a negative
// total counts as no tiles.
__global__ __launch_bounds__(kTabThreads) void k_tile_table(const int32_t* __restrict__ seg, int E, int rows, int tm,
                                                            int cap, int32_t* __restrict__ count,
                                                            Tile* __restrict__ tiles) {
    __shared__ int buf[kTabThreads];
    __shared__ int first[kMaxE + 1];
    const int t = threadIdx.x;
    auto off = [&](int e) { return min(max(seg[e], 0), rows); };
    int n[4], local = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int e = 4 * t + j;
        n[j] = e < E ? (max(off(e + 1) - off(e), 0) + tm - 1) / tm : 0;
        local += n[j];
    }
    int total;
    int base = block_exclusive_scan(local, buf, &total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (4 * t + j < E) first[4 * t + j] = base;
        base += n[j];
    }
    total = max(min(total, cap), 0);
    if (t == 0) {
        first[E] = total;
        *count = total;
    }
    __syncthreads();
    for (int i = t; i < total; i += kTabThreads) {
        int lo = 0, hi = E;  // the last expert whose first tile is at or before i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid; else hi = mid;
        }
        Tile v;
        v.e = lo;
        v.row0 = off(lo) + (i - first[lo]) * tm;
        v.row_end = max(off(lo + 1), off(lo));
        v.pad = 0;
        tiles[i] = v;
    }
}

template <int MODE, int EPI, bool AHEAD>
void run(Args p, int64_t m_tiles_cap, hipStream_t s) {
    constexpr int TNO = EPI == kEpiGlu ? 64 : 128;
    p.n_tiles = (p.N + TNO - 1) / TNO;
    p.total = (int)(m_tiles_cap * p.n_tiles);
    const unsigned grid = ((unsigned)p.total + 7u) & ~7u;  // xcd_id: whole rounds of the 8 XCDs
    hipLaunchKernelGGL((k_gemm16<MODE, EPI, 128, 128, 2, 2, AHEAD>), dim3(grid), dim3(256), 0, s, p);
}
// Reading a stage ahead pays where a CU has one workgroup, whose reads nothing else covers (512 x 1024 x 4096 47 us
// without, 37 with; 2048^3 27.6, 25.3); with two it costs (16384 x 384 x 4096 65, 69; the weight gradient of 4091 x 2048
// x 4096 74, 78), but for the transposed reads of dgrad (8192 rows, 8 experts of 2048 x 4096 163, 153).
template <int MODE, int EPI>
void run_ahead(const Args& p, int64_t m_tiles_cap, bool one, hipStream_t s) {
    if (one) run<MODE, EPI, true>(p, m_tiles_cap, s);
    else run<MODE, EPI, false>(p, m_tiles_cap, s);
}

// Multiplier and shift of div_by.
static void set_div(uint32_t d, uint32_t* mul, int32_t* shift) {
    if (d <= 1) {
        *mul = 0;
        *shift = -1;
        return;
    }
    int s = 0;
    while ((1ull << s) < d) ++s;
    *mul = (uint32_t)((1ull << (31 + s)) / d + 1);
    *shift = s - 1;
}

template <int MODE, int EPI>
void run_big(Args p, int64_t m_tiles_cap, hipStream_t s) {
    constexpr int TNO = EPI == kEpiGlu ? kBigT / 2 : kBigT;
    p.n_tiles = (p.N + TNO - 1) / TNO;
    p.total = (int)(m_tiles_cap * p.n_tiles);
    const unsigned grid = std::min(((unsigned)p.total + 7u) & ~7u, std::max((unsigned)device_cus() & ~7u, 8u));
    set_div((uint32_t)(kGroupM * p.n_tiles), &p.group_mul, &p.group_shift);
    hipLaunchKernelGGL((k_gemm16_big<MODE, EPI>), dim3(grid), dim3(64 * kBigWaves), 0, s, p);
}

template <int EPI, int MB, int KS>
void run_skinny(Args p, hipStream_t s) {
    constexpr int TN = (EPI == kEpiGlu ? 8 : 16) * (kSkWaves / KS);
    p.n_tiles = (p.N + TN - 1) / TN;
    int64_t mt = (p.rows + 16 * MB - 1) / (16 * MB);
    if (p.seg) mt = std::min<int64_t>(p.rows, mt + p.E);
    hipLaunchKernelGGL((k_gemm16_skinny<EPI, MB, KS>), dim3((unsigned)(mt * p.n_tiles)), dim3(64 * kSkWaves), 0, s, p);
}
// K in as few parts as give the chip waves enough, some 2048: a part costs its share of the sum through LDS (fc2 of 64
// tokens, 384 experts: 522 us in 2 parts, 653 in 4, 986 in 8; 16 rows x 4096 x 4096, 256 blocks: 35, 20 and 12).
template <int EPI, int MB>
void run_skinny_k(const Args& p, hipStream_t s) {
    const int64_t mt = (p.rows + 16 * MB - 1) / (16 * MB);
    const int64_t blocks = (p.seg ? std::min<int64_t>(p.rows, mt + p.E) : mt) * ((p.N + 15) / 16);
    if (blocks >= 1024) run_skinny<EPI, MB, 2>(p, s);
    else if (blocks >= 512) run_skinny<EPI, MB, 4>(p, s);
    else run_skinny<EPI, MB, 8>(p, s);
}
// Rows of x a workgroup takes: those of a typical expert, up to 64 where that still gives the chip workgroups (64 rows
// x 4096 x 4096: 23 us with 64, 27 with 32; 128 x 1024 x 4096: 23 and 15).
template <int EPI>
void run_skinny_rows(const Args& p, int64_t active, hipStream_t s) {
    const int64_t per = (p.rows + active - 1) / active, blocks = EPI == kEpiGlu ? p.N / 8 : (p.N + 15) / 16;
    if (per <= 16) run_skinny_k<EPI, 1>(p, s);
    else if (per > 32 && (p.rows + 63) / 64 * blocks >= 256) run_skinny_k<EPI, 4>(p, s);
    else run_skinny_k<EPI, 2>(p, s);
}

}  // namespace g16

using namespace g16;

constexpr int kMinTileM = 128;

static int64_t tile_cap(int64_t rows, int64_t E, int tm) { return (rows + tm - 1) / tm + E; }

size_t gemm16_ws_bytes(int64_t rows, int64_t E) {
    Carver c(nullptr);
    c.take<int32_t>(1);
    c.take<Tile>((size_t)tile_cap(std::max<int64_t>(rows, 0), std::max<int64_t>(E, 1), kMinTileM));
    return c.need;
}

bool gemm16_dims_ok(int mode, bool glu, int64_t rows, int64_t E, int64_t M, int64_t N, int64_t K) {
    const int64_t i31 = (int64_t)1 << 31;
    if (rows < 0 || rows >= i31 - 256 || E < 1 || E > kMaxE || N < 8 || N % 8 != 0 || N > (1 << 22)) return false;
    if (mode == kWgrad) {
        if (M < 8 || M % 8 != 0 || M > (1 << 22)) return false;
        return grid_ok(E * ((M + 127) / 128) * ((N + 127) / 128) + 8, 256);
    }
    if (K < 8 || K % 8 != 0 || K > (1 << 22)) return false;
    // one expert's weights are one buffer descriptor
    if ((glu ? 2 : 1) * N * K * 2 > kMaxBytes) return false;
    const int tn = glu ? 64 : 128;
    return grid_ok(tile_cap(rows, E, kMinTileM) * ((N + tn - 1) / tn) + 8, 256);
}

// Whether 256 x 256 tiles (one persistent workgroup per CU) beat 128 x 128 ones (two workgroups per CU), by the rounds
// that the chip makes over them. A K step of a big tile takes a CU 13 units, one of two small tiles at once 11; a CU that
// has one small tile only, 7. Measured, small against big, us, bf16 outputs of FWD: 2048 x 4096 x 4096 73, 88; 4096^3 152,
// 112; 3000 x 7000 x 1000 76, 62; 6000 x 6000 x 600 79, 67; fc1 of 384 experts at 4096 tokens 1326, 1413, at 8192 1909,
// 1490. Weight gradients, of E experts with R rows each, fp32 outputs, then bf16:
//   384 of 4096 x 1024, R =   64   1329, 1240   1036,  716        8 of 2048 x 4096, R = 2048   340, 289   314, 266
//                       R =  128   1971, 1282   1353,  988        8 of 4096 x 1024, R = 2048   164, 150   139, 138
//                       R =  341   2636, 2017   1959, 1579      270 of  192 x  152, R =  128    19,  38    17,  36
//                       R = 1024   4306, 3738   3748, 3387        1 of 1024 x 4096, R = 4096    52, 118    50, 117
//   384 of 2048 x 4096, R =  341   5311, 4134   3569, 3020        1 of 2048 x 4096, R = 4096    70, 120    68, 118
//    64 of 1024 x 1024, R =  256    100,   76     57,   57        1 of 4096 x 4096, R = 4096   149, 133   141, 131
//   384 of 4096 x 1024, R =  341, accumulating   3867, 3618   2785, 2821
// The rule takes the faster side of each, or one within 1.5 %; outputs twice as wide change none of them.
static bool big_tiles(double big, double small, int cus) {
    const double t_small = small <= cus ? 7.0 : 11.0 * std::max(1.0, small / (2.0 * cus));
    return 13.0 * std::max(1.0, std::ceil(big / cus)) < t_small;
}

void launch_gemm16(int mode, int epi, Args p, void* ws, hipStream_t s) {
    set_div(p.a_div, &p.a_mul, &p.a_shift);
    set_div(p.b_div, &p.b_mul, &p.b_shift);
    const int64_t n_big = (p.N + (epi == kEpiGlu ? 127 : 255)) / (epi == kEpiGlu ? 128 : 256);
    const int64_t n_small = (p.N + (epi == kEpiGlu ? 63 : 127)) / (epi == kEpiGlu ? 64 : 128);
    const int cus = device_cus();
    if (mode == kWgrad) {
        const int64_t mb = (p.M + 255) / 256 * (int64_t)p.E, ms = (p.M + 127) / 128 * (int64_t)p.E;
        if (big_tiles((double)mb * n_big, (double)ms * n_small, cus)) {
            p.m_tiles = (p.M + 255) / 256;
            run_big<kWgrad, kEpiOut>(p, mb, s);
        } else {
            p.m_tiles = (p.M + 127) / 128;
            run_ahead<kWgrad, kEpiOut>(p, ms, ms * n_small <= cus, s);
        }
        return;
    }
    if (p.rows == 0) return;
    // Few tiles leave the 128 x 128 kernel with the latency of its K steps, 0.55 us each however few its workgroups; the
    // skinny kernel's time is that of its traffic: x once per 16 rows of weights, at about 8 TB/s from the caches, and the
    // weights once per block of rows, at about 5. (One token, 384 experts, fc1: 30 us against 47; two tokens: 60 against
    // 50; 32 rows x 4096 x 4096: 15 against 37; 512 x 1024 x 4096: 43 against 37.)
    const int64_t active = p.seg ? std::min<int64_t>(p.E, p.rows) : 1;
    if (mode == kFwd) {
        const int64_t blocks = epi == kEpiGlu ? p.N / 8 : (p.N + 15) / 16;
        const double skinny = ((double)p.rows * blocks / 8 + (double)(active + p.rows / 64) * blocks * 16 / 5) * p.K * 2e-6;
        const double tiles = (double)(active + p.rows / 128) * n_small;
        // (its workgroups are at most five per tile: the bound keeps a launch below 2^32 work-items)
        if (tiles < (1 << 18) && skinny < 0.55 * ((p.K + 63) / 64) * std::max(1.0, tiles / 512)) {
            if (epi == kEpiGlu) run_skinny_rows<kEpiGlu>(p, active, s);
            else if (epi == kEpiAct) run_skinny_rows<kEpiAct>(p, active, s);
            else run_skinny_rows<kEpiOut>(p, active, s);
            return;
        }
    }
    // m-tiles: exact for one segment, half a tile more than its rows fill for a typical expert
    auto m_tiles = [&](int tm) {
        if (!p.seg) return (double)((p.rows + tm - 1) / tm);
        return std::max((double)active, (double)p.rows / tm + 0.5 * active);
    };
    const bool big = big_tiles(m_tiles(256) * n_big, m_tiles(128) * n_small, cus);
    const int tm = big ? 256 : 128;
    int64_t mt;
    if (p.seg) {
        Carver cv(ws);
        int32_t* count = cv.take<int32_t>(1);
        mt = tile_cap(p.rows, p.E, tm);
        Tile* tiles = cv.take<Tile>((size_t)mt);
        hipLaunchKernelGGL(k_tile_table, dim3(1), dim3(kTabThreads), 0, s, p.seg, p.E, p.rows, tm, (int)mt, count,
                           tiles);
        p.tiles = tiles;
        p.tile_count = count;
    } else {
        mt = (p.rows + tm - 1) / tm;
    }
    if (big) {
        if (mode == kDgrad) run_big<kDgrad, kEpiOut>(p, mt, s);
        else if (epi == kEpiGlu) run_big<kFwd, kEpiGlu>(p, mt, s);
        else if (epi == kEpiAct) run_big<kFwd, kEpiAct>(p, mt, s);
        else run_big<kFwd, kEpiOut>(p, mt, s);
        return;
    }
    const bool one = m_tiles(128) * n_small <= cus;  // tile per CU
    if (mode == kDgrad) run<kDgrad, kEpiOut, true>(p, mt, s);
    else if (epi == kEpiGlu) run_ahead<kFwd, kEpiGlu>(p, mt, one, s);
    else if (epi == kEpiAct) run_ahead<kFwd, kEpiAct>(p, mt, one, s);
    else run_ahead<kFwd, kEpiOut>(p, mt, one, s);
}

}  // namespace nvq
