// nvq_gemm16.hip -- tile tables and launches of the BF16 matrix products.
#include "nvq_gemm16_big.hpp"
#include "nvq_gemm16_skinny.hpp"

#include <algorithm>

namespace nvq {
namespace g16 {

constexpr int kTabThreads = 1024;
constexpr int kMaxE = 4096;

// The m-tiles of E expert segments, one entry each: expert, first row, end of
// the expert's rows. One workgroup: prefix sums of the experts' tile counts in
// LDS (four experts per thread), then every thread fills entries t, t + 1024,
// ... by binary search. Offsets are clamped to [0, rows] and a decreasing one
// counts as an empty segment, so no entry points outside the rows and none is
// written past `cap`.
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
    total = min(total, cap);
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

template <int MODE, int EPI, int TM, int TN, int WM, int WN>
void run(Args p, int64_t m_tiles_cap, hipStream_t s) {
    constexpr int TNO = EPI == kEpiGlu ? TN / 2 : TN;
    p.n_tiles = (p.N + TNO - 1) / TNO;
    const int64_t grid = m_tiles_cap * p.n_tiles;
    hipLaunchKernelGGL((k_gemm16<MODE, EPI, TM, TN, WM, WN>), dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, p);
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
    const int64_t total = m_tiles_cap * p.n_tiles;
    const int64_t grid = std::min<int64_t>(total, device_cus());
    set_div((uint32_t)(kGroupM * p.n_tiles), &p.group_mul, &p.group_shift);
    hipLaunchKernelGGL((k_gemm16_big<MODE, EPI>), dim3((unsigned)grid), dim3(64 * kBigWaves), 0, s, p, (int)total);
}

template <int EPI, int MB>
void run_skinny(Args p, hipStream_t s) {
    p.n_tiles = EPI == kEpiGlu ? p.N / 8 : (p.N + 15) / 16;
    int64_t mt = (p.rows + 16 * MB - 1) / (16 * MB);
    if (p.seg) mt = std::min<int64_t>(p.rows, mt + p.E);
    hipLaunchKernelGGL((k_gemm16_skinny<EPI, MB>), dim3((unsigned)(mt * p.n_tiles)), dim3(64 * kSkWaves), 0, s, p);
}
template <int EPI>
void run_skinny_rows(int rows, const Args& p, hipStream_t s) {
    if (rows <= 16) run_skinny<EPI, 1>(p, s);
    else if (rows <= 32) run_skinny<EPI, 2>(p, s);
    else run_skinny<EPI, 4>(p, s);
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
        return E * ((M + 127) / 128) * ((N + 127) / 128) < i31;
    }
    if (K < 8 || K % 8 != 0 || K > (1 << 22)) return false;
    // one expert's weights are one buffer descriptor
    if ((glu ? 2 : 1) * N * K * 2 > kMaxBytes) return false;
    return tile_cap(rows, E, kMinTileM) * ((N + 63) / 64) < i31;
}

void launch_gemm16(int mode, int epi, Args p, void* ws, hipStream_t s) {
    set_div(p.a_div, &p.a_mul, &p.a_shift);
    set_div(p.b_div, &p.b_mul, &p.b_shift);
    const int64_t n_big = (p.N + (epi == kEpiGlu ? 127 : 255)) / (epi == kEpiGlu ? 128 : 256);
    const int cus = device_cus();
    if (mode == kWgrad) {
        const int64_t mb = (p.M + 255) / 256 * (int64_t)p.E;
        if (mb * n_big >= cus) {
            p.m_tiles = (p.M + 255) / 256;
            run_big<kWgrad, kEpiOut>(p, mb, s);
        } else {
            p.m_tiles = (p.M + 127) / 128;
            run<kWgrad, kEpiOut, 128, 128, 2, 2>(p, (int64_t)p.m_tiles * p.E, s);
        }
        return;
    }
    if (p.rows == 0) return;
    // rows that most of the experts stay within
    const int few = p.seg ? 4 * ((p.rows + p.E - 1) / p.E) : p.rows;
    if (mode == kFwd && few <= 64) {
        if (epi == kEpiGlu) run_skinny_rows<kEpiGlu>(few, p, s);
        else if (epi == kEpiAct) run_skinny_rows<kEpiAct>(few, p, s);
        else run_skinny_rows<kEpiOut>(few, p, s);
        return;
    }
    const bool big = p.rows / p.E >= 128 && (p.rows + 255) / 256 * n_big >= cus;
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
    if (mode == kDgrad) run<kDgrad, kEpiOut, 128, 128, 2, 2>(p, mt, s);
    else if (epi == kEpiGlu) run<kFwd, kEpiGlu, 128, 128, 2, 2>(p, mt, s);
    else if (epi == kEpiAct) run<kFwd, kEpiAct, 128, 128, 2, 2>(p, mt, s);
    else run<kFwd, kEpiOut, 128, 128, 2, 2>(p, mt, s);
}

}  // namespace nvq
