// The choice of a kernel for an 8-bit product (gemm_e4m3.hpp): pure host logic,
// no HIP calls, so it can be exercised without a device.
#pragma once

#include <algorithm>

#include "select.hpp"

namespace sgemm {

// A tile, and its cost for the selection: the time of 1024 codes of K with n
// tiles per compute unit is lat_ns + n * rate_ns, and fill_ns is the rest of a
// tile (its first fetch and its epilogue; the launch is left out, as every
// plan pays it).  Measured on MI355X, random codes, float32 output without an
// epilogue: K = 1024 and 4096 (microseconds, launch included) at
//                 1024x1024     2048x2048     4096x4096
//   256x256        25.7  78      29.7  81      39.9 109.5
//   128x128        12.1  29      16.1  36      43.3 115.9
//   64x128          9.1  20      14.7  35      41.6 125.7
//   64x64           7.9  18      16.7  43      51.9 150.6
struct E4m3Tile {
    int bm, bn;
    bool reg;  // also for rows that do not start 16-byte aligned
    double lat_ns, rate_ns, fill_ns;
};
constexpr E4m3Tile kE4m3Tiles[] = {
    {256, 256, false, 0.0, 22000.0, 5800.0},
    {128, 128, true, 0.0, 5900.0, 3800.0},
    {64, 128, true, 600.0, 3400.0, 2800.0},
    {64, 64, true, 1500.0, 1900.0, 2500.0},
};
// Rows that are not 16-byte aligned go through registers: this much slower.
constexpr double kE4m3RegCost = 1.13;
// Rate at which the tiles' results reach memory, all compute units at once,
// and the second pass of a K split beyond its traffic.
constexpr double kE4m3StoreBytesPerNs = 6000.0;
constexpr double kE4m3ReduceNs = 5000.0;
constexpr int kE4m3TileCount = (int)(sizeof(kE4m3Tiles) / sizeof(kE4m3Tiles[0]));

// The streaming kernel for few rows of A, by the rows it holds: its cost is
// fill_ns plus, per 1024 codes of K, wg_ns + row_ns * M for each workgroup (16
// columns) of the fullest compute unit, or the weights' time from memory if that is more.
// Measured (microseconds, launch included) at N x K of 512 x 4096, 1024 x
// 16384 and 8192 x 8192: 4.9, 11.8 and 13.7 (16 rows: 6.6, 17.1, 17.8) with 2
// waves; 8.9, 24.7 and 27.2 for 32 rows and 13.2, 39.4 and 43.4 for 64 with 4.
struct E4m3Skinny {
    int rows;
    double wg_ns, row_ns, fill_ns;
};
constexpr E4m3Skinny kE4m3Skinny[] = {
    {16, 575.0, 23.0, 100.0},
    {32, 1350.0, 0.0, 1100.0},
    {64, 2200.0, 0.0, 2000.0},
};
constexpr int kE4m3SkinnyCount = (int)(sizeof(kE4m3Skinny) / sizeof(kE4m3Skinny[0]));
constexpr double kE4m3StreamBytesPerNs = 6000.0;
constexpr int kE4m3SplitAlign = 128;  // codes: whole slices, and 16-byte aligned starts

constexpr int kE4m3None = kE4m3TileCount;  // more tiles than a grid counts
struct E4m3Plan {
    int kernel;  // a tile, or the streaming kernel -1 - i, or kE4m3None
    int splits, k_chunk;
    long long workspace_bytes;
};

// What a gated block's plan counts besides, from memory that no cache holds.  With
// few rows every workgroup waits for the same slices of the weights at about the
// same time: a slice takes a tile's cold_ns at least, whoever else computes on the
// compute unit meanwhile (`resident` workgroups share one), and all of them the
// stream's time.  The streaming kernels read both weights' rows side by side, so half
// the workgroups share the chip.  Measured, microseconds, launches included:
//                         17 rows                     64                    128
//   two of 8192 x 8192    64x128, K in 4   33.4       35.6                  56.2
//                         64x128, K in 2   41.5       43.0                  49.0
//                         64x128           59.5       60.8                  60.4
//                         streamed         36.1       58.4
//   two of 8192 x 2048    64x64            14.3       15.8                  17.4
//                         64x64, K in 2    14.7       16.2                  23.3
//                         streamed         13.2       24.8
//   two of 2048 x 8192    64x64, K in 8    16.4       17.7                  24.0
//                         64x128, K in 4   20.6       20.9                  22.2
//                         streamed         17.1       28.6
struct E4m3Cold {
    int slice, resident;
    double cold_ns;
};
constexpr E4m3Cold kE4m3Cold[kE4m3TileCount] = {{64, 1, 0.0}, {128, 2, 950.0}, {128, 3, 900.0}, {128, 5, 880.0}};
constexpr int kE4m3ColdRows = 512;
constexpr double kE4m3ColdBytesPerNs = 6000.0;
// The streaming kernels of a gated block past 16 rows (kE4m3Skinny's from the second on):
// fill_ns, per 1024 codes of K the time of a workgroup, and the stream's rate, both by the rows.
constexpr double kE4m3GatedFillNs[kE4m3SkinnyCount - 1] = {5500.0, 8500.0};
constexpr double kE4m3GatedWgNs = 700.0, kE4m3GatedRowNs = 22.0;
constexpr double kE4m3GatedBytesPerNs = 5000.0, kE4m3GatedBytesPerNsRow = 33.0;

// gated: N counts the columns of both weights, and M is past 16 rows.
inline E4m3Plan e4m3_plan(int M, int N, int K, int cus, bool aligned, long long ws, bool gated = false)
{
    E4m3Plan best = {kE4m3None, 1, K > 0 ? K : 1, 0};
    double best_t = -1.0;
    for (int i = 0; i < kE4m3SkinnyCount; ++i) {
        const E4m3Skinny &s = kE4m3Skinny[i];
        if (M > s.rows) continue;
        const double per_cu = (double)ceil_div_ll(ceil_div_ll(N, 16), cus);
        const double work = (double)K / 1024.0 * per_cu * (s.wg_ns + s.row_ns * M),
                     stream = (double)N * K / kE4m3StreamBytesPerNs;
        best = {-1 - i, 1, K > 0 ? K : 1, 0};
        best_t = s.fill_ns + (work > stream ? work : stream);
        if (gated)
            best_t = kE4m3GatedFillNs[i - 1] +
                     std::max((double)K / 1024.0 * (kE4m3GatedWgNs + kE4m3GatedRowNs * M),
                              (double)N * K / (kE4m3GatedBytesPerNs - kE4m3GatedBytesPerNsRow * M));
        break;
    }
    for (int i = 0; i < kE4m3TileCount; ++i) {
        const E4m3Tile &v = kE4m3Tiles[i];
        if (!aligned && !v.reg) continue;
        const long long tiles = ceil_div_ll(M, v.bm) * ceil_div_ll(N, v.bn);
        int last = 0;
        for (int want : kSplitCandidates) {
            const long long per = ceil_div_ll(ceil_div_ll(K, want), kE4m3SplitAlign) * kE4m3SplitAlign;
            const int splits = (int)ceil_div_ll(K, per);
            if (splits <= last) continue;
            last = splits;
            const long long bytes = splits > 1 ? (long long)splits * M * partial_ld(N) * 4 : 0;
            if (bytes > ws || tiles * splits > INT_MAX) break;
            const double per_cu = (double)ceil_div_ll(tiles * splits, cus);
            const double k = (double)(splits > 1 ? per : K) / 1024.0 * (aligned ? 1.0 : kE4m3RegCost);
            double t = v.fill_ns + k * (v.lat_ns + per_cu * v.rate_ns) +
                       4.0 * splits * (double)M * (double)N / kE4m3StoreBytesPerNs;
            if (gated && M <= kE4m3ColdRows) {
                const E4m3Cold &c = kE4m3Cold[i];
                const double slices = k * 1024.0 / c.slice;
                const double rounds = (double)ceil_div_ll((long long)per_cu, c.resident);
                const double work = v.fill_ns + std::max(slices * rounds * c.cold_ns, (double)N * K / kE4m3ColdBytesPerNs) +
                                    4.0 * splits * (double)M * (double)N / kE4m3StoreBytesPerNs;
                t = t > work ? t : work;
            }
            if (splits > 1)
                t += kE4m3ReduceNs + 4.0 * (splits + 1) * (double)M * (double)N / kReduceBytesPerNs;
            if (best_t < 0.0 || t < best_t) {
                best = {i, splits, splits > 1 ? (int)per : K, bytes};
                best_t = t;
            }
        }
    }
    return best;
}

// A gated block of N columns a weight takes the kernel of a product of twice the
// columns: as much work, as many workgroups and, with a K split, as many partial
// sums.  But up to 16 rows always stream: the gated form reads its rows of A once
// for both weights, which the plain one's rates do not know (8192 x 8192,
// microseconds: 1 row 25.7, against 37.2 with K split over tiles; 11 rows 27.0
// against 29.5).
inline E4m3Plan e4m3_gated_plan(int M, int N, int K, int cus, bool aligned, long long ws)
{
    if (M <= kE4m3Skinny[0].rows) return {-1, 1, K, 0};
    const int wide = N <= kMaxDim / 2 ? 2 * N : kMaxDim;
    E4m3Plan p = e4m3_plan(M, wide, K, cus, aligned, ws, true);
    // (the halves' rows are padded one by one)
    if (p.splits > 1) p.workspace_bytes = 8ll * p.splits * M * partial_ld(N);
    return p.workspace_bytes <= ws ? p : e4m3_plan(M, wide, K, cus, aligned, 0, true);
}

}  // namespace sgemm
