// The choice of a kernel for an 8-bit product (gemm_e4m3.hpp): pure host logic,
// no HIP calls, so it can be exercised without a device.
#pragma once

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
    double ns;  // its cost by the model
};

inline E4m3Plan e4m3_plan(int M, int N, int K, int cus, bool aligned, long long ws)
{
    E4m3Plan best = {kE4m3None, 1, K > 0 ? K : 1, 0, 0.0};
    double best_t = -1.0;
    for (int i = 0; i < kE4m3SkinnyCount; ++i) {
        const E4m3Skinny &s = kE4m3Skinny[i];
        if (M > s.rows) continue;
        const double per_cu = (double)ceil_div_ll(ceil_div_ll(N, 16), cus);
        const double work = (double)K / 1024.0 * per_cu * (s.wg_ns + s.row_ns * M),
                     stream = (double)N * K / kE4m3StreamBytesPerNs;
        best = {-1 - i, 1, K > 0 ? K : 1, 0, 0.0};
        best_t = s.fill_ns + (work > stream ? work : stream);
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
            if (splits > 1)
                t += kE4m3ReduceNs + 4.0 * (splits + 1) * (double)M * (double)N / kReduceBytesPerNs;
            if (best_t < 0.0 || t < best_t) {
                best = {i, splits, splits > 1 ? (int)per : K, bytes, 0.0};
                best_t = t;
            }
        }
    }
    best.ns = best_t;
    return best;
}

}  // namespace sgemm
