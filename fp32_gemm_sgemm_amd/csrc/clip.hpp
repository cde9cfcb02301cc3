// The Euclidean norm of all elements of many tensors, and the tensors scaled
// down to a largest norm:
//
//   n = sqrt(sum over tensors and elements of x^2),
//   c = min(1, max_norm / (n + eps)),  y = c x
//
// Squares and their sums are float64, where a float32's square is exact and
// cannot overflow, at no cost: the kernels are bound by memory (two conversions
// and sums an element against 4 bytes read).
//
// The tensors' elements are cut into chunks of kClipChunk; a workgroup takes a
// run of consecutive chunks, so it looks its first tensor up once and walks the
// table from there.  clip_norm_kernel leaves one partial sum a workgroup.
// clip_scale_kernel's workgroups each add those partial sums again, in the same
// order and so to the same bits, instead of waiting for a kernel that would do
// it for all: 2048 numbers from L2 cost about 2 us against 3 for a launch.  It
// takes the same run of chunks from its end, where the last level cache still
// holds what the norm's pass read last.  Where there is little to do one
// workgroup does all of it in one launch.
#pragma once

#include "common.hpp"
#include "layernorm.hpp"

namespace sgemm {

// One tensor: rows x cols elements; y null where nothing is written.
struct ClipTensor {
    const float *x;
    float *y;
    int64_t cols;
    int rows, ldx, ldy;
    int first;  // its first chunk
};

constexpr int kClipChunk = 4096;
constexpr int kClipThreads = 256;
constexpr int kClipOneThreads = 1024;
constexpr int kClipInline = 96;    // tensors whose table travels with the launch (3840 of its 4096 bytes)
constexpr int kClipMaxWgs = 2048;  // workgroups, and so partial sums

struct ClipArgs {
    const ClipTensor *table;  // where `here` is too short for it
    double *part;             // one sum a workgroup
    float *norm;
    double max_norm, eps;
    int count, chunks, per_wg, parts;
    int in_place;             // every y is its x: nothing to write where c is 1
    ClipTensor here[kClipInline];
};
static_assert(sizeof(ClipArgs) + sizeof(void *) <= 4096, "kernel arguments");

// Rows of a tensor that share a chunk (1: a row has chunks of its own), and
// the chunks of a row.
__host__ __device__ inline int clip_rows(int64_t cols)
{
    return cols < kClipChunk ? (int)(kClipChunk / (cols > 0 ? cols : 1)) : 1;
}
__host__ __device__ inline int64_t clip_row_chunks(int64_t cols) { return (cols + kClipChunk - 1) / kClipChunk; }

// Calls f(element offset in x, offset in y, columns from there on to the row's end) for
// each group of four of chunk k of tensor e, dealt to NT threads.
template <int NT, typename F> __device__ __forceinline__ void clip_chunk(const ClipTensor &e, int k, F f)
{
    const int tid = threadIdx.x;
    const int rpc = clip_rows(e.cols);
    if (rpc == 1) {
        int64_t row = 0, col = (int64_t)k * kClipChunk;
        if (e.rows > 1) {
            const int64_t per_row = clip_row_chunks(e.cols);
            row = k / per_row;
            col = (k - row * per_row) * kClipChunk;
        }
        const int n = (int)(e.cols - col < kClipChunk ? e.cols - col : kClipChunk);
        const int64_t ix = row * e.ldx + col, iy = row * e.ldy + col;
#pragma unroll
        for (int j = 0; j < kClipChunk / (4 * NT); ++j) {
            const int i = 4 * (j * NT + tid);
            if (i < n) f(ix + i, iy + i, n - i);
        }
    } else {
        const int64_t row0 = (int64_t)k * rpc;
        const int rows = (int)(e.rows - row0 < rpc ? e.rows - row0 : rpc);
        const unsigned cols = (unsigned)e.cols, groups = (cols + 3) / 4;
        const int all = rows * (int)groups;
        for (int i = tid; i < all; i += NT) {
            const unsigned r = (unsigned)i / groups, c = 4 * ((unsigned)i - r * groups);
            f((row0 + r) * e.ldx + c, (row0 + r) * e.ldy + c, (int)(cols - c));
        }
    }
}

// The tensor that chunk c belongs to: the last one whose first chunk is not past it.
__device__ __forceinline__ int clip_find(const ClipTensor *table, int count, int c)
{
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// This thread's sum of squares over chunks [c0, c1).
template <int NT>
__device__ __forceinline__ double clip_squares(const ClipArgs &a, const ClipTensor *table, int c0, int c1)
{
    double sum = 0.0;
    if (c0 >= c1) return sum;
    int i = clip_find(table, a.count, c0);
    for (int c = c0; c < c1; ++c) {
        while (i + 1 < a.count && table[i + 1].first <= c) ++i;
        const ClipTensor e = table[i];
        clip_chunk<NT>(e, c - e.first, [&](int64_t ix, int64_t, int left) {
            float v[4];
            load_cols<4>(e.x + ix, 0, left, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += (double)v[j] * (double)v[j];
        });
    }
    return sum;
}

// y = c x over chunks [c0, c1), from the last one back.
template <int NT>
__device__ __forceinline__ void clip_write(const ClipArgs &a, const ClipTensor *table, int c0, int c1, float c)
{
    if (c0 >= c1 || (a.in_place && c == 1.0f)) return;
    int i = clip_find(table, a.count, c1 - 1);
    for (int k = c1 - 1; k >= c0; --k) {
        while (table[i].first > k) --i;
        const ClipTensor e = table[i];
        clip_chunk<NT>(e, k - e.first, [&](int64_t ix, int64_t iy, int left) {
            float v[4];
            load_cols<4>(e.x + ix, 0, left, v);
            store_row<4>(e.y + iy, 0, left, v, c, 0.0f);
        });
    }
}

// c of the sum of all squares.  (A norm of NaN gives NaN.)
__device__ __forceinline__ float clip_factor(const ClipArgs &a, double total)
{
    const double q = a.max_norm / (sqrt(total) + a.eps);
    return q >= 1.0 ? 1.0f : (float)q;
}

// HERE: the table is in the launch's arguments, else in memory.
template <bool HERE> __global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(ClipArgs a)
{
    __shared__ RowSums<kClipThreads> sums;
    const ClipTensor *const table = HERE ? a.here : a.table;
    const int64_t c0 = (int64_t)blockIdx.x * a.per_wg;
    const int c1 = (int)(c0 + a.per_wg < a.chunks ? c0 + a.per_wg : a.chunks);
    double sum[1] = {clip_squares<kClipThreads>(a, table, (int)c0, c1)};
    int turn = 0;
    row_all<kClipThreads, AddOp>(sum, &sums, turn);
    if (threadIdx.x == 0) a.part[blockIdx.x] = sum[0];
}

// WRITE false: the norm alone, by one workgroup.
template <bool HERE, bool WRITE> __global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(ClipArgs a)
{
    __shared__ RowSums<kClipThreads> sums;
    double total[1] = {0.0};
    for (int p = threadIdx.x; p < a.parts; p += kClipThreads) total[0] += a.part[p];
    int turn = 0;
    row_all<kClipThreads, AddOp>(total, &sums, turn);
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm) *a.norm = (float)sqrt(total[0]);
    if constexpr (WRITE) {
        const ClipTensor *const table = HERE ? a.here : a.table;
        const int64_t c0 = (int64_t)blockIdx.x * a.per_wg;
        const int c1 = (int)(c0 + a.per_wg < a.chunks ? c0 + a.per_wg : a.chunks);
        clip_write<kClipThreads>(a, table, (int)c0, c1, clip_factor(a, total[0]));
    }
}

// All of it by one workgroup.
template <bool HERE, bool WRITE> __global__ void __launch_bounds__(kClipOneThreads) clip_one_kernel(ClipArgs a)
{
    __shared__ RowSums<kClipOneThreads> sums;
    const ClipTensor *const table = HERE ? a.here : a.table;
    double total[1] = {clip_squares<kClipOneThreads>(a, table, 0, a.chunks)};
    int turn = 0;
    row_all<kClipOneThreads, AddOp>(total, &sums, turn);
    if (threadIdx.x == 0 && a.norm) *a.norm = (float)sqrt(total[0]);
    if constexpr (WRITE) clip_write<kClipOneThreads>(a, table, 0, a.chunks, clip_factor(a, total[0]));
}

// A part of a table that is too long for a launch, to the workspace.
__global__ void __launch_bounds__(128) clip_table_kernel(ClipArgs a, ClipTensor *to)
{
    static_assert(kClipInline <= 128, "an entry a thread");
    if ((int)threadIdx.x < a.count) to[threadIdx.x] = a.here[threadIdx.x];
}

}  // namespace sgemm
