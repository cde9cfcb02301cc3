// The Euclidean norm of all elements of many tensors, and the tensors scaled
// down to a largest norm:
//
//   n = sqrt(sum over tensors and elements of x^2),
//   c = min(1, max_norm / (n + eps)),  y = c x
//
// A c below float32's normal range (large values under a small limit) is kept as
// 2^-126 times a normal number and applied in two steps: the first is exact but for
// results below all of float32, so y has the roundings of c and of the
// product like any other.
//
// Squares and their sums are float64, where a float32's square is exact and
// cannot overflow, at no cost: the kernels are bound by memory (two conversions
// and sums an element against 4 bytes read).
//
// The tensors' elements are cut into chunks of kClipChunk, dealt to the
// workgroups in turns.  clip_norm_kernel leaves one partial sum a workgroup.
// clip_scale_kernel's workgroups each add those partial sums again, in the same
// order and so to the same bits, instead of waiting for a kernel that would do
// it for all: 2048 numbers from L2 cost about 2 us against 3 for a launch.  It
// takes the turns from the last one back, whose values the last level cache
// still holds from the norm's pass, and passes that cache by with its own loads
// and stores, which are the last use of a value in this call.  Measured on 2^29
// values (2 GiB) as bare loops, microseconds for both kernels: 1056 so, 1171 with
// plain loads and stores, 1128 where a workgroup takes consecutive chunks; on 2^24
// values 29.0, 32.2 and 32.6.  These kernels, which look their chunks up, take 1111
// for 2^29.  Where there is little to do one workgroup does all of it in one launch.
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
    int count, chunks, parts;
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

// Chunk k of tensor e, dealt to NT threads in groups of four: whole(offset in x,
// offset in y) once where the chunk is kClipChunk elements of one row (a thread's
// groups are then 4 NT apart), else part(offsets, columns from there on to the row's end)
// for each group.
template <int NT, typename W, typename P>
__device__ __forceinline__ void clip_chunk(const ClipTensor &e, int k, W whole, P part)
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
        const int64_t ix = row * e.ldx + col, iy = row * e.ldy + col, left = e.cols - col;
        if (left >= kClipChunk) {
            whole(ix + 4 * tid, iy + 4 * tid);
            return;
        }
        for (int i = 4 * tid; i < (int)left; i += 4 * NT) part(ix + i, iy + i, (int)left - i);
    } else {
        const int64_t row0 = (int64_t)k * rpc;
        const int rows = (int)(e.rows - row0 < rpc ? e.rows - row0 : rpc);
        const unsigned cols = (unsigned)e.cols, groups = (cols + 3) / 4;
        const int all = rows * (int)groups;
        for (int i = tid; i < all; i += NT) {
            const unsigned r = (unsigned)i / groups, c = 4 * ((unsigned)i - r * groups);
            part((row0 + r) * e.ldx + c, (row0 + r) * e.ldy + c, (int)(cols - c));
        }
    }
}

// The tensor that chunk c belongs to, among lo .. hi: the last one whose first chunk is
// not past it.
__device__ __forceinline__ int clip_find(const ClipTensor *table, int lo, int hi, int c)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Walks the table along with a workgroup's chunks, forwards or back.
struct ClipWalk {
    const ClipTensor *const table;
    const int count, chunks;
    ClipTensor e;     // the present tensor
    int i, end;       // its place, and the first chunk past it

    __device__ __forceinline__ ClipWalk(const ClipTensor *t, int n, int all) : table(t), count(n), chunks(all), i(0), end(0) {}

    __device__ __forceinline__ void to(int at)
    {
        i = at;
        e = table[i];
        end = i + 1 < count ? table[i + 1].first : chunks;
    }
    __device__ __forceinline__ void start(int c) { to(clip_find(table, 0, count - 1, c)); }
    __device__ __forceinline__ void forwards(int c)
    {
        if (c < end) return;
        to(i + 1);
        if (c >= end) to(clip_find(table, i + 1, count - 1, c));
    }
    __device__ __forceinline__ void back(int c)
    {
        if (c >= e.first) return;
        to(i - 1);
        if (c < e.first) to(clip_find(table, 0, i - 1, c));
    }
};

// This thread's sum of squares over chunks first, first + step, ...
template <int NT>
__device__ __forceinline__ double clip_squares(const ClipArgs &a, const ClipTensor *table, int first, int step)
{
    double sum = 0.0;
    if (first >= a.chunks) return sum;
    constexpr int G = kClipChunk / (4 * NT);  // groups of a thread
    ClipWalk w(table, a.count, a.chunks);
    w.start(first);
    for (int64_t c = first; c < a.chunks; c += step) {
        w.forwards((int)c);
        clip_chunk<NT>(
            w.e, (int)c - w.e.first,
            [&](int64_t ix, int64_t) {
                f32x4 v[G];
#pragma unroll
                for (int j = 0; j < G; ++j) v[j] = *reinterpret_cast<const f32x4u *>(w.e.x + ix + j * 4 * NT);
#pragma unroll
                for (int j = 0; j < G; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum += (double)v[j][q] * (double)v[j][q];
            },
            [&](int64_t ix, int64_t, int left) {
                float v[4];
                load_cols<4>(w.e.x + ix, 0, left, v);
#pragma unroll
                for (int q = 0; q < 4; ++q) sum += (double)v[q] * (double)v[q];
            });
    }
    return sum;
}

// c = first * second.
struct ClipFactor {
    float first, second;
};

// c of the sum of all squares.  (A norm of NaN gives NaN.)
__device__ __forceinline__ ClipFactor clip_factor(const ClipArgs &a, double total)
{
    const double c = a.max_norm / (sqrt(total) + a.eps);
    if (c >= 1.0) return {1.0f, 1.0f};
    return c < 0x1p-126 ? ClipFactor{0x1p-126f, (float)(c * 0x1p126)} : ClipFactor{1.0f, (float)c};
}

// y = c x over the same chunks, from the last one back.
template <int NT>
__device__ __forceinline__ void clip_write(const ClipArgs &a, const ClipTensor *table, int first, int step,
                                           const ClipFactor &c)
{
    if (first >= a.chunks || (a.in_place && c.second == 1.0f && c.first == 1.0f)) return;
    constexpr int G = kClipChunk / (4 * NT);
    ClipWalk w(table, a.count, a.chunks);
    int64_t k = first + (int64_t)((a.chunks - 1 - first) / step) * step;
    w.start((int)k);
    for (; k >= first; k -= step) {
        w.back((int)k);
        clip_chunk<NT>(
            w.e, (int)k - w.e.first,
            [&](int64_t ix, int64_t iy) {
                f32x4u v[G];
#pragma unroll
                for (int j = 0; j < G; ++j)
                    v[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u *>(w.e.x + ix + j * 4 * NT));
#pragma unroll
                for (int j = 0; j < G; ++j)
                    __builtin_nontemporal_store(v[j] * c.first * c.second, reinterpret_cast<f32x4u *>(w.e.y + iy + j * 4 * NT));
            },
            [&](int64_t ix, int64_t iy, int left) {
                float v[4];
                load_cols<4>(w.e.x + ix, 0, left, v);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] *= c.first;
                store_row<4>(w.e.y + iy, 0, left, v, c.second, 0.0f);
            });
    }
}

// HERE: the table is in the launch's arguments, else in memory.
template <bool HERE> __global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(ClipArgs a)
{
    __shared__ RowSums<kClipThreads> sums;
    double sum[1] = {clip_squares<kClipThreads>(a, HERE ? a.here : a.table, (int)blockIdx.x, (int)gridDim.x)};
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
    if constexpr (WRITE)
        clip_write<kClipThreads>(a, HERE ? a.here : a.table, (int)blockIdx.x, (int)gridDim.x,
                                 clip_factor(a, total[0]));
}

// All of it by one workgroup.  (So few chunks are few tensors: the table is `here`.)
template <bool WRITE> __global__ void __launch_bounds__(kClipOneThreads) clip_one_kernel(ClipArgs a)
{
    __shared__ RowSums<kClipOneThreads> sums;
    double total[1] = {clip_squares<kClipOneThreads>(a, a.here, 0, 1)};
    int turn = 0;
    row_all<kClipOneThreads, AddOp>(total, &sums, turn);
    if (threadIdx.x == 0 && a.norm) *a.norm = (float)sqrt(total[0]);
    if constexpr (WRITE) clip_write<kClipOneThreads>(a, a.here, 0, 1, clip_factor(a, total[0]));
}

// A part of a table that is too long for a launch, to the workspace.
__global__ void __launch_bounds__(128) clip_table_kernel(ClipArgs a, ClipTensor *to)
{
    static_assert(kClipInline <= 128, "an entry a thread");
    if ((int)threadIdx.x < a.count) to[threadIdx.x] = a.here[threadIdx.x];
}

}  // namespace sgemm
