// The layer norm with the residual's addition (output in float32 or in 8 bits
// with a scale a row), and its gradient with the sums of the weight's and the
// bias's gradients.
//
//   S = X + R,  m = mean(S),  d = S - m,  r = 1 / sqrt(mean(d^2) + eps),
//   Y = d r w + b
//
// Like the RMS norm (rowops.hpp, whose forms by row length these kernels take)
// they are bound by memory and make one pass: a row stays in the registers of
// one wave or one workgroup.  Mean and variance come from one reduction: sums
// of e = S - x0 and of e^2 in float64, x0 the row's first value, with
//
//   m = x0 + mean(e),  var = mean(e^2) - mean(e)^2,
//
// where the difference cancels by a factor of D at most, as the first value
// itself adds (m - x0)^2 / D to the variance: what is lost of float64's 53 bits
// is log2(D), and no square overflows.  (The vector unit adds and multiplies
// float64 at float32's rate.)  The mean is kept in two float32 parts, so that a
// row whose mean is far from zero loses nothing but its own representation.
//
// Measured (microseconds, TB/s of what has to be read and written): 8192 x 8192 98 and
// 5.5, with the residual and S stored 200 and 5.4, its codes 180 and 4.9 (float64 work
// for two values of Y an element beside the loads), the gradient with dS 202 and 5.3;
// 65536 x 512 42, 100, 85 and 101.
//
// A code is that of Y / scale in float64, rounded to float32 and then to 8 bits,
// so that next to the border of two codes it goes the formula's way but for the
// rounding of S.  It needs a second reduction, as the largest |Y| is not a
// multiple of r once b is added.
#pragma once

#include "common.hpp"
#include "epilogue.hpp"
#include "rowops.hpp"

namespace sgemm {

// ---- sums over the threads of a row ---------------------------------------------------

// x of the lane that DPP control CTRL names.
template <int CTRL> __device__ __forceinline__ float dpp_lane(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ double dpp_lane(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// x of both rows of 16 lanes (SWAP 16) or both halves of 32 (SWAP 32), in a and b.
template <int SWAP> __device__ __forceinline__ void swap_lanes(uint32_t x, uint32_t &a, uint32_t &b)
{
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 r = SWAP == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                               : __builtin_amdgcn_permlane32_swap(x, x, false, false);
    a = r[0];
    b = r[1];
}
template <int SWAP> __device__ __forceinline__ void both_lanes(float x, float &a, float &b)
{
    uint32_t p, q;
    swap_lanes<SWAP>(__builtin_bit_cast(uint32_t, x), p, q);
    a = __builtin_bit_cast(float, p);
    b = __builtin_bit_cast(float, q);
}
template <int SWAP> __device__ __forceinline__ void both_lanes(double x, double &a, double &b)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    uint32_t p0, q0, p1, q1;
    swap_lanes<SWAP>((uint32_t)u, p0, q0);
    swap_lanes<SWAP>((uint32_t)(u >> 32), p1, q1);
    a = __builtin_bit_cast(double, ((uint64_t)p1 << 32) | p0);
    b = __builtin_bit_cast(double, ((uint64_t)q1 << 32) | q0);
}

struct AddOp {
    template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
// (NaN is left out of a maximum)
struct MaxOp {
    __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};

// x combined over a wave, the same bits in every lane: pairs of lanes, of
// quads and of halves of a row of 16 through DPP, rows and halves of the wave
// through the swaps.  No step goes through LDS, as __shfl_xor's do.
template <typename Op, typename T> __device__ __forceinline__ T wave_all(T x)
{
    const Op op;
    x = op(x, dpp_lane<0xB1>(x));   // quad_perm 1 0 3 2
    x = op(x, dpp_lane<0x4E>(x));   // quad_perm 2 3 0 1
    x = op(x, dpp_lane<0x141>(x));  // row_half_mirror
    x = op(x, dpp_lane<0x140>(x));  // row_mirror
    T a, b;
    both_lanes<16>(x, a, b);
    x = op(a, b);
    both_lanes<32>(x, a, b);
    return op(a, b);
}

// LDS of a workgroup's reductions: two halves that take turns, so that one
// barrier a reduction is enough (a half is written again two reductions later).
template <int NT> struct RowSums {
    static constexpr int kWaves = NT / 64;
    double v[2][4 * kWaves];
};

// N values combined over the NT threads that share a row.
template <int NT, typename Op, typename T, int N>
__device__ __forceinline__ void row_all(T (&x)[N], RowSums<NT> *sums, int &turn)
{
    static_assert(N <= 4, "room for four values a wave");
    const Op op;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = wave_all<Op>(x[i]);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64;
        static_assert(W == 4 || W == 8 || W == 16, "waves of a workgroup");
        T *const v = reinterpret_cast<T *>(sums->v[turn]);
        if constexpr (kLdsPoison) {
            float *const f = reinterpret_cast<float *>(sums->v[turn]);
            if (threadIdx.x < 8 * W) lds_poison(f + threadIdx.x, 1);
            lds_poison_done();
            __syncthreads();
        }
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i * W + wave] = x[i];
        }
        __syncthreads();
        // each lane takes one wave's value (held by every thread at once they would
        // cost 2 W registers a value) and adds the W of them across its neighbours
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = v[i * W + (threadIdx.x & (W - 1))];
            x[i] = op(x[i], dpp_lane<0xB1>(x[i]));
            x[i] = op(x[i], dpp_lane<0x4E>(x[i]));
            if constexpr (W >= 8) x[i] = op(x[i], dpp_lane<0x141>(x[i]));
            if constexpr (W >= 16) x[i] = op(x[i], dpp_lane<0x140>(x[i]));
        }
        turn ^= 1;
    }
}

// 1 / sqrt(x), x > 0: the hardware's estimate and two of Newton's steps.  (The
// compiler's division and root take four times the instructions, one after the
// other, while a row waits.)
__device__ __forceinline__ double inv_sqrt(double x)
{
    double y = __builtin_amdgcn_rsq(x);
#pragma unroll
    for (int i = 0; i < 2; ++i) y = y * __builtin_fma(-0.5 * x * y, y, 1.5);
    return y;
}

// A mean in two float32 parts.
struct Mean {
    float hi, lo;
    __device__ __forceinline__ explicit Mean(double m) : hi((float)m), lo((float)(m - (double)hi)) {}
    __device__ __forceinline__ float from(float s) const { return (s - hi) - lo; }
};

// ---- forward ------------------------------------------------------------------------------

struct LnArgs : RowArgs {
    const float *b;
};

// NT threads share a row, V groups of 4 values each (V == 0: any D); Q8: the
// output is codes.  Threads, rows a workgroup holds and V as row_kernel's.
template <int NT, int V, bool Q8>
__global__ void __launch_bounds__(NT > 256 ? NT : 256) layernorm_kernel(LnArgs a)
{
    constexpr int RPB = NT >= 256 ? 1 : 256 / NT;
    static_assert(RPB == 1 || NT == 64, "a row is one wave's or one workgroup's");
    __shared__ RowSums<NT> sums;
    const int t = RPB == 1 ? threadIdx.x : threadIdx.x & 63;
    const int sub = RPB == 1 ? 0 : threadIdx.x >> 6;
    const int D = a.D;
    const double inv_d = 1.0 / D;
    // Q8: w and b of this thread's columns, for all its rows (read in every row, as
    // the float32 form does, each group is waited for twice: 8192 x 8192 with
    // residual 219 us against 180)
    constexpr int VR = V > 0 && Q8 ? V : 1;
    float wr[VR][4], br[VR][4];
    if constexpr (V > 0 && Q8) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 4 * (i * NT + t);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                wr[i][j] = col + j < D ? 1.0f : 0.0f;
                br[i][j] = 0.0f;
            }
            if (a.w && col < D) load_cols<4>(a.w + col, col, D, wr[i]);
            if (a.b && col < D) load_cols<4>(a.b + col, col, D, br[i]);
        }
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const float *x = a.X + row * a.ldx;
        const float *r = a.R ? a.R + row * a.ldr : nullptr;
        float *so = a.S ? a.S + row * a.lds : nullptr;
        // S of one group (zeros past D)
        auto load_s = [&](int col, float (&s)[4]) {
            load_cols<4>(x + col, col, D, s);
            if (r) {
                float q[4];
                load_cols<4>(r + col, col, D, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] += q[j];
            }
        };
        // (bases that the compiler takes for this row's own: it would keep w's and
        // b's addresses for every group in vector registers from row to row)
        const float *wp = a.w, *bp = a.b;
        asm volatile("" : "+s"(wp), "+s"(bp));
        auto affine = [&](int col, float (&w)[4], float (&b)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = 1.0f;
                b[j] = 0.0f;
            }
            if (wp) load_cols<4>(wp + col, col, D, w);
            if (bp) load_cols<4>(bp + col, col, D, b);
        };
        // Y of one group from S, in float32 and in float64
        auto narrow = [&](int col, const float (&s)[4], const Mean &m, float inv, float (&y)[4]) {
            float w[4], b[4];
            affine(col, w, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __builtin_fmaf(m.from(s[j]) * inv, w[j], b[j]);
        };
        auto wide = [&](float s, double m, double inv, float w, float b) {
            return __builtin_fma(((double)s - m) * inv, (double)w, (double)b);
        };
        // a row's scale from its largest |Y|; returns the factor from Y to its
        // code's value
        auto set_scale = [&](double big) {
            const double scale = fmax(big * (1.0 / kE4m3Max), (double)kE4m3MinScale);
            if (t == 0) a.scale[row] = (float)scale;
            return 1.0 / scale;
        };
        // the mean and r of the sums of e and e^2
        auto moments = [&](const double (&sum)[2], double x0, double &mean, double &inv) {
            const double e = sum[0] * inv_d;
            mean = x0 + e;
            inv = inv_sqrt(fmax(sum[1] * inv_d - e * e, 0.0) + a.eps);
        };

        if constexpr (V > 0) {
            // S is stored after the reduction's barrier: it may be X or R, whose
            // first value every thread reads
            const double x0 = (double)(r ? x[0] + r[0] : x[0]);
            float s[V][4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
                if (col < D) load_s(col, s[i]);
            }
            double sum[2] = {0.0, 0.0};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double e = col + j < D ? (double)s[i][j] - x0 : 0.0;
                    sum[0] += e;
                    sum[1] += e * e;
                }
            }
            row_all<NT, AddOp>(sum, &sums, turn);
            double mean, inv;
            moments(sum, x0, mean, inv);
            if (so) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int col = 4 * (i * NT + t);
                    if (col < D) store_row<4>(so + col, col, D, s[i], 1.0f, 0.0f);
                }
            }
            if constexpr (Q8) {
                double big[1] = {0.0};
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // (w and b are 0 past the row)
                        const double y = fabs(wide(s[i][j], mean, inv, wr[i][j], br[i][j]));
                        big[0] = y > big[0] ? y : big[0];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                row_all<NT, MaxOp>(big, &sums, turn);
                const double f = set_scale(big[0]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int col = 4 * (i * NT + t);
                    float c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // (computed again: the compiler would keep float64 values of
                        // all groups if it saw that they are the same)
                        asm volatile("" : "+v"(s[i][j]));
                        c[j] = (float)(wide(s[i][j], mean, inv, wr[i][j], br[i][j]) * f);
                    }
                    if (col < D) store_codes(a.Q + row * a.ldq + col, col, D, c);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                const Mean m(mean);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int col = 4 * (i * NT + t);
                    if (col < D) {
                        float y[4];
                        narrow(col, s[i], m, (float)inv, y);
                        store_row<4>(a.Y + row * a.ldy + col, col, D, y, 1.0f, 0.0f);
                    }
                    asm volatile("" ::: "memory");
                }
            }
        } else {
            const double x0 = (double)(r ? x[0] + r[0] : x[0]);
            // every thread has read x0 before S, which may be X or R, is written
            __syncthreads();
            double sum[2] = {0.0, 0.0};
            for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                float s[4];
                load_s((int)c, s);
                if (so) store_row<4>(so + c, (int)c, D, s, 1.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double e = c + j < D ? (double)s[j] - x0 : 0.0;
                    sum[0] += e;
                    sum[1] += e * e;
                }
            }
            row_all<NT, AddOp>(sum, &sums, turn);
            double mean, inv;
            moments(sum, x0, mean, inv);
            // (each thread reads what it wrote itself: with S given, X and R may
            // be the memory it went to)
            auto again = [&](int col, float (&s)[4]) {
                if (so) load_cols<4>(so + col, col, D, s);
                else load_s(col, s);
            };
            if constexpr (Q8) {
                // f(column, its four values of Y) for this thread's groups
                auto each = [&](auto f) {
                    for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                        float s[4], w[4], b[4];
                        double y[4];
                        again((int)c, s);
                        affine((int)c, w, b);
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = wide(s[j], mean, inv, w[j], b[j]);
                        f((int)c, y);
                    }
                };
                double big[1] = {0.0};
                each([&](int c, const double (&y)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) big[0] = c + j < D && fabs(y[j]) > big[0] ? fabs(y[j]) : big[0];
                });
                row_all<NT, MaxOp>(big, &sums, turn);
                const double f = set_scale(big[0]);
                each([&](int c, const double (&y)[4]) {
                    const float v[4] = {(float)(y[0] * f), (float)(y[1] * f), (float)(y[2] * f), (float)(y[3] * f)};
                    store_codes(a.Q + row * a.ldq + c, c, D, v);
                });
            } else {
                const Mean m(mean);
                for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                    float s[4], y[4];
                    again((int)c, s);
                    narrow((int)c, s, m, (float)inv, y);
                    store_row<4>(a.Y + row * a.ldy + c, (int)c, D, y, 1.0f, 0.0f);
                }
            }
        }
    }
}

// ---- gradient -------------------------------------------------------------------------------

// What the column pass of long rows needs of a row.
struct LnRow {
    float hi, lo, inv;
};

struct LnGradArgs {
    const float *dY, *S, *w, *dS;
    float *dX;
    float *part;   // partial sums, [workgroup][2 D]: dw, then db (null: not wanted)
    LnRow *rows3;  // V == 0 with sums: every row's mean and r, for the column pass
    int64_t ldy, lds, ldds, lddx;
    int rows, D;
    float eps;
};

//   g = dY w,  h = d r,  dX = r (g - mean(g) - h mean(g h)) + dS,
//   dw = sum over rows of dY h,  db = sum over rows of dY
//
// Both means are at most as large as g and h is at most sqrt(D), so nothing leaves
// float32 whatever the row's size.  (As d r^3 mean(g d) the factor of d goes with the
// inverse square of the spread: 0 in float32 from 1e23 on, infinite below 1e-19.)
//
// A workgroup takes rows blockIdx.x, + gridDim.x, ... (times its rows at once)
// and keeps the sums of its own columns in registers, as row_grad_kernel does;
// the form for any D leaves them to a column pass.
template <int NT, int V>
__global__ void __launch_bounds__(NT > 256 ? NT : 256) layernorm_grad_kernel(LnGradArgs a)
{
    constexpr int RPB = NT >= 256 ? 1 : 256 / NT;
    constexpr int VS = V > 0 ? V : 1;
    static_assert(RPB == 1 || NT == 64, "a row is one wave's or one workgroup's");
    __shared__ RowSums<NT> sums;
    // short rows: the waves' sums meet here
    __shared__ __attribute__((aligned(16))) float meet[RPB == 1 ? 4 : (RPB - 1) * 512 * VS];
    const int t = RPB == 1 ? threadIdx.x : threadIdx.x & 63;
    const int sub = RPB == 1 ? 0 : threadIdx.x >> 6;
    const int D = a.D;
    const double inv_d = 1.0 / D;
    float dw[VS][4], db[VS][4], w[VS][4];
#pragma unroll
    for (int i = 0; i < VS; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dw[i][j] = db[i][j] = 0.0f;
            w[i][j] = 1.0f;
        }
        if (V > 0 && a.w && 4 * (i * NT + t) < D) load_cols<4>(a.w + 4 * (i * NT + t), 4 * (i * NT + t), D, w[i]);
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const float *dy = a.dY + row * a.ldy;
        const float *s = a.S + row * a.lds;
        const float *ds = a.dS ? a.dS + row * a.ldds : nullptr;
        float *dx = a.dX + row * a.lddx;
        // r (g - mean g - h mean(g h))
        auto write = [&](int col, const float (&g)[4], const float (&h)[4], float r, float mg, float mgh) {
            float o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = r * ((g[j] - mg) - h[j] * mgh);
            if (ds) {
                float q[4];
                load_cols<4>(ds + col, col, D, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += q[j];
            }
            store_row<4>(dx + col, col, D, o, 1.0f, 0.0f);
        };
        const double x0 = (double)s[0];
        if constexpr (V > 0) {
            float y[VS][4], x[VS][4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[i][j] = x[i][j] = 0.0f;
                if (col < D) {
                    load_cols<4>(s + col, col, D, x[i]);
                    load_cols<4>(dy + col, col, D, y[i]);
                }
            }
            double q[4] = {0.0, 0.0, 0.0, 0.0};  // e, e^2, g, g e
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                auto add = [&](int j) {
                    const double e = (double)x[i][j] - x0, g = (double)(y[i][j] * w[i][j]);
                    q[0] += e;
                    q[1] += e * e;
                    q[2] += g;
                    q[3] += g * e;
                };
                if (col + 3 < D) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) add(j);
                } else {
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (col + j < D) add(j);
                }
            }
            row_all<NT, AddOp>(q, &sums, turn);
            const double e = q[0] * inv_d, rd = inv_sqrt(fmax(q[1] * inv_d - e * e, 0.0) + a.eps);
            const Mean m(x0 + e);
            const float r = (float)rd, mg = (float)(q[2] * inv_d);
            const float mgh = (float)((q[3] - e * q[2]) * inv_d * rd);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                if (col < D) {
                    float g[4], h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] = y[i][j] * w[i][j];
                        h[j] = m.from(x[i][j]) * r;
                        dw[i][j] += y[i][j] * h[j];
                        db[i][j] += y[i][j];
                    }
                    write(col, g, h, r, mg, mgh);
                }
            }
        } else {
            auto load = [&](int col, float (&g)[4], float (&x)[4]) {
                load_cols<4>(dy + col, col, D, g);
                load_cols<4>(s + col, col, D, x);
                if (a.w) {
                    float u[4];
                    load_cols<4>(a.w + col, col, D, u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[j] *= u[j];
                }
            };
            double q[4] = {0.0, 0.0, 0.0, 0.0};
            for (int64_t col = 4 * t; col < D; col += 4 * NT) {
                float g[4], x[4];
                load((int)col, g, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double e = col + j < D ? (double)x[j] - x0 : 0.0;
                    q[0] += e;
                    q[1] += e * e;
                    q[2] += (double)g[j];
                    q[3] += (double)g[j] * e;
                }
            }
            row_all<NT, AddOp>(q, &sums, turn);
            const double e = q[0] * inv_d, rd = inv_sqrt(fmax(q[1] * inv_d - e * e, 0.0) + a.eps);
            const Mean m(x0 + e);
            const float r = (float)rd, mg = (float)(q[2] * inv_d);
            const float mgh = (float)((q[3] - e * q[2]) * inv_d * rd);
            for (int64_t col = 4 * t; col < D; col += 4 * NT) {
                float g[4], x[4];
                load((int)col, g, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = m.from(x[j]) * r;
                write((int)col, g, x, r, mg, mgh);
            }
            if (a.rows3 && t == 0) a.rows3[row] = LnRow{m.hi, m.lo, r};
        }
    }
    if constexpr (V > 0) {
        if (!a.part) return;
        float *out = a.part + (int64_t)blockIdx.x * (2 * (int64_t)D);
        if constexpr (RPB > 1) {
            if constexpr (kLdsPoison) {
                for (int i = threadIdx.x; i < (RPB - 1) * 512 * VS; i += 256) lds_poison(&meet[i], 1);
                lds_poison_done();
                __syncthreads();
            }
            // waves 1..3 hand their sums to wave 0, which adds them in order
            if (sub > 0) {
#pragma unroll
                for (int i = 0; i < VS; ++i) {
                    float *const p = &meet[(((sub - 1) * VS + i) * 128 + t) * 4];
                    *reinterpret_cast<f32x4 *>(p) = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
                    *reinterpret_cast<f32x4 *>(p + 256) = f32x4{db[i][0], db[i][1], db[i][2], db[i][3]};
                }
            }
            __syncthreads();
            if (sub > 0) return;
#pragma unroll
            for (int v = 0; v < RPB - 1; ++v)
#pragma unroll
                for (int i = 0; i < VS; ++i) {
                    const float *const p = &meet[((v * VS + i) * 128 + t) * 4];
                    const f32x4 q = *reinterpret_cast<const f32x4 *>(p), u = *reinterpret_cast<const f32x4 *>(p + 256);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dw[i][j] += q[j];
                        db[i][j] += u[j];
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < VS; ++i) {
            const int col = 4 * (i * NT + t);
            if (col < D) {
                store_row<4>(out + col, col, D, dw[i], 1.0f, 0.0f);
                store_row<4>(out + D + col, col, D, db[i], 1.0f, 0.0f);
            }
        }
    }
}

// ---- sums over rows of two kinds at once ------------------------------------------------------

// Long rows: a workgroup covers 256 columns of one chunk of rows
// (blockIdx.y), 4 rows at a time; part is [chunk][2 N].
struct LnColArgs {
    const float *dY, *S;
    const LnRow *rows3;
    float *part;
    int64_t ldy, lds;
    int M, N, rows_per_chunk;
};

__global__ void __launch_bounds__(256) layernorm_col_kernel(LnColArgs a)
{
    __shared__ __attribute__((aligned(16))) float red[3 * 64 * 8];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t col64 = 4 * ((int64_t)blockIdx.x * 64 + tx);
    const bool in = col64 < a.N;
    const int col = in ? (int)col64 : 0;
    const int64_t m0 = (int64_t)blockIdx.y * a.rows_per_chunk;
    const int64_t m1 = m0 + a.rows_per_chunk < a.M ? m0 + a.rows_per_chunk : a.M;
    f32x4 dw = {0.0f, 0.0f, 0.0f, 0.0f}, db = dw;
    if (in) {
#pragma unroll 2
        for (int64_t m = m0 + ty; m < m1; m += 4) {
            float y[4], x[4];
            load_cols<4>(a.dY + m * a.ldy + col, col, a.N, y);
            load_cols<4>(a.S + m * a.lds + col, col, a.N, x);
            const LnRow r = a.rows3[m];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dw[j] += y[j] * (((x[j] - r.hi) - r.lo) * r.inv);
                db[j] += y[j];
            }
        }
    }
    if constexpr (kLdsPoison) {
        for (int i = threadIdx.x; i < 3 * 64 * 8; i += 256) lds_poison(&red[i], 1);
        lds_poison_done();
        __syncthreads();
    }
    if (ty > 0) {
        f32x4 *const p = reinterpret_cast<f32x4 *>(&red[((ty - 1) * 64 + tx) * 8]);
        p[0] = dw;
        p[1] = db;
    }
    __syncthreads();
    if (ty > 0 || !in) return;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const f32x4 *const p = reinterpret_cast<const f32x4 *>(&red[(i * 64 + tx) * 8]);
        dw += p[0];
        db += p[1];
    }
    float *const out = a.part + (int64_t)blockIdx.y * (2 * (int64_t)a.N);
    const float w[4] = {dw[0], dw[1], dw[2], dw[3]}, b[4] = {db[0], db[1], db[2], db[3]};
    store_row<4>(out + col, col, a.N, w, 1.0f, 0.0f);
    store_row<4>(out + a.N + col, col, a.N, b, 1.0f, 0.0f);
}

// first[n] = part[0][n] + part[1][n] + ... for n < N, second[n - N] the same
// for N <= n < 2 N (a null output is left out): col_sum_kernel's order and
// geometry over the 2 N columns, from column `base` on.
__global__ void __launch_bounds__(kColSumThreads) pair_sum_kernel(const float *part, int parts, int N, int64_t base,
                                                                  float *first, float *second)
{
    constexpr int TX = 8, TY = kColSumThreads / TX, C = 4 * TX, S = 8;
    __shared__ __attribute__((aligned(16))) float red[TY * C];
    __shared__ float red2[S * C];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int64_t n2 = 2 * (int64_t)N;
    const int64_t col = base + (int64_t)C * blockIdx.x + 4 * tx;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < n2) {
#pragma unroll 4
        for (int p = ty; p < parts; p += TY) {
            const float *const q = part + (int64_t)p * n2 + col;
            if (col + 3 < n2) {
                sum += *reinterpret_cast<const f32x4u *>(q);
            } else {
                // (2 N is even: two columns are left)
                sum[0] += q[0];
                sum[1] += q[1];
            }
        }
    }
    if constexpr (kLdsPoison) {
        for (int i = threadIdx.x; i < TY * C; i += kColSumThreads) lds_poison(&red[i], 1);
        if (threadIdx.x < S * C) lds_poison(&red2[threadIdx.x], 1);
        lds_poison_done();
        __syncthreads();
    }
    *reinterpret_cast<f32x4 *>(&red[ty * C + 4 * tx]) = sum;
    __syncthreads();
    const int c = threadIdx.x % C, s = threadIdx.x / C;
    if (s < S) {
        float v = red[s * (TY / S) * C + c];
#pragma unroll
        for (int i = 1; i < TY / S; ++i) v += red[(s * (TY / S) + i) * C + c];
        red2[s * C + c] = v;
    }
    __syncthreads();
    const int64_t n = base + (int64_t)C * blockIdx.x + threadIdx.x;
    if (threadIdx.x >= C || n >= n2) return;
    float v = red2[threadIdx.x];
#pragma unroll
    for (int i = 1; i < S; ++i) v += red2[i * C + threadIdx.x];
    float *const out = n < N ? first : second;
    if (out) out[n < N ? n : n - N] = v;
}

}  // namespace sgemm
