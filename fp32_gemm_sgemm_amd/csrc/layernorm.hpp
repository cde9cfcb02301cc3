// The layer norm with the residual's addition (output in float32 or in 8 bits
// with a scale a row), and its gradient with the sums of the weight's and the
// bias's gradients.
//
//   S = X + R,  m = mean(S),  d = S - m,  r = 1 / sqrt(mean(d^2) + eps),
//   Y = d r w + b
//
// Like the RMS norm (rowops.hpp, whose forms by row length these kernels take)
// they are bound by memory and make one pass: a row stays in the registers of
// one wave or one workgroup.  Unlike it, the squares need the mean first, so a
// row costs two reductions (and the 8-bit form a third, as the largest |Y| is
// not a multiple of r once b is added).  The mean is summed in float64 from the
// start and kept in two float32 parts, so that a row whose mean is far from
// zero loses nothing but its own representation: d is S - m to a rounding or two.
// Longer rows are read twice (8-bit: three times); their sums are taken about the row's
// first value x0 in float64, mean(d^2) = mean((S - x0)^2) - (m - x0)^2, where
// the difference cancels by a factor of D at most, as the first value itself
// adds (m - x0)^2 / D to the mean of the squares.
//
// A code is that of Y / scale in float64 (which the vector unit computes at
// float32's rate), rounded to float32 and then to 8 bits, so that next to the
// border of two codes it goes the formula's way but for the rounding of S.  The
// forward's squares are float64 too, so they cannot overflow.
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
    double v[2][3 * kWaves];
};

// N values combined over the NT threads that share a row.
template <int NT, typename Op, typename T, int N>
__device__ __forceinline__ void row_all(T (&x)[N], RowSums<NT> *sums, int &turn)
{
    static_assert(N <= 3, "room for three values a wave");
    const Op op;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = wave_all<Op>(x[i]);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64;
        T *const v = reinterpret_cast<T *>(sums->v[turn]);
        if constexpr (kLdsPoison) {
            float *const f = reinterpret_cast<float *>(sums->v[turn]);
            if (threadIdx.x < 6 * W) lds_poison(f + threadIdx.x, 1);
            lds_poison_done();
            __syncthreads();
        }
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i * W + wave] = x[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = v[i * W];
#pragma unroll
            for (int w = 1; w < W; ++w) x[i] = op(x[i], v[i * W + w]);
        }
        turn ^= 1;
    }
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
        // Y of one group: from d, or from S in float64
        auto affine = [&](int col, float (&w)[4], float (&b)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = 1.0f;
                b[j] = 0.0f;
            }
            if (a.w) load_cols<4>(a.w + col, col, D, w);
            if (a.b) load_cols<4>(a.b + col, col, D, b);
        };
        auto value = [&](int col, const float (&d)[4], float inv, float (&y)[4]) {
            float w[4], b[4];
            affine(col, w, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __builtin_fmaf(d[j] * inv, w[j], b[j]);
        };
        auto wide = [&](int col, const float (&s)[4], double m, double inv, double (&y)[4]) {
            float w[4], b[4];
            affine(col, w, b);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = __builtin_fma(((double)s[j] - m) * inv, (double)w[j], (double)b[j]);
        };
        // a row's scale from its largest |Y|; returns the factor from Y to its
        // code's value
        auto set_scale = [&](double big) {
            const double scale = fmax(big / kE4m3Max, (double)kE4m3MinScale);
            if (t == 0) a.scale[row] = (float)scale;
            return 1.0 / scale;
        };
        auto codes = [&](int col, const double (&y)[4], double f) {
            float c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = (float)(y[j] * f);
            store_codes(a.Q + row * a.ldq + col, col, D, c);
        };

        if constexpr (V > 0) {
            float s[V][4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
                if (col < D) load_s(col, s[i]);
            }
            double sum[1] = {0.0};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                if (so && col < D) store_row<4>(so + col, col, D, s[i], 1.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[0] += (double)s[i][j];
            }
            row_all<NT, AddOp>(sum, &sums, turn);
            const double mean = sum[0] / D;
            const Mean m(mean);
            double var[1] = {0.0};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!Q8) s[i][j] = m.from(s[i][j]);
                    const double d = Q8 ? (double)s[i][j] - mean : (double)s[i][j];
                    if (col + j < D) var[0] += d * d;
                }
            }
            row_all<NT, AddOp>(var, &sums, turn);
            const double inv = 1.0 / sqrt(var[0] / D + a.eps);
            if constexpr (Q8) {
                double y[4], big[1] = {0.0};
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int col = 4 * (i * NT + t);
                    if (col >= D) continue;
                    wide(col, s[i], mean, inv, y);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (col + j < D) big[0] = fmax(big[0], fabs(y[j]));
                }
                row_all<NT, MaxOp>(big, &sums, turn);
                const double f = set_scale(big[0]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int col = 4 * (i * NT + t);
                    if (col >= D) continue;
                    wide(col, s[i], mean, inv, y);
                    codes(col, y, f);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int col = 4 * (i * NT + t);
                    if (col >= D) continue;
                    float y[4];
                    value(col, s[i], (float)inv, y);
                    store_row<4>(a.Y + row * a.ldy + col, col, D, y, 1.0f, 0.0f);
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
            const double e = sum[0] / D, mean = x0 + e;
            const double inv = 1.0 / sqrt(fmax(sum[1] / D - e * e, 0.0) + a.eps);
            // (each thread reads what it wrote itself: with S given, X and R may
            // be the memory it went to)
            auto again = [&](int col, float (&s)[4]) {
                if (so) load_cols<4>(so + col, col, D, s);
                else load_s(col, s);
            };
            if constexpr (Q8) {
                double big[1] = {0.0};
                for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                    float s[4];
                    double y[4];
                    again((int)c, s);
                    wide((int)c, s, mean, inv, y);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c + j < D) big[0] = fmax(big[0], fabs(y[j]));
                }
                row_all<NT, MaxOp>(big, &sums, turn);
                const double f = set_scale(big[0]);
                for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                    float s[4];
                    double y[4];
                    again((int)c, s);
                    wide((int)c, s, mean, inv, y);
                    codes((int)c, y, f);
                }
            } else {
                const Mean m(mean);
                for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                    float s[4], y[4];
                    again((int)c, s);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] = m.from(s[j]);
                    value((int)c, s, (float)inv, y);
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

//   g = dY w,  dX = r (g - mean(g)) - d r^3 mean(g d) + dS,
//   dw = sum over rows of dY d r,  db = sum over rows of dY
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
        // r (g - mean g) - d c
        auto write = [&](int col, const float (&g)[4], const float (&d)[4], float r, float mg, float c) {
            float o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = r * (g[j] - mg) - d[j] * c;
            if (ds) {
                float q[4];
                load_cols<4>(ds + col, col, D, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += q[j];
            }
            store_row<4>(dx + col, col, D, o, 1.0f, 0.0f);
        };
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
            double sum[1] = {0.0};
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[0] += (double)x[i][j];
            row_all<NT, AddOp>(sum, &sums, turn);
            const Mean m(sum[0] / D);
            float q[3] = {0.0f, 0.0f, 0.0f};  // d^2, g, g d
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = col + j < D ? m.from(x[i][j]) : 0.0f;
                    const float g = y[i][j] * w[i][j];
                    q[0] += x[i][j] * x[i][j];
                    q[1] += g;
                    q[2] += g * x[i][j];
                }
            }
            row_all<NT, AddOp>(q, &sums, turn);
            const float inv_d = 1.0f / (float)D;
            const float r = 1.0f / sqrtf(q[0] * inv_d + a.eps);
            const float mg = q[1] * inv_d, c = q[2] * inv_d * r * r * r;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                if (col < D) {
                    float g[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] = y[i][j] * w[i][j];
                        dw[i][j] += y[i][j] * (x[i][j] * r);
                        db[i][j] += y[i][j];
                    }
                    write(col, g, x[i], r, mg, c);
                }
            }
        } else {
            const double x0 = (double)s[0];
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
            double q[2] = {0.0, 0.0}, p[2] = {0.0, 0.0};  // e, e^2 and g, g e of e = S - x0
            for (int64_t col = 4 * t; col < D; col += 4 * NT) {
                float g[4], x[4];
                load((int)col, g, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double e = col + j < D ? (double)x[j] - x0 : 0.0;
                    q[0] += e;
                    q[1] += e * e;
                    p[0] += (double)g[j];
                    p[1] += (double)g[j] * e;
                }
            }
            row_all<NT, AddOp>(q, &sums, turn);
            row_all<NT, AddOp>(p, &sums, turn);
            const double e = q[0] / D;
            const Mean m(x0 + e);
            const double rd = 1.0 / sqrt(fmax(q[1] / D - e * e, 0.0) + a.eps);
            const float r = (float)rd, mg = (float)(p[0] / D), c = (float)((p[1] - e * p[0]) / D * rd * rd * rd);
            for (int64_t col = 4 * t; col < D; col += 4 * NT) {
                float g[4], x[4];
                load((int)col, g, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = m.from(x[j]);
                write((int)col, g, x, r, mg, c);
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
