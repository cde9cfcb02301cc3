// Row and column operators beside the product: the RMS norm with the
// residual's addition (output in float32 or in 8 bits with a scale a row), its
// gradient, the quantisation of rows, and the elementwise part of a layer's
// gradient with the bias gradient.
//
// All are bound by memory: a few operations per element read or written.  The
// row operators therefore make one pass: a row is held in the registers of one
// wave or one workgroup (up to kRowCached values), its statistics are reduced
// across them, and what is written comes from the registers.  Longer rows are
// read a second time (from L2, mostly).  Sums are added in a fixed order: per
// thread, then a butterfly of lane shuffles, then the waves in order through
// LDS; column sums per workgroup over a fixed set of rows, then over the
// workgroups in order by a second kernel.  They are float32, but for the forward
// norm's across threads (float64, see row_kernel).
#pragma once

#include "common.hpp"
#include "epilogue.hpp"

namespace sgemm {

constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3MinScale = 1.17549435e-38f;  // 2^-126

// Four adjacent bytes at any address.
typedef uint32_t u32u __attribute__((aligned(1)));

// Four values to four e4m3 codes, rounded to nearest even.  The values are at
// most 448 in magnitude (up to the scale's rounding, which still rounds to 448).
__device__ __forceinline__ uint32_t pack_e4m3(const float (&v)[4])
{
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
    return (uint32_t)p;
}

// s * w * (f_hi + f_lo), rounded once: with the parts that the products'
// roundings drop (so no product may be fused into a later sum).
__device__ __forceinline__ float code_value(float s, float w, float f_hi, float f_lo)
{
#pragma clang fp contract(off)
    const float p = s * w;
    const float p_lo = __builtin_fmaf(s, w, -p);
    const float v = p * f_hi;
    return v + (__builtin_fmaf(p, f_hi, -v) + __builtin_fmaf(p, f_lo, p_lo * f_hi));
}

// Codes of the values at columns below D.
__device__ __forceinline__ void store_codes(unsigned char *p, int col, int D, const float (&v)[4])
{
    const uint32_t c = pack_e4m3(v);
    if (col + 3 < D) {
        *reinterpret_cast<u32u *>(p) = c;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + j < D) p[j] = (unsigned char)(c >> (8 * j));
    }
}

template <int NT> struct RowRed {
    double a[NT / 64];
    float b[NT / 64];
};

// Sums (and one maximum) over the NT threads that share a row.  A workgroup
// that reduces once per row alternates between two halves of `red` (`turn`),
// so one barrier a row is enough: the half is written again two rows later.
template <int NT, typename TA>
__device__ __forceinline__ void row_reduce(TA &a, float &b, bool b_is_max, RowRed<NT> *red, int turn)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        a += __shfl_xor(a, off);
        const float o = __shfl_xor(b, off);
        b = b_is_max ? fmaxf(b, o) : b + o;
    }
    if constexpr (NT > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            red[turn].a[wave] = a;
            red[turn].b[wave] = b;
        }
        __syncthreads();
        a = (TA)red[turn].a[0];
        b = red[turn].b[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w) {
            a += (TA)red[turn].a[w];
            b = b_is_max ? fmaxf(b, red[turn].b[w]) : b + red[turn].b[w];
        }
    }
}

// LDS race check build: the half that the next row will write is set to NaN
// after the barrier that ends its last use.
template <int NT> __device__ __forceinline__ void row_poison(RowRed<NT> *red, int turn)
{
    if constexpr (kLdsPoison && NT > 64) {
        if (threadIdx.x < sizeof(RowRed<NT>) / 4) lds_poison(reinterpret_cast<float *>(&red[turn]) + threadIdx.x, 1);
        lds_poison_done();
        __syncthreads();
    }
}

struct RowArgs {
    const float *X, *R, *w;
    float *S, *Y;
    unsigned char *Q;
    float *scale;
    int64_t ldx, ldr, lds, ldy, ldq;
    int rows, D;
    float eps;
};

// Longest row held in registers: 1024 threads of 4 groups of 4.
constexpr int kRowCached = 16384;

// Y = (S * w) * r, S = X + R, r = 1 / sqrt(mean(S^2) + eps) (NORM; else Y = X),
// to float32 or (Q8) to e4m3 codes with the row's scale.  As rounding keeps
// order, max|Y| is max|S * w| * r, so the statistics need one reduction.  A
// thread adds its few squares in float32, the threads' sums are added in
// float64 (a few operations a row), and a code's value is the product S w r /
// scale with the unrounded scale, carried in two float32 parts: next to the
// border of two codes it goes the way the formula says, but for the roundings of
// S and of the row's largest S * w, both float32.  (Codes of 8192 x 8192 random rows
// that differ from the 64-bit formula's: quantised, none, 34 with the factor in
// float32; of a norm, on its float32 S, 11 to 20, all by the largest S * w: none
// when that product is taken in 64 bits, which costs 1 to 8%, 5.3 to 5.7 us at 1 x
// 8192 and 163 to 166 at 8192 x 8192.)
//
// NT threads share a row, V groups of 4 values each (D <= 4 NT V); V == 0 is the
// form for any D, which reads the row twice.  A workgroup has max(NT, 256)
// threads, so short rows (NT = 64) go four to a workgroup and need no LDS.
template <int NT, int V, bool NORM, bool Q8>
__global__ void __launch_bounds__(NT > 256 ? NT : 256) row_kernel(RowArgs a)
{
    constexpr int RPB = NT >= 256 ? 1 : 256 / NT;  // rows a workgroup holds at once
    static_assert(RPB == 1 || NT == 64, "a row is one wave's or one workgroup's");
    __shared__ RowRed<NT> red[RPB == 1 ? 2 : 1];
    const int t = RPB == 1 ? threadIdx.x : threadIdx.x & 63;
    const int sub = RPB == 1 ? 0 : threadIdx.x >> 6;
    const int D = a.D;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const float *x = a.X + row * a.ldx;
        const float *r = a.R ? a.R + row * a.ldr : nullptr;
        float *so = a.S ? a.S + row * a.lds : nullptr;
        row_poison<NT>(red, turn);
        float sum = 0.0f, big = 0.0f;
        float inv_rms = 1.0f;
        // S * w to its code's value: a factor in two parts, and a power of two
        // for a row so small that the factor alone would overflow
        float f_hi = 0.0f, f_lo = 0.0f, f_exp = 1.0f;

        // S of one group (masked to D), stored when wanted
        auto load_s = [&](int col, float (&s)[4]) {
            load_cols<4>(x + col, col, D, s);
            if (r) {
                float q[4];
                load_cols<4>(r + col, col, D, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] += q[j];
            }
        };
        auto stats = [&](int col, const float (&s)[4]) {
            float w[4] = {1.0f, 1.0f, 1.0f, 1.0f};
            if (Q8 && NORM && a.w) load_cols<4>(a.w + col, col, D, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (NORM) sum += s[j] * s[j];
                if (Q8) big = fmaxf(big, fabsf(NORM ? s[j] * w[j] : s[j]));
            }
        };
        auto finish_stats = [&]() {
            double total = sum;
            row_reduce<NT>(total, big, true, red, turn);
            const double r = NORM ? 1.0 / sqrt(total / D + a.eps) : 1.0;
            inv_rms = (float)r;
            if (Q8) {
                const double scale = fmax(big * r / kE4m3Max, (double)kE4m3MinScale);
                double f = r / scale;
                if (f > 1e38) {
                    f *= 0x1p-120;
                    f_exp = 0x1p120f;
                }
                f_hi = (float)f;
                f_lo = (float)(f - f_hi);
                if (t == 0) a.scale[row] = (float)scale;
            }
        };
        auto write = [&](int col, const float (&s)[4]) {
            float y[4], w[4] = {1.0f, 1.0f, 1.0f, 1.0f};
            if (NORM && a.w) load_cols<4>(a.w + col, col, D, w);
            if (Q8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = code_value(s[j], NORM ? w[j] : 1.0f, f_hi, f_lo) * f_exp;
                store_codes(a.Q + row * a.ldq + col, col, D, y);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = s[j] * w[j] * inv_rms;
                store_row<4>(a.Y + row * a.ldy + col, col, D, y, 1.0f, 0.0f);
            }
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
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                if (col < D) {
                    if (so) store_row<4>(so + col, col, D, s[i], 1.0f, 0.0f);
                    stats(col, s[i]);
                }
            }
            finish_stats();
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                if (col < D) write(col, s[i]);
            }
        } else {
            for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                float s[4];
                load_s((int)c, s);
                if (so) store_row<4>(so + c, (int)c, D, s, 1.0f, 0.0f);
                stats((int)c, s);
            }
            finish_stats();
            for (int64_t c = 4 * t; c < D; c += 4 * NT) {
                float s[4];
                // (each thread reads what it wrote itself: with S given, X and R
                // may be the memory it went to)
                if (so) load_cols<4>(so + c, (int)c, D, s);
                else load_s((int)c, s);
                write((int)c, s);
            }
        }
        turn ^= RPB == 1 ? 1 : 0;
    }
}

struct RowGradArgs {
    const float *dY, *S, *w, *dS;
    float *dX;
    float *dw;       // partial sums: [workgroup][D] (null: not wanted)
    float *inv_rms;  // V == 0 with dw: r of every row, for the column pass
    int64_t ldy, lds, ldds, lddx;
    int rows, D;
    float eps;
};

// dX = r g - S r^3 mean(g S) + dS, g = dY w; a workgroup takes rows
// blockIdx.x, + gridDim.x, ... (times its rows at once) and keeps the sums
// dw = sum dY S r of its own columns in registers.  Threads and V as
// row_kernel; the form for any D leaves dw to a column pass over r.
template <int NT, int V>
__global__ void __launch_bounds__(NT > 256 ? NT : 256) row_grad_kernel(RowGradArgs a)
{
    constexpr int RPB = NT >= 256 ? 1 : 256 / NT;
    constexpr int VS = V > 0 ? V : 1;
    static_assert(RPB == 1 || NT == 64, "a row is one wave's or one workgroup's");
    __shared__ RowRed<NT> red[RPB == 1 ? 2 : 1];
    // short rows: the waves' dw sums meet here
    __shared__ __attribute__((aligned(16))) float dw_lds[RPB == 1 ? 4 : (RPB - 1) * 256 * VS];
    const int t = RPB == 1 ? threadIdx.x : threadIdx.x & 63;
    const int sub = RPB == 1 ? 0 : threadIdx.x >> 6;
    const int D = a.D;
    const float inv_d = 1.0f / (float)D;
    float dw[VS][4], w[VS][4];
#pragma unroll
    for (int i = 0; i < VS; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dw[i][j] = 0.0f;
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
        row_poison<NT>(red, turn);
        float sum = 0.0f, dot = 0.0f;
        auto write = [&](int col, const float (&g)[4], const float (&x)[4], float r, float c) {
            float o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = r * g[j] - x[j] * c;
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
                    load_cols<4>(dy + col, col, D, y[i]);
                    load_cols<4>(s + col, col, D, x[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum += x[i][j] * x[i][j];
                    dot += y[i][j] * w[i][j] * x[i][j];
                }
            row_reduce<NT>(sum, dot, false, red, turn);
            const float r = 1.0f / sqrtf(sum * inv_d + a.eps);
            const float c = dot * inv_d * r * r * r;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = 4 * (i * NT + t);
                if (col < D) {
                    float g[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] = y[i][j] * w[i][j];
                        dw[i][j] += y[i][j] * (x[i][j] * r);
                    }
                    write(col, g, x[i], r, c);
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
            for (int64_t col = 4 * t; col < D; col += 4 * NT) {
                float g[4], x[4];
                load((int)col, g, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum += x[j] * x[j];
                    dot += g[j] * x[j];
                }
            }
            row_reduce<NT>(sum, dot, false, red, turn);
            const float r = 1.0f / sqrtf(sum * inv_d + a.eps);
            const float c = dot * inv_d * r * r * r;
            for (int64_t col = 4 * t; col < D; col += 4 * NT) {
                float g[4], x[4];
                load((int)col, g, x);
                write((int)col, g, x, r, c);
            }
            if (a.inv_rms && t == 0) a.inv_rms[row] = r;
        }
        turn ^= RPB == 1 ? 1 : 0;
    }
    if constexpr (V > 0) {
        if (!a.dw) return;
        float *out = a.dw + (int64_t)blockIdx.x * D;
        if constexpr (RPB > 1) {
            if constexpr (kLdsPoison) {
                for (int i = threadIdx.x; i < (RPB - 1) * 256 * VS; i += 256) lds_poison(&dw_lds[i], 1);
                lds_poison_done();
                __syncthreads();
            }
            // waves 1..3 hand their sums to wave 0, which adds them in order
            if (sub > 0) {
#pragma unroll
                for (int i = 0; i < VS; ++i)
                    *reinterpret_cast<f32x4 *>(&dw_lds[(((sub - 1) * VS + i) * 64 + t) * 4]) =
                        f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
            }
            __syncthreads();
            if (sub > 0) return;
#pragma unroll
            for (int v = 0; v < RPB - 1; ++v)
#pragma unroll
                for (int i = 0; i < VS; ++i) {
                    const f32x4 q = *reinterpret_cast<const f32x4 *>(&dw_lds[((v * VS + i) * 64 + t) * 4]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dw[i][j] += q[j];
                }
        }
#pragma unroll
        for (int i = 0; i < VS; ++i) {
            const int col = 4 * (i * NT + t);
            if (col < D) store_row<4>(out + col, col, D, dw[i], 1.0f, 0.0f);
        }
    }
}

// ---- column sums -----------------------------------------------------------------
// What a column pass computes per element before it is summed over the rows.
constexpr int kColAct = 0;   // dY * act'(Z) (stored to dZ when wanted)
constexpr int kColNorm = 1;  // dY * S * r[row]: the weight gradient of long rows

struct ColArgs {
    const float *Y, *Z, *r;  // kColAct: dY, Z; kColNorm: dY, S, r
    float *out;              // kColAct: dZ or null
    float *part;             // [chunk][N] sums, or null
    int64_t ldy, ldz, ldo;
    int M, N, act;
    int rows_per_chunk;
};

// A workgroup covers 4 TX columns of one chunk of rows (blockIdx.y), TX = 64
// or 16 lanes along the columns and 256 / TX rows at a time.  A lane reads
// its next row before it works on the present one and stores it: loads and
// stores retire in order on one counter, so a row read after a store would wait
// for that store (512 x 8192 with gelu: 14.1 us without, 13.5 so; two or four
// rows at once are 14.9 and 15.1, as they leave less of the slope's arithmetic
// to overlap).
template <int KIND, int TX>
__global__ void __launch_bounds__(256) col_kernel(ColArgs a)
{
    constexpr int TY = 256 / TX;
    __shared__ __attribute__((aligned(16))) float red[(TY - 1) * TX * 4];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int64_t col64 = 4 * ((int64_t)blockIdx.x * TX + tx);
    const bool in = col64 < a.N;
    const int col = in ? (int)col64 : 0;
    const int64_t m0 = (int64_t)blockIdx.y * a.rows_per_chunk;
    const int64_t m1 = m0 + a.rows_per_chunk < a.M ? m0 + a.rows_per_chunk : a.M;
    constexpr bool NORM = KIND == kColNorm;
    const bool reads_z = NORM || a.act != SGEMM_ACT_NONE;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
        typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
        const bool whole = col + 3 < a.N;
        f32x4 y = {}, z = {};
        float r = 0.0f;
        auto read = [&](int64_t m) {
            const float *const py = a.Y + m * a.ldy + col, *const pz = a.Z + m * a.ldz + col;
            if (whole) {
                y = *reinterpret_cast<const f32x4u *>(py);
                if (reads_z) z = *reinterpret_cast<const f32x4u *>(pz);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[j] = col + j < a.N ? py[j] : 0.0f;
                    if (reads_z) z[j] = col + j < a.N ? pz[j] : 0.0f;
                }
            }
            if constexpr (NORM) r = a.r[m];
        };
        int64_t m = m0 + ty;
        if (m < m1) read(m);
        while (m < m1) {
            f32x4 x = y, s = z;
            const float f = r;
            const int64_t at = m;
            m += TY;
            if (m < m1) read(m);
            if constexpr (NORM) {
                x *= s * f;
            } else if (reads_z) {
                epi_map<true>(a.act, s);
                x *= s;
            }
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += v[j] = x[j];
            if constexpr (!NORM)
                if (a.out) store_row<4>(a.out + at * a.ldo + col, col, a.N, v, 1.0f, 0.0f);
        }
    }
    if (!a.part) return;  // (the same for every thread)
    if constexpr (kLdsPoison) {
        for (int i = threadIdx.x; i < (TY - 1) * TX * 4; i += 256) lds_poison(&red[i], 1);
        lds_poison_done();
        __syncthreads();
    }
    if (ty > 0) *reinterpret_cast<f32x4 *>(&red[((ty - 1) * TX + tx) * 4]) = f32x4{sum[0], sum[1], sum[2], sum[3]};
    __syncthreads();
    if (ty > 0 || !in) return;
#pragma unroll
    for (int i = 0; i < TY - 1; ++i) {
        const f32x4 q = *reinterpret_cast<const f32x4 *>(&red[(i * TX + tx) * 4]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += q[j];
    }
    store_row<4>(a.part + (int64_t)blockIdx.y * a.N + col, col, a.N, sum, 1.0f, 0.0f);
}

// out[n] = part[0][n] + part[1][n] + ...: 8 lanes along the columns (32 of
// them) and 128 along the parts, each adding every 128th in order, then their
// sums in two fixed stages.  The many threads keep the chain of dependent reads
// short: 1024 parts of 64 columns take 3 us, with 256 threads 8.
constexpr int kColSumThreads = 1024;
__global__ void __launch_bounds__(kColSumThreads) col_sum_kernel(const float *part, int parts, int N, float *out)
{
    constexpr int TX = 8, TY = kColSumThreads / TX, C = 4 * TX, S = 8;  // S sums of TY / S in the first stage
    __shared__ __attribute__((aligned(16))) float red[TY * C];
    __shared__ float red2[S * C];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int64_t col64 = (int64_t)C * blockIdx.x + 4 * tx;
    const bool in = col64 < N;
    const int col = in ? (int)col64 : 0;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
#pragma unroll 4
        for (int p = ty; p < parts; p += TY) {
            float q[4];
            load_cols<4>(part + (int64_t)p * N + col, col, N, q);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += q[j];
        }
    }
    if constexpr (kLdsPoison) {
        for (int i = threadIdx.x; i < TY * C; i += kColSumThreads) lds_poison(&red[i], 1);
        if (threadIdx.x < S * C) lds_poison(&red2[threadIdx.x], 1);
        lds_poison_done();
        __syncthreads();
    }
    *reinterpret_cast<f32x4 *>(&red[ty * C + 4 * tx]) = f32x4{sum[0], sum[1], sum[2], sum[3]};
    __syncthreads();
    const int c = threadIdx.x % C, s = threadIdx.x / C;
    if (s < S) {
        float v = red[s * (TY / S) * C + c];
#pragma unroll
        for (int i = 1; i < TY / S; ++i) v += red[(s * (TY / S) + i) * C + c];
        red2[s * C + c] = v;
    }
    __syncthreads();
    const int64_t n = (int64_t)C * blockIdx.x + threadIdx.x;
    if (threadIdx.x >= C || n >= N) return;
    float v = red2[threadIdx.x];
#pragma unroll
    for (int i = 1; i < S; ++i) v += red2[i * C + threadIdx.x];
    out[n] = v;
}

// Zeros (the column sums of no rows; a fill that a graph may capture).
__global__ void __launch_bounds__(256) fill_zero_kernel(float *p, int n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

}  // namespace sgemm
