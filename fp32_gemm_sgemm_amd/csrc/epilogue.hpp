// The epilogue of a product: bias, activation (or the derivative of one) and
// residual, applied to a result while it is still in registers or LDS, so the
// product's output makes one trip to memory instead of one per operation.
//
//   z = alpha * sum + bias[n]
//   y = act(z)                      (z also stored when `pre` is set), or
//   y = z * act'(grad_pre[m][n])    when `grad_pre` is set,
//   C = y + residual[m][n]
//
// The activations, with sigma(t) = 1 / (1 + exp(-t)) and Phi the normal
// distribution function:
//   relu       max(z, 0), NaN kept          derivative  1 where z > 0, else 0
//   gelu       z Phi(z)                                  Phi(z) + z phi(z)
//   gelu_tanh  z sigma(2u), u = c (z + a z^3): the tanh form, since
//              (1 + tanh u) / 2 = sigma(2u); c = sqrt(2/pi), a = 0.044715
//                                          s + 2c z s (1 - s) (1 + 3 a z^2)
//   silu       z sigma(z)                                s (1 + z (1 - s))
// Everything is float32, on the hardware's 2^x and reciprocal (about one unit
// in the last place each).  Phi is computed from
// its own polynomial (gelu_terms): without branches, and with its relative
// accuracy kept in the lower tail, where (1 + erf) / 2 cancels.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "sgemm_ops.h"

namespace sgemm {

// Device pointers of one launch (null: that part is left out).  `ld_*` are
// row strides and `batch_*` the elements between batch entries.
struct Epi {
    const float *scale_a, *scale_b;  // 8-bit operands: a factor per row and per column of C
    const float *bias;
    float *pre;
    const float *grad_pre;
    const float *residual;
    int64_t batch_bias, batch_pre, batch_grad_pre, batch_residual;
    int ld_pre, ld_grad_pre, ld_residual;
    int act;
};

// One float of global memory.  (The compiler may lose track of a pointer's
// address space on its way through a modified argument struct, and a generic
// load also occupies the LDS counter.)
__device__ __forceinline__ float load_global(const float *p)
{
    typedef const __attribute__((address_space(1))) float global_float;
    return *(global_float *)(uintptr_t)p;
}

// exp(-t) for t >= 0 (infinity and NaN give 0), within about 2 units in the last
// place down to 2^-126 and 0 below: the hardware's 2^x of t log2(e) carried in
// two parts.  (The math library's expf takes three times the instructions for
// the arguments that cannot occur here; a 256 x 256 tile's epilogue is bound by
// them.)
__device__ __forceinline__ float exp_neg(float t)
{
#pragma clang fp contract(off)
    constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147181f;
    const float x = fminf(t, 200.0f);
    const float hi = x * kLog2e;
    const float lo = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -hi));
    const float r = __builtin_amdgcn_exp2f(-hi);
    return __builtin_fmaf(r, -kLn2 * lo, r);
}

// sigma(t) and 1 - sigma(t), each with its own relative accuracy: from
// exp(-|t|), which neither overflows nor cancels.  (NaN gives 1 and 0: what they
// are multiplied by is NaN then.)
__device__ __forceinline__ float sigmoid_f32(float t, float &rest)
{
    const float e = exp_neg(fabsf(t));
    const float q = __builtin_amdgcn_rcpf(1.0f + e), p = e * q;
    rest = t < 0.0f ? q : p;
    return t < 0.0f ? p : q;
}
__device__ __forceinline__ float sigmoid_f32(float t)
{
    float rest;
    return sigmoid_f32(t, rest);
}

constexpr float kGeluC = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752440f;
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;

// Phi(z) and exp(-z^2 / 2).  With a = |z| / sqrt 2 the tail is
//   Phi(-|z|) = erfc(a) / 2 = exp(-a^2) t P(t) / 2,  t = 1 / (1 + a / 2),
// Hastings' form of the error function (Approximations for Digital Computers,
// 1955; Abramowitz and Stegun 7.1.26) with another step in t and of higher
// degree: P, of degree 8, is fitted here to exp(a^2) erfc(a) / t in relative
// error over a in [0, 10.6] (4.4e-8).  The exponent is z^2 / 2 of z itself with
// the square's rounding carried: from the rounded a it would move the
// exponential by a^2 times a's rounding, 1.2e-5 at z = -12.8.  Measured over
// z in [-12.9, 0]: gelu within 5e-7 of its value.  Past |z| = 14.85 the
// exponential is 0 in float32.
__device__ __forceinline__ void gelu_terms(float z, float &phi_cdf, float &gauss)
{
#pragma clang fp contract(off)  // s is the rounded square wherever it is used
    const float x = fminf(fabsf(z), 14.85f);
    const float s = x * x;
    gauss = exp_neg(0.5f * s) * (1.0f - 0.5f * __builtin_fmaf(x, x, -s));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f * kSqrtHalf, x, 1.0f));
    float p = -0.05921298f;
    p = __builtin_fmaf(p, t, 0.28527875f);
    p = __builtin_fmaf(p, t, -0.48865957f);
    p = __builtin_fmaf(p, t, 0.27973996f);
    p = __builtin_fmaf(p, t, -0.02778005f);
    p = __builtin_fmaf(p, t, 0.20317615f);
    p = __builtin_fmaf(p, t, 0.24297989f);
    p = __builtin_fmaf(p, t, 0.28239236f);
    p = __builtin_fmaf(p, t, 0.28208544f);
    const float tail = 0.5f * gauss * (t * p);
    phi_cdf = z > 0.0f ? 1.0f - tail : tail;
}

// Past |z| = 16 the sigmoid of gelu_tanh is exactly 0 or 1 in float32
// (exp(-317)); clamping there keeps z^3 finite.  NaN passes.
__device__ __forceinline__ float gelu_clamp(float z)
{
    return z > 16.0f ? 16.0f : (z < -16.0f ? -16.0f : z);
}

__device__ __forceinline__ float act_value(int act, float z)
{
    switch (act) {
    case SGEMM_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case SGEMM_ACT_GELU: {
        float cdf, gauss;
        gelu_terms(z, cdf, gauss);
        return z * cdf;
    }
    case SGEMM_ACT_GELU_TANH: {
        const float c = gelu_clamp(z);
        return z * sigmoid_f32(2.0f * kGeluC * (c + kGeluA * c * c * c));
    }
    case SGEMM_ACT_SILU: return z * sigmoid_f32(z);
    default: return z;
    }
}

__device__ __forceinline__ float act_slope(int act, float z)
{
    switch (act) {
    case SGEMM_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case SGEMM_ACT_GELU: {
        float cdf, gauss;
        gelu_terms(z, cdf, gauss);
        return cdf + z * (kInvSqrt2Pi * gauss);
    }
    case SGEMM_ACT_GELU_TANH: {
        const float c = gelu_clamp(z);
        float rest;
        const float s = sigmoid_f32(2.0f * kGeluC * (c + kGeluA * c * c * c), rest);
        return s + 2.0f * kGeluC * c * s * rest * (1.0f + 3.0f * kGeluA * c * c);
    }
    case SGEMM_ACT_SILU: {
        float rest;
        const float s = sigmoid_f32(z, rest);
        return s * (1.0f + z * rest);
    }
    default: return 1.0f;
    }
}

// W adjacent floats at p, of which those at columns below N exist (col is the
// first one's column); the others read as zero.
template <int W>
__device__ __forceinline__ void load_cols(const float *p, int col, int N, float (&x)[W])
{
    if constexpr (W > 1) {
        if (col + W - 1 < N) {
            typedef float vec_t __attribute__((ext_vector_type(W), aligned(4)));
            const vec_t v = *reinterpret_cast<const vec_t *>(p);
#pragma unroll
            for (int j = 0; j < W; ++j) x[j] = v[j];
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) x[j] = col + j < N ? p[j] : 0.0f;
}

// Applies the epilogue of batch entry z to W adjacent results v (already
// scaled by alpha) of row `row`, columns col .. col + W - 1 (masked to N).
template <int W>
__device__ __forceinline__ void epi_apply(const Epi &e, int z, int row, int col, int N, float (&v)[W])
{
    float x[W];
    if (e.scale_a) {
        const float s = load_global(e.scale_a + row);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= s;
    }
    if (e.scale_b) {
        load_cols<W>(e.scale_b + col, col, N, x);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= x[j];
    }
    if (e.bias) {
        load_cols<W>(e.bias + z * e.batch_bias + col, col, N, x);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += x[j];
    }
    if (e.grad_pre) {
        load_cols<W>(e.grad_pre + z * e.batch_grad_pre + (int64_t)row * e.ld_grad_pre + col, col, N, x);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= act_slope(e.act, x[j]);
    } else {
        if (e.pre)
            store_row<W>(e.pre + z * e.batch_pre + (int64_t)row * e.ld_pre + col, col, N, v, 1.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = act_value(e.act, v[j]);
    }
    if (e.residual) {
        load_cols<W>(e.residual + z * e.batch_residual + (int64_t)row * e.ld_residual + col, col, N, x);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += x[j];
    }
}

// A product's arguments with an epilogue (beta is not used: the residual
// takes its place).
struct EpiGemmArgs : GemmArgs {
    Epi e;
};

// Kernel argument of the GEMM kernels with (EPI) and without an epilogue.
template <bool EPI> struct KernelArgs { typedef GemmArgs T; };
template <> struct KernelArgs<true> { typedef EpiGemmArgs T; };

// act (SLOPE: act') of four values: one branch for all of them.
template <bool SLOPE> __device__ __forceinline__ void epi_map(int act, f32x4 &v)
{
    auto map = [&](auto a) {
        constexpr int ACT = decltype(a)::value;
        f32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = SLOPE ? act_slope(ACT, v[j]) : act_value(ACT, v[j]);
        v = r;
    };
    if (act == SGEMM_ACT_RELU) map(std::integral_constant<int, SGEMM_ACT_RELU>());
    else if (act == SGEMM_ACT_GELU) map(std::integral_constant<int, SGEMM_ACT_GELU>());
    else if (act == SGEMM_ACT_GELU_TANH) map(std::integral_constant<int, SGEMM_ACT_GELU_TANH>());
    else if (act == SGEMM_ACT_SILU) map(std::integral_constant<int, SGEMM_ACT_SILU>());
    else if (SLOPE) map(std::integral_constant<int, SGEMM_ACT_NONE>());
}

// The epilogue of one wave's results, staged R rows at a time in the wave's own
// LDS region as rows of WT floats (16-byte aligned).  Row rr of the region is
// row row0 + RS * rr of C; the first column, col0, is the same for all of a
// wave's regions.
//
// The activation's code is in rolled loops over the region, so it stands once
// however many accumulators the wave holds.  Every access to C, `pre`,
// `grad_pre` and the residual is 16 bytes per lane along a row: a lane keeps
// its four columns (bias and column scales are read once) and walks down the
// rows.  Loads and stores retire in order on one counter, so a load issued
// after a store waits for it: reads are issued B steps at a time before the
// stores of those rows, and nothing is read in between (with one step at a time
// a 2048 x 2048 x 1024 product of 8-bit operands spent 13 of its 29 us waiting
// for its own stores).  SCALES: row and column scales may be given.
//
// What it costs, on the float32 256x256 tile at 2048 x 8192 x 2048 (one tile per
// compute unit, so nothing hides it): the product alone 462 us, with bias 462,
// with gelu and the stored pre-activation 475, with a residual 472, with gelu's
// slope 479; the same product and the passes over its output one after the
// other take 606.  Tiles that reach past the last row or column run the same
// steps with masks (1728 x 1292 x 494 with bias: 37.0 us, 39.1 when each step
// waited for its own store; 8-bit 1000 x 1000 x 1000: 12.6 against 14.2).
template <int R, int WT, int RS, bool SCALES> struct StagedEpi {
    static constexpr int QR = WT / 4;     // 16-byte groups per row
    static constexpr int STEP = 64 / QR;  // rows a wave covers at once
    static constexpr int STEPS = R / STEP;
    static constexpr int BF = STEPS < 8 ? STEPS : SCALES ? 8 : 4;  // steps whose reads are in flight together
    static constexpr int BE = BF < 4 ? BF : BF / 2;                // and at an edge (more would take registers from the loop)
    static constexpr int RSTEP = RS * STEP;
    static_assert(64 % QR == 0 && R % STEP == 0 && STEPS % BF == 0 && STEPS % BE == 0 && R <= 64, "whole wave steps");

    const EpiGemmArgs &g;
    const int z, lane, col0;
    f32x4 scale, bias;

    __device__ __forceinline__ int col() const { return col0 + 4 * (lane % QR); }

    __device__ __forceinline__ StagedEpi(const EpiGemmArgs &args, int batch, int l, int c0)
        : g(args), z(batch), lane(l), col0(c0)
    {
        scale = f32x4{g.alpha, g.alpha, g.alpha, g.alpha};
        bias = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (SCALES && g.e.scale_b) scale = columns(g.e.scale_b);
        if (g.e.bias) bias = columns(g.e.bias + z * g.e.batch_bias);
    }

    // The lane's four columns of a row vector, zeros past N.
    __device__ __forceinline__ f32x4 columns(const float *p) const
    {
        if (col0 + WT <= g.N) return *reinterpret_cast<const f32x4u *>(p + col());
        float x[4];
        load_cols<4>(p + col(), col(), g.N, x);
        return f32x4{x[0], x[1], x[2], x[3]};
    }

    // The scale of the region's row `lane` (of R), to be read for all regions
    // before the first is stored.
    __device__ __forceinline__ float row_scale(int row0) const
    {
        if (!SCALES || !g.e.scale_a) return 1.0f;
        return load_global(g.e.scale_a + min(row0 + RS * (lane % R), g.M - 1));
    }

    __device__ __forceinline__ void store(float *lds, int row0, float row_scale) const
    {
        if (col0 + WT > g.N || row0 + RS * (R - 1) >= g.M) store_form<true>(lds, row0, row_scale);
        else store_form<false>(lds, row0, row_scale);
    }

    // EDGE: the region reaches past the last row or column; reads and writes
    // are masked, in the same order.
    template <bool EDGE> __device__ __forceinline__ void store_form(float *lds, int row0, float row_scale) const
    {
        constexpr int B = EDGE ? BE : BF;
        const Epi &e = g.e;
        const int cc = 4 * (lane % QR), rl = lane / QR;
        const int row = row0 + RS * rl;
        // steps in which this lane has a row and a column
        const int mine = !EDGE ? STEPS : col0 + cc < g.N ? (g.M - row + RSTEP - 1) / RSTEP : 0;
        float *const src = lds + rl * WT + cc;
        // (with a null base these addresses are never used)
        const float *gp = e.grad_pre + z * e.batch_grad_pre + (int64_t)row * e.ld_grad_pre + col();
        const float *res = e.residual + z * e.batch_residual + (int64_t)row * e.ld_residual + col();
        float *pre = e.pre + z * e.batch_pre + (int64_t)row * e.ld_pre + col();
        float *out = g.C + (int64_t)row * g.ldc + col();
        auto read = [&](const float *p, int i, int64_t ld) {
            p += i * RSTEP * ld;
            if constexpr (EDGE) {
                float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (i < mine) load_cols<4>(p, col(), g.N, x);
                return f32x4{x[0], x[1], x[2], x[3]};
            } else {
                return (f32x4)*reinterpret_cast<const f32x4u *>(p);
            }
        };
        auto write = [&](float *p, int i, int64_t ld, const f32x4 &v) {
            p += i * RSTEP * ld;
            if constexpr (EDGE) {
                const float x[4] = {v[0], v[1], v[2], v[3]};
                if (i < mine) store_row<4>(p, col(), g.N, x, 1.0f, 0.0f);
            } else {
                *reinterpret_cast<f32x4u *>(p) = v;
            }
        };
        // z of step i from its staged sum
        auto linear = [&](int i, const f32x4 &s) {
            const float sa = SCALES ? __shfl(row_scale, rl + i * STEP) : 1.0f;
            return s * sa * scale + bias;
        };
#pragma unroll 1
        for (int i0 = 0; i0 < STEPS; i0 += B) {
            float *const at = src + i0 * (STEP * WT);
            f32x4 y[B], v[B];
            if (e.residual)
#pragma unroll
                for (int b = 0; b < B; ++b)
                    y[b] = read(res, i0 + b, e.ld_residual);
            if (e.grad_pre) {
                // the sums to registers, grad_pre in their place
#pragma unroll
                for (int b = 0; b < B; ++b)
                    v[b] = read(gp, i0 + b, e.ld_grad_pre);
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    f32x4 *const p = reinterpret_cast<f32x4 *>(at + b * (STEP * WT));
                    const f32x4 s = *p;
                    *p = v[b];
                    v[b] = s;
                }
#pragma unroll 1
                for (int b = 0; b < B; ++b) {
                    f32x4 *const p = reinterpret_cast<f32x4 *>(at + b * (STEP * WT));
                    f32x4 x = *p;
                    epi_map<true>(e.act, x);
                    *p = x;
                }
#pragma unroll
                for (int b = 0; b < B; ++b)
                    v[b] = linear(i0 + b, v[b]) * *reinterpret_cast<const f32x4 *>(at + b * (STEP * WT));
            } else if (e.act == SGEMM_ACT_NONE) {
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    v[b] = linear(i0 + b, *reinterpret_cast<const f32x4 *>(at + b * (STEP * WT)));
                    if (e.pre) write(pre, i0 + b, e.ld_pre, v[b]);
                }
            } else {
#pragma unroll 1
                for (int b = 0; b < B; ++b) {
                    f32x4 *const p = reinterpret_cast<f32x4 *>(at + b * (STEP * WT));
                    f32x4 x = linear(i0 + b, *p);
                    if (e.pre) write(pre, i0 + b, e.ld_pre, x);
                    epi_map<false>(e.act, x);
                    *p = x;
                }
#pragma unroll
                for (int b = 0; b < B; ++b) v[b] = *reinterpret_cast<const f32x4 *>(at + b * (STEP * WT));
            }
            if (e.residual)
#pragma unroll
                for (int b = 0; b < B; ++b) v[b] += y[b];
#pragma unroll
            for (int b = 0; b < B; ++b) write(out, i0 + b, g.ldc, v[b]);
        }
    }
};

}  // namespace sgemm
