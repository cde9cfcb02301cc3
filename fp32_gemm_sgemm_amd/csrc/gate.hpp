// The epilogue of a gated feed-forward block, and the elementwise part of its
// gradient.
//
//   g = sum A Bg + bg,  u = sum A Bu + bu   (8-bit operands: times their scales)
//   C = act(g) * u,     g and u also stored where the gradient will need them
//
//   dg = dY * u * act'(g),  du = dY * act(g),  dbg, dbu their column sums
//
// The activations are those of epilogue.hpp.
//
// The gradient is bound by memory: three matrices read, two written and the sums kept
// in registers, 2048 x 8192 in 62 us (5.5 TB/s).  515 x 2051 takes 9.8 us and the sums'
// second kernel 4: each workgroup has two or four rows of a thread, one after the other.
#pragma once

#include "common.hpp"
#include "epilogue.hpp"
#include "rowops.hpp"

namespace sgemm {

// Device pointers of one call (null: that part is left out).
struct Gate {
    const float *scale_a, *scale_gate, *scale_up;  // 8-bit operands
    const float *bias_gate, *bias_up;
    float *pre_gate, *pre_up;
    int64_t ld_pre_gate, ld_pre_up;
    int act;
};

// The gated block of W adjacent pairs of sums (row `row`, columns col .. col +
// W - 1, masked to N), left in g.
template <int W>
__device__ __forceinline__ void gate_apply(const Gate &e, int row, int col, int N, float (&g)[W], float (&u)[W])
{
    const float sa = e.scale_a ? load_global(e.scale_a + row) : 1.0f;
    // (one scale after the other: their product may leave float32 where the sum's does not)
    auto affine = [&](const float *scale, const float *bias, float (&v)[W]) {
        float x[W];
        if (e.scale_a) {
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] *= sa;
        }
        if (scale) {
            load_cols<W>(scale + col, col, N, x);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] *= x[j];
        }
        if (bias) {
            load_cols<W>(bias + col, col, N, x);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += x[j];
        }
    };
    affine(e.scale_gate, e.bias_gate, g);
    affine(e.scale_up, e.bias_up, u);
    if (e.pre_gate) store_row<W>(e.pre_gate + row * e.ld_pre_gate + col, col, N, g, 1.0f, 0.0f);
    if (e.pre_up) store_row<W>(e.pre_up + row * e.ld_pre_up + col, col, N, u, 1.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < W; ++j) g[j] = act_value(e.act, g[j]) * u[j];
}

// The gated block of one wave's sums, staged in the wave's own LDS region: R
// rows of WT gate sums, then R rows of WT up sums.  Row rr of the region is row
// row0 + RS * rr of C, the first column is col0.  As in StagedEpi the
// activation's code stands once, in a rolled loop, and every access to memory
// is 16 bytes a lane along a row; nothing but the columns' biases and scales is
// read, so no store is waited for.  Without C only pre_gate and pre_up are
// written (the partial sums of a K split).
template <int R, int WT, int RS, bool SCALES> struct StagedGate {
    static constexpr int QR = WT / 4;     // 16-byte groups per row
    static constexpr int STEP = 64 / QR;  // rows a wave covers at once
    static constexpr int STEPS = R / STEP;
    static_assert(64 % QR == 0 && R % STEP == 0 && R <= 64, "whole wave steps");

    const Gate &e;
    float *const C;
    const int64_t ldc;
    const int M, N, lane, col0;
    f32x4 scale_gate, scale_up, bias_gate, bias_up;

    __device__ __forceinline__ int col() const { return col0 + 4 * (lane % QR); }

    __device__ __forceinline__ f32x4 columns(const float *p, float other) const
    {
        if (!p) return f32x4{other, other, other, other};
        float x[4];
        load_cols<4>(p + col(), col(), N, x);
        return f32x4{x[0], x[1], x[2], x[3]};
    }

    __device__ __forceinline__ StagedGate(const Gate &gate, float *c, int64_t ld, int m, int n, int l, int c0)
        : e(gate), C(c), ldc(ld), M(m), N(n), lane(l), col0(c0)
    {
        if (SCALES) {
            scale_gate = columns(e.scale_gate, 1.0f);
            scale_up = columns(e.scale_up, 1.0f);
        }
        bias_gate = columns(e.bias_gate, 0.0f);
        bias_up = columns(e.bias_up, 0.0f);
    }

    // The scale of the region's row `lane` (of R), to be read for all regions
    // before the first is stored.
    __device__ __forceinline__ float row_scale(int row0) const
    {
        if (!SCALES || !e.scale_a) return 1.0f;
        return load_global(e.scale_a + min(row0 + RS * (lane % R), M - 1));
    }

    __device__ __forceinline__ void store(const float *lds, int row0, float row_scale) const
    {
        const int cc = 4 * (lane % QR), rl = lane / QR;
        const bool whole = col0 + WT <= N;  // (the same for the wave)
        auto write = [&](float *p, const f32x4 &v) {
            if (whole) {
                *reinterpret_cast<f32x4u *>(p) = v;
            } else {
                const float x[4] = {v[0], v[1], v[2], v[3]};
                store_row<4>(p, col(), N, x, 1.0f, 0.0f);
            }
        };
#pragma unroll 1
        for (int i = 0; i < STEPS; ++i) {
            const int rr = rl + i * STEP;
            const int row = row0 + RS * rr;
            const float sa = SCALES ? __shfl(row_scale, rr) : 1.0f;
            const float *const p = lds + rr * WT + cc;
            f32x4 g = *reinterpret_cast<const f32x4 *>(p), u = *reinterpret_cast<const f32x4 *>(p + R * WT);
            if (SCALES) {
                g = g * sa * scale_gate;
                u = u * sa * scale_up;
            }
            g += bias_gate;
            u += bias_up;
            const bool in = row < M && col() < N;
            if (in && e.pre_gate) write(e.pre_gate + row * e.ld_pre_gate + col(), g);
            if (in && e.pre_up) write(e.pre_up + row * e.ld_pre_up + col(), u);
            if (!C) continue;
            epi_map<false>(e.act, g);
            if (in) write(C + row * ldc + col(), g * u);
        }
    }
};

// ---- two products' sums from a workspace ---------------------------------------------------

// G and U as `splits` partial sums each (a K split's; 0: none, K is empty), in
// rows of ldp floats: P[which][split][M][ldp].
struct GateReduceArgs {
    const float *P;
    float *C;
    int64_t split_p, half_p, quads;  // quads: M * ldp / 4
    int64_t base;                    // this launch's first
    int M, N, ldp, ldc, splits;
    Gate e;
};

__global__ void __launch_bounds__(256) gate_reduce_kernel(GateReduceArgs r)
{
    const int64_t q = r.base + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= r.quads) return;
    const int qpr = r.ldp >> 2;
    const int row = (int)(q / qpr);
    const int col = 4 * (int)(q - (int64_t)row * qpr);
    if (col >= r.N) return;
    f32x4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (r.splits > 0) {
            const float *p = r.P + h * r.half_p + (int64_t)row * r.ldp + col;
            s[h] = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll 4
            for (int t = 1; t < r.splits; ++t) s[h] += *reinterpret_cast<const f32x4 *>(p + t * r.split_p);
        }
    }
    float g[4], u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        g[j] = s[0][j];
        u[j] = s[1][j];
    }
    gate_apply<4>(r.e, row, col, r.N, g, u);
    store_row<4>(r.C + (int64_t)row * r.ldc + col, col, r.N, g, 1.0f, 0.0f);
}

// ---- gradient --------------------------------------------------------------------------------

struct GateGradArgs {
    const float *dY, *G, *U;
    float *dG, *dU;  // null: not wanted
    float *part;     // [chunk][2 N] sums of dG, then of dU, or null
    int64_t ldy, ldg, ldu, lddg, lddu;
    int M, N, act, rows_per_chunk;
};

// act(v) and act'(v) of four values: one branch for all of them.
__device__ __forceinline__ void act_both(int act, const f32x4 &v, f32x4 &value, f32x4 &slope)
{
    value = v;
    slope = v;
    epi_map<false>(act, value);
    epi_map<true>(act, slope);
}

// Geometry as col_kernel: a workgroup covers 4 TX columns of one chunk of rows,
// 256 / TX rows at a time, and reads its next row before it works on the
// present one and stores it.
template <int TX> __global__ void __launch_bounds__(256) gate_grad_kernel(GateGradArgs a)
{
    constexpr int TY = 256 / TX;
    __shared__ __attribute__((aligned(16))) float red[(TY - 1) * TX * 8];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int64_t col64 = 4 * ((int64_t)blockIdx.x * TX + tx);
    const bool in = col64 < a.N;
    const int col = in ? (int)col64 : 0;
    const int64_t m0 = (int64_t)blockIdx.y * a.rows_per_chunk;
    const int64_t m1 = m0 + a.rows_per_chunk < a.M ? m0 + a.rows_per_chunk : a.M;
    f32x4 sg = {0.0f, 0.0f, 0.0f, 0.0f}, su = sg;
    if (in) {
        f32x4 y = {}, g = {}, u = {};
        auto read = [&](int64_t m) {
            float v[3][4];
            load_cols<4>(a.dY + m * a.ldy + col, col, a.N, v[0]);
            load_cols<4>(a.G + m * a.ldg + col, col, a.N, v[1]);
            load_cols<4>(a.U + m * a.ldu + col, col, a.N, v[2]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = v[0][j];
                g[j] = v[1][j];
                u[j] = v[2][j];
            }
        };
        auto write = [&](float *p, const f32x4 &x) {
            const float v[4] = {x[0], x[1], x[2], x[3]};
            store_row<4>(p, col, a.N, v, 1.0f, 0.0f);
        };
        int64_t m = m0 + ty;
        if (m < m1) read(m);
        while (m < m1) {
            const f32x4 dy = y, up = u, z = g;
            const int64_t at = m;
            m += TY;
            if (m < m1) read(m);
            f32x4 value, slope;
            act_both(a.act, z, value, slope);
            const f32x4 dg = dy * up * slope, du = dy * value;
            sg += dg;
            su += du;
            if (a.dG) write(a.dG + at * a.lddg + col, dg);
            if (a.dU) write(a.dU + at * a.lddu + col, du);
        }
    }
    if (!a.part) return;  // (the same for every thread)
    if constexpr (kLdsPoison) {
        for (int i = threadIdx.x; i < (TY - 1) * TX * 8; i += 256) lds_poison(&red[i], 1);
        lds_poison_done();
        __syncthreads();
    }
    if (ty > 0) {
        f32x4 *const p = reinterpret_cast<f32x4 *>(&red[((ty - 1) * TX + tx) * 8]);
        p[0] = sg;
        p[1] = su;
    }
    __syncthreads();
    if (ty > 0 || !in) return;
#pragma unroll
    for (int i = 0; i < TY - 1; ++i) {
        const f32x4 *const p = reinterpret_cast<const f32x4 *>(&red[(i * TX + tx) * 8]);
        sg += p[0];
        su += p[1];
    }
    float *const out = a.part + (int64_t)blockIdx.y * (2 * (int64_t)a.N);
    const float x[4] = {sg[0], sg[1], sg[2], sg[3]}, v[4] = {su[0], su[1], su[2], su[3]};
    store_row<4>(out + col, col, a.N, x, 1.0f, 0.0f);
    store_row<4>(out + a.N + col, col, a.N, v, 1.0f, 0.0f);
}

}  // namespace sgemm
