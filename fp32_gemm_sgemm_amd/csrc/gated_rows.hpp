// The gated feed-forward block in float32 for few rows of A (single tokens):
// up to four rows at a time on vector FMAs, both weights streamed once from
// memory straight into registers.
//
// Bound by that stream: 8 bytes of weights against 2 operations a row, so the
// kernels' shape is what keeps many 16-byte loads in flight and nothing
// between them: one row and two weights of 8192 x 2048 take 23.2 us, 5.8 TB/s (29
// stored (K, N); the smallest tile 37).  The streams' order is the weights':
//
//   k-contiguous (weights stored (N, K)): a wave takes two columns' rows of
//     both weights, its lanes run along k.  A's rows are read along with them,
//     from L1 (every wave of a compute unit reads the same ones).
//   index-contiguous (stored (K, N)): a workgroup takes 32 columns, eight lanes
//     each reading a 128-byte row segment of both weights; its 128 lane groups
//     split K.  A is staged in LDS, kRowsChunk values of k at a time.
//
// Sums are added in a fixed order: per lane, by butterflies over the lanes, then
// the waves in order through LDS.  More rows of A than four are further rows of
// workgroups, each streaming the weights again: it is the form for calls that
// no tile serves (row strides past 32-bit offsets), not for speed.
#pragma once

#include "common.hpp"
#include "gate.hpp"
#include "layernorm.hpp"

namespace sgemm {

constexpr int kGatedRows = 4;  // rows of A a workgroup takes

struct GatedRowsArgs {
    const float *A, *B[2];  // B: the gate's weights, the other ones
    float *C;
    int64_t lda, ldb[2], ldc;
    int M, N, K;
    int m_base;      // this launch's first row and column
    int64_t n_base;
    Gate e;
};

// ---- weights stored (N, K) ---------------------------------------------------------------
// WK waves of a workgroup's four share two columns and split K; MR rows of A.
template <int MR, int WK> __global__ void __launch_bounds__(256) gated_rows_kc_kernel(GatedRowsArgs g)
{
    constexpr int P = 2;               // columns of a wave
    constexpr int COLS = P * (4 / WK);  // and of a workgroup
    __shared__ float red[4 * 2 * P * MR];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % WK;
    const int64_t x0 = g.n_base + (int64_t)blockIdx.x * COLS, n0 = x0 + P * (wave / WK);
    const int m0 = g.m_base + (int)blockIdx.y * kGatedRows;
    const int K = g.K;
    const float *b[2][P], *a[MR];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < P; ++p) b[h][p] = g.B[h] + (n0 + p < g.N ? n0 + p : g.N - 1) * g.ldb[h];
#pragma unroll
    for (int r = 0; r < MR; ++r) a[r] = g.A + min(m0 + r, g.M - 1) * g.lda;
    f32x4 acc[2][P][MR];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int r = 0; r < MR; ++r) acc[h][p][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int64_t k = 4 * (lane + 64 * part);
#pragma unroll 4
    for (; k + 3 < K; k += 256 * WK) {
        f32x4 w[2][P], x[MR];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p)
                w[h][p] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u *>(b[h][p] + k));
#pragma unroll
        for (int r = 0; r < MR; ++r) x[r] = *reinterpret_cast<const f32x4u *>(a[r] + k);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int r = 0; r < MR; ++r) acc[h][p][r] += w[h][p] * x[r];
    }
    if (k < K) {
        // the lane whose four values reach past K
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int r = 0; r < MR; ++r)
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (k + j < K) acc[h][p][r][j] += b[h][p][k + j] * a[r][k + j];
    }
    if constexpr (kLdsPoison) {
        if (threadIdx.x < 4 * 2 * P * MR) lds_poison(&red[threadIdx.x], 1);
        lds_poison_done();
        __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int r = 0; r < MR; ++r) {
                const f32x4 v = acc[h][p][r];
                const float s = wave_all<AddOp>((v[0] + v[1]) + (v[2] + v[3]));
                if (lane == 0) red[((wave * 2 + h) * P + p) * MR + r] = s;
            }
    __syncthreads();
    const int t = threadIdx.x;
    if (t >= COLS * MR) return;
    const int c = t / MR, r = t % MR;
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int at = ((c / P * WK * 2 + h) * P + c % P) * MR + r;
        s[h] = red[at];
#pragma unroll
        for (int q = 1; q < WK; ++q) s[h] += red[at + q * 2 * P * MR];
    }
    const int64_t col = x0 + c;
    const int row = m0 + r;
    if (row >= g.M || col >= g.N) return;
    float v[1] = {s[0]}, u[1] = {s[1]};
    gate_apply<1>(g.e, row, (int)col, g.N, v, u);
    g.C[row * g.ldc + col] = v[0];
}

// ---- weights stored (K, N) ---------------------------------------------------------------
constexpr int kRowsChunk = 4096;  // values of k staged at once
constexpr int kRowsThreads = 1024;

template <int MR> __global__ void __launch_bounds__(kRowsThreads) gated_rows_xc_kernel(GatedRowsArgs g)
{
    constexpr int XQ = 8, XB = 4 * XQ, GROUPS = kRowsThreads / XQ, W = kRowsThreads / 64;
    constexpr int STAGE = kRowsChunk * MR, RED = W * 2 * MR * XB;
    __shared__ __attribute__((aligned(16))) float lds[STAGE > RED ? STAGE : RED];
    const int tid = threadIdx.x, xq = tid % XQ, kg = tid / XQ;
    const int lane = tid & 63, wave = tid >> 6;
    const int64_t x0 = g.n_base + (int64_t)blockIdx.x * XB;
    const int64_t xc = x0 + 4 * xq;
    const int m0 = g.m_base + (int)blockIdx.y * kGatedRows;
    const int K = g.K, N = g.N;
    const bool whole = xc + 3 < N, some = xc < N;
    f32x4 acc[2][MR];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < MR; ++r) acc[h][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto poison = [&]() {
        if constexpr (kLdsPoison) {
            for (int i = tid; i < (STAGE > RED ? STAGE : RED); i += kRowsThreads) lds_poison(&lds[i], 1);
            lds_poison_done();
            __syncthreads();
        }
    };
    for (int64_t c0 = 0; c0 < K; c0 += kRowsChunk) {
        const int n = (int)(K - c0 < kRowsChunk ? K - c0 : kRowsChunk);
        poison();
#pragma unroll
        for (int r = 0; r < MR; ++r) {
            const float *const a = g.A + min(m0 + r, g.M - 1) * g.lda + c0;
            for (int i = tid; i < n; i += kRowsThreads) lds[i * MR + r] = a[i];
        }
        __syncthreads();
        auto step = [&](int i, const f32x4 (&w)[2]) {
            float x[MR];
#pragma unroll
            for (int r = 0; r < MR; ++r) x[r] = lds[i * MR + r];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < MR; ++r) acc[h][r] += w[h] * x[r];
        };
        const float *p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) p[h] = g.B[h] + (c0 + kg) * g.ldb[h] + xc;
        if (whole) {
#pragma unroll 8
            for (int i = kg; i < n; i += GROUPS) {
                f32x4 w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[h] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u *>(p[h]));
                    p[h] += GROUPS * g.ldb[h];
                }
                step(i, w);
            }
        } else if (some) {
            for (int i = kg; i < n; i += GROUPS) {
                f32x4 w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[h][j] = xc + j < N ? p[h][j] : 0.0f;
                    p[h] += GROUPS * g.ldb[h];
                }
                step(i, w);
            }
        }
        __syncthreads();
    }
    poison();
    // eight lane groups of a wave, then the waves
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < MR; ++r) {
#pragma unroll
            for (int off = XQ; off < 64; off <<= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[h][r][j] += __shfl_xor(acc[h][r][j], off);
            if (lane < XQ) *reinterpret_cast<f32x4 *>(&lds[((wave * 2 + h) * MR + r) * XB + 4 * xq]) = acc[h][r];
        }
    __syncthreads();
    if (tid >= MR * XB) return;
    const int r = tid / XB, x = tid % XB;
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s[h] = lds[(h * MR + r) * XB + x];
#pragma unroll
        for (int w = 1; w < W; ++w) s[h] += lds[((w * 2 + h) * MR + r) * XB + x];
    }
    const int64_t col = x0 + x;
    const int row = m0 + r;
    if (row >= g.M || col >= N) return;
    float v[1] = {s[0]}, u[1] = {s[1]};
    gate_apply<1>(g.e, row, (int)col, N, v, u);
    g.C[row * g.ldc + col] = v[0];
}

}  // namespace sgemm
