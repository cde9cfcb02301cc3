// Products of two 8-bit (OCP e4m3) matrices with float32 sums, both stored
// k-contiguous (A: M x K, B: N x K).
//
//   C[m][n] = epilogue(scale_a[m] * scale_b[n] * sum_k A[m][k] B[n][k])
//
// The scales are one factor per row and per column of C, so they leave the
// sum and meet in the epilogue (epilogue.hpp).
//
// Codes travel as bytes (memory, L2, LDS) and become bfloat16 in registers,
// where every e4m3 value is exact, for the 16-bit matrix instructions
// (v_mfma_f32_32x32x16_bf16, v_mfma_f32_16x16x32_bf16).  The 8-bit matrix
// instructions have twice the rate (4.4 against 2.3 PFLOP/s measured on
// registers), but they do not keep float32 sums: the products of one
// instruction are aligned and cut before they are added.  Measured against 64
// bits on normal values, their results are off by 1.3e-5 of their norm at any K
// (128, 1024, 8192; the 32-deep and the 128-deep form alike), those of the
// 16-bit instructions by 9e-9, 4e-8 and 1.2e-7, which is float32's own rounding.
// Large products are bound by the card's power: 8192^3 takes 0.66 ms on codes
// of zero and 0.81 ms on random ones, where float16 takes 1% longer than
// bfloat16.
//
// gemm_e4m3_kernel: LDS tiles.  A slice of a tile is the same bytes as a slice
// of the float32 kernel's NT form (four codes in the place of a float), so the
// fetch assignment, the LDS layout and its conflict-free swizzle are
// DlOperand's (sgemm_mfma_dl.hpp) on "floats" of four codes: BKF of them per
// row and slice.  A lane reads 16-byte chunks; one MFMA takes half of one per
// operand.  Which k a chunk's bytes are does not matter as long as both
// operands agree, as every k is summed.
//
// gemm_e4m3_skinny_kernel: few rows of A (single tokens).  The weights stream
// once from memory straight into registers; see there.
#pragma once

#include "common.hpp"
#include "epilogue.hpp"
#include "sgemm_mfma_dl.hpp"

namespace sgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4u __attribute__((ext_vector_type(4), aligned(1)));

// A, B point at bytes and lda, ldb count them; C, ldc and the rest as in
// GemmArgs.  With a K split, C is the workspace and the epilogue is left to
// the reduction.
struct E4m3Args : EpiGemmArgs {
    int64_t ld_a, ld_b;
};

// 16 codes of one row from column col on; those at or past `lim` read as zero.
__device__ __forceinline__ i32x4 load_chunk(const unsigned char *row, int col, int lim)
{
    if (col + 16 <= lim) return *reinterpret_cast<const i32x4u *>(row + col);
    i32x4 v = {0, 0, 0, 0};
    if (col < lim) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int b = row[min(col + i, lim - 1)];
            v[i / 4] |= col + i < lim ? b << (8 * (i % 4)) : 0;
        }
    }
    return v;
}

template <int MB> struct E4m3Acc { typedef f32x16 T; };
template <> struct E4m3Acc<16> { typedef f32x4 T; };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes (dwords 2 half, 2 half + 1 of a chunk) as bfloat16, exactly.
__device__ __forceinline__ bf16x8 codes_bf16(const i32x4 &c, int half)
{
    const int lo = c[2 * half], hi = c[2 * half + 1];
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// 16 (MB = 32) or 32 (MB = 16) values of MB rows of A and B, eight per lane.
template <int MB>
__device__ __forceinline__ typename E4m3Acc<MB>::T mfma_bf16(bf16x8 a, bf16x8 b, typename E4m3Acc<MB>::T c)
{
    if constexpr (MB == 32) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

template <int BM, int BN, int BKF, int WAVES_M, int WAVES_N, int STAGES, int MB> struct E4m3Traits {
    static constexpr int NW = WAVES_M * WAVES_N;
    static constexpr int NT = NW * 64;
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
    static constexpr int RM = WTM / MB, NB = WTN / MB;
    typedef DlOperand<BM, BKF, WTM, NW, true, false, MB> OpA;
    typedef DlOperand<BN, BKF, WTN, NW, true, false, MB> OpB;
    static constexpr int A_FLOATS = BM * BKF;
    static constexpr int STAGE_FLOATS = (BM + BN) * BKF;
    static constexpr int LDS_FLOATS = STAGES * STAGE_FLOATS;
    static constexpr int G = BKF / (MB == 32 ? 8 : 16);  // k groups (one chunk per lane) per slice
    static_assert(G % 2 == 0, "fragment buffers alternate per k group");
    static_assert(NB == 1 || NB == 2 || NB == 4, "a lane's adjacent columns");
    static_assert(LDS_FLOATS * 4 <= 160 * 1024, "LDS budget of one CU");
};

// REG: the operands' rows do not start 16-byte aligned (or are too far apart
// for 32-bit offsets): slices go through registers, loaded at any address,
// and are written to LDS one MFMA step later.
template <int BM, int BN, int BKF, int WAVES_M, int WAVES_N, int STAGES, int MB, bool REG>
__global__ void __launch_bounds__(WAVES_M * WAVES_N * 64) gemm_e4m3_kernel(E4m3Args g)
{
    typedef E4m3Traits<BM, BN, BKF, WAVES_M, WAVES_N, STAGES, MB> T;
    typedef typename T::OpA OpA;
    typedef typename T::OpB OpB;
    typedef typename E4m3Acc<MB>::T acc_t;
    constexpr int NW = T::NW, WTM = T::WTM, WTN = T::WTN, RM = T::RM, NB = T::NB;
    constexpr int ACC = MB == 32 ? 16 : 4;
    constexpr int A_LOADS = OpA::LOADS, B_LOADS = OpB::LOADS;
    constexpr int STAGE_FLOATS = T::STAGE_FLOATS, A_FLOATS = T::A_FLOATS;
    constexpr int G = T::G;
    constexpr int BK = 4 * BKF;  // codes per row and slice
    typedef __attribute__((address_space(3))) void lds_void;
    __shared__ __attribute__((aligned(1024))) float smem[T::LDS_FLOATS];
    // keeps the accumulators in AGPRs
    asm volatile("" ::: "a0");

    const Work w = map_work(g);
    const int kb = w.split * g.k_chunk;
    const unsigned char *A = reinterpret_cast<const unsigned char *>(g.A) + kb;
    const unsigned char *B = reinterpret_cast<const unsigned char *>(g.B) + kb;
    g.C += w.split * g.split_c;
    const int M = g.M, N = g.N, K = min(g.K - kb, g.k_chunk);
    const int m0 = w.tm * BM, n0 = w.tn * BN;
    A += (int64_t)m0 * g.ld_a;
    B += (int64_t)n0 * g.ld_b;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;

    acc_t acc[RM][NB];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < ACC; ++r) acc[i][j][r] = 0.0f;

    // ---- fetch: load j of this thread brings 16 codes of row a_row[j] (of the
    // tile, clamped to the last row: what rows past M or N compute is never
    // stored) from column a_col[j] of the slice
    int a_row[A_LOADS], a_col[A_LOADS], b_row[B_LOADS], b_col[B_LOADS];
#pragma unroll
    for (int j = 0; j < A_LOADS; ++j) {
        OpA::place(j, wave, lane, a_row[j], a_col[j]);
        a_row[j] = min(a_row[j], M - 1 - m0);
        a_col[j] *= 4;
    }
#pragma unroll
    for (int j = 0; j < B_LOADS; ++j) {
        OpB::place(j, wave, lane, b_row[j], b_col[j]);
        b_row[j] = min(b_row[j], N - 1 - n0);
        b_col[j] *= 4;
    }
    uint32_t a_off[A_LOADS], b_off[B_LOADS];  // direct loads: 32-bit offsets
    if constexpr (!REG) {
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j) a_off[j] = (uint32_t)a_row[j] * (uint32_t)g.ld_a + (uint32_t)a_col[j];
#pragma unroll
        for (int j = 0; j < B_LOADS; ++j) b_off[j] = (uint32_t)b_row[j] * (uint32_t)g.ld_b + (uint32_t)b_col[j];
    }

    auto poison_stage = [&](int s) {
        if constexpr (kLdsPoison) {
#pragma unroll
            for (int j = 0; j < A_LOADS; ++j)
                lds_poison(smem + s * STAGE_FLOATS + ((j * NW + wave) * 64 + lane) * 4, 4);
#pragma unroll
            for (int j = 0; j < B_LOADS; ++j)
                lds_poison(smem + s * STAGE_FLOATS + A_FLOATS + ((j * NW + wave) * 64 + lane) * 4, 4);
            lds_poison_done();
        }
    };
    // registers of one slice (REG), and their way to LDS
    i32x4 ra[REG ? A_LOADS : 1], rb[REG ? B_LOADS : 1];
    auto load_regs = [&](int kt, auto full) {
        constexpr bool FULL = decltype(full)::value;
        const int k0 = kt * BK;
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j) {
            const unsigned char *row = A + a_row[j] * g.ld_a;
            if constexpr (FULL) ra[j] = *reinterpret_cast<const i32x4u *>(row + k0 + a_col[j]);
            else ra[j] = load_chunk(row, k0 + a_col[j], K);
        }
#pragma unroll
        for (int j = 0; j < B_LOADS; ++j) {
            const unsigned char *row = B + b_row[j] * g.ld_b;
            if constexpr (FULL) rb[j] = *reinterpret_cast<const i32x4u *>(row + k0 + b_col[j]);
            else rb[j] = load_chunk(row, k0 + b_col[j], K);
        }
    };
    auto write_regs = [&](int s) {
        poison_stage(s);
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j)
            *reinterpret_cast<i32x4 *>(smem + s * STAGE_FLOATS + ((j * NW + wave) * 64 + lane) * 4) = ra[j];
#pragma unroll
        for (int j = 0; j < B_LOADS; ++j)
            *reinterpret_cast<i32x4 *>(smem + s * STAGE_FLOATS + A_FLOATS + ((j * NW + wave) * 64 + lane) * 4) =
                rb[j];
    };
    // Slice kt straight to stage s.  Only the last slice can reach past K: its
    // chunks wholly past K read as zero (an offset past the resource), and if
    // one is cut (K not a multiple of 16) the slice goes through registers.
    auto fetch = [&](int kt, int s, auto full) {
        constexpr bool FULL = decltype(full)::value;
        poison_stage(s);
        const int k0 = kt * BK;
        const int lim = K - k0;
        if (!FULL && (lim & 15) && lim < BK) {
#pragma unroll
            for (int j = 0; j < A_LOADS; ++j) {
                const i32x4 v = load_chunk(A + a_row[j] * g.ld_a, k0 + a_col[j], K);
                *reinterpret_cast<i32x4 *>(smem + s * STAGE_FLOATS + ((j * NW + wave) * 64 + lane) * 4) = v;
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < B_LOADS; ++j) {
                const i32x4 v = load_chunk(B + b_row[j] * g.ld_b, k0 + b_col[j], K);
                *reinterpret_cast<i32x4 *>(smem + s * STAGE_FLOATS + A_FLOATS +
                                           ((j * NW + wave) * 64 + lane) * 4) = v;
                __builtin_amdgcn_sched_barrier(0);
            }
            return;
        }
        const auto ar = make_rsrc(reinterpret_cast<const float *>(A + k0), (int64_t)kOobOffset);
        const auto br = make_rsrc(reinterpret_cast<const float *>(B + k0), (int64_t)kOobOffset);
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j) {
            const int off = (int)(FULL || a_col[j] < lim ? a_off[j] : kOobOffset);
            float *dst = smem + s * STAGE_FLOATS + (j * NW + wave) * 64 * 4;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_void *)dst, 16, off, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < B_LOADS; ++j) {
            const int off = (int)(FULL || b_col[j] < lim ? b_off[j] : kOobOffset);
            float *dst = smem + s * STAGE_FLOATS + A_FLOATS + (j * NW + wave) * 64 * 4;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(br, (lds_void *)dst, 16, off, 0, 0, 0);
        }
    };

    // ---- fragments: block b's row for a lane is LDS row wave_offset + MB*b +
    // (lane mod MB); its 16-byte chunk number c is stored at c ^ f(row).  K
    // group gi is chunk KQ*gi + h, h the lane's half (MB = 32, KQ = 2) or
    // quarter (MB = 16, KQ = 4): two MFMAs per pair of blocks.
    constexpr int KQ = MB == 32 ? 2 : 4;
    const int lr = lane & (MB - 1), h = MB == 32 ? lane >> 5 : lane >> 4;
    const int u = h ^ chunk_swizzle<BKF, MB>(lr);
    struct Frag {
        i32x4 a[RM], b[NB];
    };
    struct Half {  // one half of a group's codes, as bfloat16
        bf16x8 a[RM], b[NB];
    };
    const int a_base = (wm * WTM + lr) * BKF, b_base = A_FLOATS + (wn * WTN + lr) * BKF;
    auto read_frag = [&](int s, int gi, Frag &f) {
        const float *base = smem + s * STAGE_FLOATS + 4 * ((KQ * gi) ^ u);
#pragma unroll
        for (int i = 0; i < RM; ++i) f.a[i] = *reinterpret_cast<const i32x4 *>(base + a_base + i * MB * BKF);
#pragma unroll
        for (int j = 0; j < NB; ++j) f.b[j] = *reinterpret_cast<const i32x4 *>(base + b_base + j * MB * BKF);
    };
    auto convert = [&](const Frag &f, int half, Half &o) {
#pragma unroll
        for (int i = 0; i < RM; ++i) o.a[i] = codes_bf16(f.a[i], half);
#pragma unroll
        for (int j = 0; j < NB; ++j) o.b[j] = codes_bf16(f.b[j], half);
    };
    auto mma = [&](const Half &f) {
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = mfma_bf16<MB>(f.a[i], f.b[j], acc[i][j]);
    };

    // ---- main loop ---------------------------------------------------------------
    // Slice kt's first k group is in registers when it begins.  Before its last
    // group every thread waits for its own part of slice kt+1 (and its own
    // reads of slice kt), and one barrier follows: every wave's part of slice
    // kt+1 is in LDS, and slice kt's stage is free, as its last group is in
    // registers.  Among the last group's MFMAs the next slice's first group is
    // read and the fetch of slice kt+STAGES into that free stage is issued, so
    // a fetch has STAGES - 1 slices' time to arrive.  Each half's codes are
    // converted among the MFMAs of the half before.  REG: slice kt+1 is written
    // to LDS before the barrier from registers whose loads were issued a slice
    // earlier.
    constexpr int LOADS = A_LOADS + B_LOADS;
    constexpr int VM = (STAGES - 2) * LOADS, VM0 = (STAGES - 1) * LOADS;
    static_assert(VM0 < 64, "vmcnt field holds 6 bits");
    static_assert(!REG || STAGES == 2, "registers hold one slice ahead of the two in LDS");
    constexpr int WAIT_ALL = 7 << 4;  // vmcnt(0) lgkmcnt(0)
    constexpr int WAIT_LATER = (VM & 15) | (7 << 4) | ((VM >> 4) << 14);     // slices kt+2.. in flight
    constexpr int WAIT_FIRST = (VM0 & 15) | (7 << 4) | ((VM0 >> 4) << 14);  // slices 1.. in flight
    const int nk = (K + BK - 1) / BK;
    const int nfull = K / BK;  // slices wholly inside K
    auto barrier = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    typedef DlTag<true> Y;
    typedef DlTag<false> X;
    Frag f[2];
    Half hv[2];
    if constexpr (REG) {
        load_regs(0, X());
        write_regs(0);
        if (nk > 1) load_regs(1, X());
        __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));  // lgkmcnt(0)
    } else {
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (s < nk) fetch(s, s, X());
        if (STAGES - 1 < nk) __builtin_amdgcn_s_waitcnt(WAIT_FIRST);
        else __builtin_amdgcn_s_waitcnt(WAIT_ALL);
    }
    barrier();
    read_frag(0, 0, f[0]);
    convert(f[0], 0, hv[0]);
    // One slice, in stage s.  FULL: a fetch is issued, of a slice wholly inside K.
    auto slice = [&](int kt, int s, auto full) {
        constexpr bool FULL = decltype(full)::value;
        const int s1 = s + 1 == STAGES ? 0 : s + 1;  // stage of slice kt+1
        const bool next = FULL || kt + 1 < nk;
        const bool more = FULL || kt + STAGES < nk;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            __builtin_amdgcn_sched_barrier(0);
            Frag &cur = f[gi & 1], &nxt = f[(gi + 1) & 1];
            if (gi + 1 < G) {
                read_frag(s, gi + 1, nxt);
            } else {
                if constexpr (REG) {
                    if (next) write_regs(s1);
                    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));  // lgkmcnt(0)
                } else {
                    if (FULL || kt + STAGES - 1 < nk) __builtin_amdgcn_s_waitcnt(WAIT_LATER);
                    else __builtin_amdgcn_s_waitcnt(WAIT_ALL);
                }
                barrier();
                __builtin_amdgcn_sched_barrier(0);
                if (next) read_frag(s1, 0, nxt);
                if (more) {
                    if constexpr (REG) load_regs(kt + 2, full);
                    else fetch(kt + STAGES, s, full);
                }
            }
            convert(cur, 1, hv[1]);
            mma(hv[0]);
            // the group's reads, loads and conversions among its MFMAs
            constexpr int CV = (4 * (RM + NB) + RM * NB - 1) / (RM * NB);
#pragma unroll
            for (int i = 0; i < RM * NB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // DS read
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // VMEM read
                __builtin_amdgcn_sched_group_barrier(0x002, CV, 0);  // VALU
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
            }
            __builtin_amdgcn_sched_barrier(0);
            if (gi + 1 < G || next) convert(nxt, 0, hv[0]);
            mma(hv[1]);
#pragma unroll
            for (int i = 0; i < RM * NB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
                __builtin_amdgcn_sched_group_barrier(0x002, CV, 0);  // VALU
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int kt = 0, s = 0;
    while (kt + STAGES < nfull) {
        slice(kt, s, Y());
        ++kt;
        s = s + 1 == STAGES ? 0 : s + 1;
    }
    while (kt < nk) {
        slice(kt, s, X());
        ++kt;
        s = s + 1 == STAGES ? 0 : s + 1;
    }

    // ---- epilogue, staged through LDS as in the float32 kernel ------------------------
    constexpr int SHARE = T::LDS_FLOATS / NW;
    static_assert(MB * WTN <= SHARE && SHARE % 256 == 0, "a wave's share holds a block row");
    typedef float vec_t __attribute__((ext_vector_type(NB)));
    __syncthreads();
    float *const mine = smem + wave * SHARE;
    const StagedEpi<MB, WTN, RM, true> epi(g, 0, lane, n0 + wn * WTN);
    float scale[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) scale[i] = epi.row_scale(m0 + wm * WTM + i);
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        if constexpr (kLdsPoison) {
            lds_poison(mine + lane * (SHARE / 64), SHARE / 64);
            lds_poison_done();
        }
#pragma unroll
        for (int r = 0; r < ACC; ++r) {
            float *p = mine + (MB == 32 ? 8 * (r >> 2) + 4 * h + (r & 3) : 4 * h + r) * WTN + NB * lr;
            if constexpr (NB == 1) {
                *p = acc[i][0][r];
            } else {
                vec_t v;
#pragma unroll
                for (int j = 0; j < NB; ++j) v[j] = acc[i][j][r];
                *reinterpret_cast<vec_t *>(p) = v;
            }
        }
        asm volatile("" ::: "memory");
        epi.store(mine, m0 + wm * WTM + i, scale[i]);
        asm volatile("" ::: "memory");
    }
}

// ---- few rows -------------------------------------------------------------------------
// Up to 16 RM rows of A: a workgroup computes them for 16 columns (rows of B),
// on 16x16x32 MFMAs, with K dealt to its W waves in turns of 128 codes, so that
// one round of the waves reads W consecutive 128-byte lines of each of the 16
// weight rows.  Nothing is shared through LDS but the waves' partial results:
// every weight is used by one workgroup alone and goes from memory to the
// registers that feed the MFMA, DEPTH steps ahead; A's few rows are read from
// L2 by every workgroup.  One token of an 8192 x 8192 layer takes 13.7 us (4.9
// TB/s of weights, the launch included), against 12.7 us at the rate of a large
// copy; 2 steps ahead take 13.8, 4 take 14.5, 4 waves 14.9 and 8 waves 14.4 us,
// and two column blocks per wave (half of A's reads, half the workgroups) 20.
// Rows of A past M and of B past N are read as the last
// one and never stored; codes past K read as zero.
template <int W, int RM> struct SkinnyTraits {
    static constexpr int NT = W * 64;
    static constexpr int DEPTH = 3;
    static constexpr int LDS_FLOATS = W * RM * 256;
};

template <int W, int RM> __global__ void __launch_bounds__(W * 64) gemm_e4m3_skinny_kernel(E4m3Args g)
{
    typedef SkinnyTraits<W, RM> T;
    constexpr int D = T::DEPTH;
    __shared__ __attribute__((aligned(16))) float red[T::LDS_FLOATS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, h = lane >> 4;
    const int M = g.M, N = g.N, K = g.K;
    if constexpr (kLdsPoison) {
        for (int i = tid; i < T::LDS_FLOATS; i += T::NT) lds_poison(&red[i], 1);
        lds_poison_done();
        __syncthreads();
    }
    // (64 bits: the last workgroup's next column can pass 2^31)
    for (int64_t c0 = 16 * (int64_t)blockIdx.x; c0 < N; c0 += 16 * (int64_t)gridDim.x) {
        const int n0 = (int)c0;
        const unsigned char *b = reinterpret_cast<const unsigned char *>(g.B) + min(n0 + lr, N - 1) * g.ld_b;
        const unsigned char *a[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i)
            a[i] = reinterpret_cast<const unsigned char *>(g.A) + min(16 * i + lr, M - 1) * g.ld_a;
        f32x4 acc[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        struct Frag {
            i32x4 b[2], a[RM][2];
        };
        // step q of this wave, wholly inside K
        auto load = [&](int q, Frag &f) {
            const int k = 128 * (wave + W * q) + 16 * h;
#pragma unroll
            for (int c = 0; c < 2; ++c) f.b[c] = *reinterpret_cast<const i32x4u *>(b + k + 64 * c);
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) f.a[i][c] = *reinterpret_cast<const i32x4u *>(a[i] + k + 64 * c);
        };
        auto mma = [&](const Frag &f) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const bf16x8 y = codes_bf16(f.b[c], half);
#pragma unroll
                    for (int i = 0; i < RM; ++i) acc[i] = mfma_bf16<16>(codes_bf16(f.a[i][c], half), y, acc[i]);
                }
        };
        const int nfull = K / 128;                                      // whole steps of all waves
        const int mine = nfull > wave ? (nfull - 1 - wave) / W + 1 : 0;  // of this one
        if (mine > 0) {
            // steps past the last reload it (in bounds, never multiplied in)
            const int last = mine - 1;
            Frag f[D];
#pragma unroll
            for (int d = 0; d < D; ++d) load(min(d, last), f[d]);
            int q0 = 0;
            for (; q0 + D <= mine; q0 += D) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    mma(f[d]);
                    load(min(q0 + D + d, last), f[d]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int d = 0; d < D - 1; ++d)
                if (q0 + d < mine) mma(f[d]);
        }
        if (K % 128 != 0 && wave == nfull % W) {
            // the cut step
            const int k = 128 * nfull + 16 * h;
            Frag f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f.b[c] = load_chunk(b, k + 64 * c, K);
#pragma unroll
                for (int i = 0; i < RM; ++i) f.a[i][c] = load_chunk(a[i], k + 64 * c, K);
            }
            mma(f);
        }
        // the waves' partial results, added in wave order
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[((wave * RM + i) * 4 + r) * 64 + lane] = acc[i][r];
        __syncthreads();
        for (int o = tid; o < RM * 256; o += T::NT) {
            float v[1] = {red[o]};
#pragma unroll
            for (int x = 1; x < W; ++x) v[0] += red[x * RM * 256 + o];
            // accumulator r of lane l is D[4 (l / 16) + r][l mod 16]
            const int i = o >> 8, r = (o >> 6) & 3, l = o & 63;
            const int row = 16 * i + 4 * (l >> 4) + r, col = n0 + (l & 15);
            if (row < M && col < N) {
                epi_apply<1>(g.e, 0, row, col, N, v);
                g.C[(int64_t)row * g.ldc + col] = v[0];
            }
        }
        __syncthreads();
    }
}

}  // namespace sgemm
