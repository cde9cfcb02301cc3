// The gated feed-forward block in float32 on the matrix cores: both
// projections of one tile of A, the activation and their product in one kernel,
//
//   C = act(A op(Bg) + bg) * (A op(Bu) + bu).
//
// It is the direct-load kernel of sgemm_mfma_dl.hpp (its LDS layout, fetch
// assignment, swizzle and cross-slice pipeline; the reasons are there) with two
// B operands: a stage holds a BM-row slice of A and slices of the same BN / 2
// columns of Bg and of Bu, each laid out as an operand of its own, and a wave
// holds the sums of both for the same outputs.  So A is read once for the two
// products, the sums never leave the registers before they are multiplied, and
// a tile does the work of a BM x BN one.  Nothing in it needs the two weights
// to be one tensor, or apart from each other.
//
// Bound by the matrix cores (BM x BN tiles of one large product, 2 M N K each): 2048
// x 8192 x 2048, 137 GFLOP, takes 931 us on 256x256 tiles (148 TFLOP/s, matrix cores
// busy 92% of the cycles), 944 on 128x128 and 1016 on 64x64; two plain products into
// memory and a second pass 961.  Those win where the outputs have few tiles and K is
// split: 515 x 2051 x 1023 takes 57 us so, and 60 to 61 on 64x64 tiles with 4-byte
// loads, which the plan takes there: its model has the two 5% apart the other way.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "gate.hpp"
#include "sgemm_mfma_dl.hpp"

namespace sgemm {

// B and ldb are the gate's, C the output; beta, alpha and the batch are not used.
struct GatedArgs : GemmArgs {
    const float *B_up;
    int ldb_up;
    Gate e;
};

template <int BM, int BN, int BK, int WAVES_M, int WAVES_N, int STAGES, bool TB, bool DW, int MB> struct GatedTraits {
    static constexpr int NW = WAVES_M * WAVES_N;
    static constexpr int NT = NW * 64;
    static constexpr int BH = BN / 2;         // outputs' columns of a tile
    static constexpr int WTM = BM / WAVES_M;
    static constexpr int WTH = BH / WAVES_N;  // and of a wave
    static constexpr int RM = WTM / MB;
    static constexpr int NB = WTH / MB;
    typedef DlOperand<BM, BK, WTM, NW, true, DW, MB> OpA;
    typedef DlOperand<BH, BK, WTH, NW, TB, DW, MB> OpB;
    static constexpr int A_FLOATS = BM * BK, B_FLOATS = BH * BK;
    static constexpr int STAGE_FLOATS = A_FLOATS + 2 * B_FLOATS;
    static constexpr int LDS_FLOATS = STAGES * STAGE_FLOATS;
    static_assert(NB == 1 || NB == 2, "a lane's adjacent columns");
    static_assert(STAGES >= 2, "at least two LDS stages");
    static_assert(LDS_FLOATS * 4 <= 160 * 1024, "LDS budget of one CU");
};

template <int BM, int BN, int BK, int WAVES_M, int WAVES_N, int STAGES, bool TB, bool DW, int MB>
__global__ void __launch_bounds__(WAVES_M * WAVES_N * 64) sgemm_gated_kernel(GatedArgs g)
{
    typedef GatedTraits<BM, BN, BK, WAVES_M, WAVES_N, STAGES, TB, DW, MB> T;
    typedef typename T::OpA OpA;
    typedef typename T::OpB OpB;
    constexpr int NW = T::NW, WTM = T::WTM, WTH = T::WTH, RM = T::RM, NB = T::NB, BH = T::BH;
    constexpr int A_LOADS = OpA::LOADS, B_LOADS = OpB::LOADS, LOADS = A_LOADS + 2 * B_LOADS;
    constexpr int STAGE_FLOATS = T::STAGE_FLOATS, A_FLOATS = T::A_FLOATS, B_FLOATS = T::B_FLOATS;
    constexpr int G = BK / (MB == 32 ? 8 : 16);  // k groups per slice
    constexpr int ACC = MB == 32 ? 16 : 4;       // accumulators per block per lane
    typedef typename std::conditional<MB == 32, f32x16, f32x4>::type acc_t;
    typedef __attribute__((address_space(3))) void lds_void;
    constexpr int EL = DW ? 1 : 4;  // floats per lane per load
    __shared__ __attribute__((aligned(1024))) float smem[T::LDS_FLOATS];
    // keeps the accumulators in AGPRs
    asm volatile("" ::: "a0");

    const Work w = map_work(g);
    const int M = g.M, N = g.N, K = g.K, lda = g.lda;
    const int m0 = w.tm * BM, n0 = w.tn * BH;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const float *const A = g.A + (int64_t)m0 * lda;
    const float *const B[2] = {TB ? g.B + (int64_t)n0 * g.ldb : g.B + n0,
                               TB ? g.B_up + (int64_t)n0 * g.ldb_up : g.B_up + n0};
    const int ldb[2] = {g.ldb, g.ldb_up};

    acc_t acc[2][RM][NB];  // of the gate, of the other projection
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int r = 0; r < ACC; ++r) acc[h][i][j][r] = 0.0f;

    // ---- fetch assignment -----------------------------------------------------------
    uint32_t a_off[A_LOADS], b_off[2][B_LOADS];
    int a_col[A_LOADS], b_col[B_LOADS];
#pragma unroll
    for (int j = 0; j < A_LOADS; ++j) OpA::assign(j, wave, lane, lda, a_off[j], a_col[j]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < B_LOADS; ++j) OpB::assign(j, wave, lane, ldb[h], b_off[h][j], b_col[j]);

    // LDS float of load j of an operand's region (of the wave, of the lane)
    auto place = [&](int j) { return (j * NW + wave) * 64 * EL; };
    auto region = [&](int s, int op) { return smem + s * STAGE_FLOATS + (op == 0 ? 0 : A_FLOATS + (op - 1) * B_FLOATS); };

    // LDS race check build: this thread's share of stage s set to NaN before its fill.
    auto poison_stage = [&](int s) {
        if constexpr (kLdsPoison) {
#pragma unroll
            for (int j = 0; j < A_LOADS; ++j) lds_poison(region(s, 0) + place(j) + lane * EL, EL);
#pragma unroll
            for (int h = 1; h < 3; ++h)
#pragma unroll
                for (int j = 0; j < B_LOADS; ++j) lds_poison(region(s, h) + place(j) + lane * EL, EL);
            lds_poison_done();
        }
    };

    // One operand's slice by direct loads; off[j] is kOobOffset where the data
    // is past the operand.
    auto load_direct = [&](__amdgpu_buffer_rsrc_t rsrc, float *base, int j, uint32_t off) {
        float *dst = base + place(j);
        if constexpr (DW) __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)dst, 4, (int)off, 0, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)dst, 16, (int)off, 0, 0, 0);
    };
    // One load through registers, masked to the floats below `lim`.
    auto load_masked = [&](__amdgpu_buffer_rsrc_t rsrc, float *base, int j, uint32_t off, int col, int lim) {
        float v[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = keep_below(buffer_load_f32(rsrc, off + 4u * e), e, lim - col);
        float *const dst = base + place(j) + lane * EL;
        if constexpr (EL == 4) *reinterpret_cast<f32x4 *>(dst) = f32x4{v[0], v[1], v[2], v[3]};
        else *dst = v[0];
        __builtin_amdgcn_sched_barrier(0);
    };

    // Fetch slice kt into stage s (sgemm_mfma_dl.hpp's fetch, for three operands).
    auto fetch = [&](int kt, int s) {
        poison_stage(s);
        const int k0 = kt * BK;
        const int a_lim = K - k0, b_lim = TB ? K - k0 : N - n0;
        const bool partial = !DW && (((a_lim & 3) && a_lim < BK) || ((b_lim & 3) && b_lim < (TB ? BK : BH)));
        const int64_t cap = g.direct ? (int64_t)kOobOffset : (int64_t)0xffffffff;
        const int64_t abytes = 4 * ((int64_t)(M - 1 - m0) * lda + (K - k0));
        const auto ar = make_rsrc(A + k0, abytes < cap ? abytes : cap);
        const bool direct = g.direct && !partial;
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j) {
            if (direct) load_direct(ar, region(s, 0), j, a_col[j] < a_lim ? a_off[j] : kOobOffset);
            else load_masked(ar, region(s, 0), j, a_off[j], a_col[j], a_lim);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float *const base = TB ? B[h] + k0 : B[h] + (int64_t)k0 * ldb[h];
            const int64_t bytes = TB ? 4 * ((int64_t)(N - 1 - n0) * ldb[h] + (K - k0))
                                     : 4 * ((int64_t)(K - 1 - k0) * ldb[h] + (N - n0));
            const auto br = make_rsrc(base, bytes < cap ? bytes : cap);
#pragma unroll
            for (int j = 0; j < B_LOADS; ++j) {
                if (direct) load_direct(br, region(s, 1 + h), j, b_col[j] < b_lim ? b_off[h][j] : kOobOffset);
                else load_masked(br, region(s, 1 + h), j, b_off[h][j], b_col[j], b_lim);
            }
        }
    };

    // Fetch of a slice wholly inside K with the tile's fixed offsets: no checks.
    uint32_t af[A_LOADS], bf[2][B_LOADS];
    auto fetch_full = [&](int kt, int s) {
        poison_stage(s);
        const int k0 = kt * BK;
        const auto ar = make_rsrc(A + k0, (int64_t)kOobOffset);
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j) load_direct(ar, region(s, 0), j, af[j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto br = make_rsrc(TB ? B[h] + k0 : B[h] + (int64_t)k0 * ldb[h], (int64_t)kOobOffset);
#pragma unroll
            for (int j = 0; j < B_LOADS; ++j) load_direct(br, region(s, 1 + h), j, bf[h][j]);
        }
    };

    // ---- fragments --------------------------------------------------------------------
    constexpr int KQ = MB == 32 ? 2 : 4;  // 16-byte chunks per k group
    const int lr = lane & (MB - 1), hl = MB == 32 ? lane >> 5 : lane >> 4;
    const int sw = hl ^ chunk_swizzle<BK, MB>(lr);
    typedef typename DlXVec<!TB, NB>::T xb_t;
    struct Frag {
        f32x4 a[RM];        // [block][t]
        f32x4 kb[2][NB];    // k-contiguous B: [which][block][t]
        xb_t xb[2][4];      // index-contiguous B: [which][t][block]
    };
    const int a_base = (wm * WTM + lr) * BK;
    const int b_base = TB ? (wn * WTH + lr) * BK : (4 * hl) * BH + wn * WTH + NB * lr;
    auto read_frag = [&](int s, int gi, Frag &f) {
        const float *const as = region(s, 0) + a_base + 4 * ((KQ * gi) ^ sw);
#pragma unroll
        for (int i = 0; i < RM; ++i) f.a[i] = *reinterpret_cast<const f32x4 *>(as + i * MB * BK);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float *const bs = region(s, 1 + h) + b_base;
            if constexpr (TB) {
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    f.kb[h][j] = *reinterpret_cast<const f32x4 *>(bs + j * MB * BK + 4 * ((KQ * gi) ^ sw));
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) f.xb[h][t] = *reinterpret_cast<const xb_t *>(bs + (4 * KQ * gi + t) * BH);
            }
        }
    };
    auto mfma_frag = [&](const Frag &f) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const float a = f.a[i][t];
                        float b;
                        if constexpr (TB) b = f.kb[h][j][t];
                        else b = dl_elem<NB>(f.xb[h][t], j);
                        if constexpr (MB == 32)
                            acc[h][i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc[h][i][j], 0, 0, 0);
                        else
                            acc[h][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, acc[h][i][j], 0, 0, 0);
                    }
    };

    // ---- main loop: sgemm_mfma_dl.hpp's cross-slice pipeline ----------------------------
    constexpr int VM = (STAGES - 2) * LOADS;
    static_assert(VM < 64, "vmcnt field holds 6 bits");
    static_assert(G % 2 == 0, "fragment buffers alternate per k group");
    constexpr int WAIT_LATER = (VM & 15) | (7 << 4) | ((VM >> 4) << 14);  // later slices in flight, lgkmcnt(0)
    constexpr int WAIT_ALL = 7 << 4;                                      // vmcnt(0) lgkmcnt(0)
    const int nk = (K + BK - 1) / BK;
    auto barrier = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    Frag f[2];
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < nk) fetch(s, s);
    if (STAGES - 2 < nk) __builtin_amdgcn_s_waitcnt(WAIT_LATER);
    else __builtin_amdgcn_s_waitcnt(WAIT_ALL);
    barrier();
    read_frag(0, 0, f[0]);
    auto slice = [&](int kt, auto full) {
        constexpr bool FULL = decltype(full)::value;
        const int s = kt % STAGES, s1 = (kt + 1) % STAGES;
        const bool next = FULL || kt + 1 < nk;
        const bool more = FULL || kt + STAGES - 1 < nk;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            __builtin_amdgcn_sched_barrier(0);
            if (gi + 1 < G) {
                read_frag(s, gi + 1, f[(gi + 1) & 1]);
                if (gi == 0) {
                    if constexpr (FULL) fetch_full(kt + STAGES - 1, (kt + STAGES - 1) % STAGES);
                    else if (more) fetch(kt + STAGES - 1, (kt + STAGES - 1) % STAGES);
                }
                mfma_frag(f[gi & 1]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // DS read
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
                }
                if (gi == 0) {
#pragma unroll
                    for (int i = 0; i < LOADS; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
                    }
                }
            } else {
                if (more) __builtin_amdgcn_s_waitcnt(WAIT_LATER);
                else __builtin_amdgcn_s_waitcnt(WAIT_ALL);
                barrier();
                __builtin_amdgcn_sched_barrier(0);
                if (next) read_frag(s1, 0, f[G & 1]);
                mfma_frag(f[gi & 1]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int kt = 0;
    const int n_lim = N - n0;
    const bool edge_chunks = !DW && !TB && (n_lim & 3) && n_lim < BH;
    if (g.direct && !edge_chunks) {
#pragma unroll
        for (int j = 0; j < A_LOADS; ++j) af[j] = OpA::full_slice_off(j, wave, lane, lda, M - m0);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < B_LOADS; ++j) bf[h][j] = OpB::full_slice_off(j, wave, lane, ldb[h], n_lim);
        const int kend = K / BK - (STAGES - 1);
        // (scalar reads for the epilogue waited for before the loop, as there)
        __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));  // lgkmcnt(0)
        for (; kt < kend; ++kt) slice(kt, DlTag<true>());
    }
    for (; kt < nk; ++kt) slice(kt, DlTag<false>());

    // ---- epilogue: both sums of CROWS rows at a time through the wave's share of LDS ------
    constexpr int SHARE = T::LDS_FLOATS / NW;
    constexpr int CR = 2 * MB * WTH <= SHARE ? ACC : ACC / 2;
    constexpr int CROWS = MB / (ACC / CR);
    static_assert(2 * CROWS * WTH <= SHARE && SHARE % 4 == 0, "a wave's share holds one chunk");
    static_assert(MB == 32 || CR == ACC, "16x16 blocks are staged whole");
    typedef float vec_t __attribute__((ext_vector_type(NB)));
    if constexpr (2 * RM * NB * ACC == 128) {
        // (kept where the MFMAs hold them, as in the plain kernel)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) asm volatile("" : "+a"(acc[h][i][j]));
    }
    __syncthreads();
    float *const mine = smem + wave * SHARE;
    const StagedGate<CROWS, WTH, RM, false> epi(g.e, g.C, g.ldc, M, N, lane, n0 + wn * WTH);
#pragma unroll
    for (int i = 0; i < RM; ++i) {
#pragma unroll
        for (int r0 = 0; r0 < ACC; r0 += CR) {
            if constexpr (kLdsPoison) {
                lds_poison(mine + lane * (SHARE / 64), SHARE / 64);
                lds_poison_done();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = r0; r < r0 + CR; ++r) {
                    const int rr = MB == 32 ? 8 * ((r - r0) >> 2) + 4 * hl + (r & 3) : 4 * hl + r;
                    float *const p = mine + (h * CROWS + rr) * WTH + NB * lr;
                    if constexpr (NB == 1) {
                        *p = acc[h][i][0][r];
                    } else {
                        vec_t v;
#pragma unroll
                        for (int j = 0; j < NB; ++j) v[j] = acc[h][i][j][r];
                        *reinterpret_cast<vec_t *>(p) = v;
                    }
                }
            asm volatile("" ::: "memory");
            epi.store(mine, m0 + wm * WTM + RM * (MB / ACC) * r0 + i, 1.0f);
            asm volatile("" ::: "memory");
        }
    }
}

}  // namespace sgemm
