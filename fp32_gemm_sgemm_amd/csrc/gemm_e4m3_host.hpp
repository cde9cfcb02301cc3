// Host side of the 8-bit product (gemm_e4m3.hpp): argument checks and the
// launches of the kernel that e4m3_plan.hpp chooses.  Included by sgemm.hip
// inside its anonymous namespace, after the helpers of the float32 product.

template <int BM, int BN, int BKF, int WM, int WN, int ST, int MB> const void *e4m3_fn()
{
    return reinterpret_cast<const void *>(&sgemm::gemm_e4m3_kernel<BM, BN, BKF, WM, WN, ST, MB, false>);
}
template <int BM, int BN, int BKF, int WM, int WN, int MB> const void *e4m3_reg_fn()
{
    return reinterpret_cast<const void *>(&sgemm::gemm_e4m3_kernel<BM, BN, BKF, WM, WN, 2, MB, true>);
}

// The kernels of kE4m3Tiles and kE4m3Skinny, in their order.
struct E4m3TileKernel {
    int threads;
    const void *direct;  // rows 16-byte aligned
    const void *reg;     // any rows (null: not compiled)
};
const E4m3TileKernel kE4m3TileKernels[sgemm::kE4m3TileCount] = {
    {512, e4m3_fn<256, 256, 16, 4, 2, 4, 32>(), nullptr},
    {256, e4m3_fn<128, 128, 32, 2, 2, 2, 32>(), e4m3_reg_fn<128, 128, 32, 2, 2, 32>()},
    {256, e4m3_fn<64, 128, 32, 2, 2, 2, 32>(), e4m3_reg_fn<64, 128, 32, 2, 2, 32>()},
    {256, e4m3_fn<64, 64, 32, 2, 2, 2, 16>(), e4m3_reg_fn<64, 64, 32, 2, 2, 16>()},
};
struct E4m3SkinnyKernel {
    int threads;
    const void *fn;
};
const E4m3SkinnyKernel kE4m3SkinnyKernels[sgemm::kE4m3SkinnyCount] = {
    {128, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<2, 1>)},
    {256, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<4, 2>)},
    {256, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<4, 4>)},
};

// Direct loads keep a tile's byte offsets (256 rows and a slice) below 2^31.
constexpr int kE4m3MaxLdDirect = 1 << 23;

bool e4m3_aligned(const void *A, int lda, const void *B, int ldb)
{
    return !misaligned(A, 16) && !misaligned(B, 16) && lda % 16 == 0 && ldb % 16 == 0 &&
           lda <= kE4m3MaxLdDirect && ldb <= kE4m3MaxLdDirect;
}

bool e4m3_sizes_ok(int M, int N, int K)
{
    return M >= 0 && N >= 0 && K >= 0 && M <= sgemm::kMaxDim && N <= sgemm::kMaxDim && K <= sgemm::kMaxDim;
}

hipError_t run_e4m3(int M, int N, int K, const void *A, int lda, const float *scale_a, const void *B, int ldb,
                    const float *scale_b, float *C, int ldc, const sgemm_epilogue *epi, void *ws, size_t ws_bytes,
                    hipStream_t stream)
{
    const int kmin = K > 1 ? K : 1, nmin = N > 1 ? N : 1;
    if (!e4m3_sizes_ok(M, N, K) || lda < kmin || ldb < kmin || ldc < nmin || lda > sgemm::kMaxDim ||
        ldb > sgemm::kMaxDim || ldc > sgemm::kMaxDim)
        return hipErrorInvalidValue;
    if (!ws) ws_bytes = 0;
    const bool empty = M == 0 || N == 0;
    Call c = make_call(0, 1, M, N, K, 1.0f, nullptr, kmin, 0, nullptr, kmin, 0, 0.0f, C, ldc, 0, 1, ws, ws_bytes);
    Span used[6];
    int n = 0;
    if (!empty) {
        if (!C || misaligned(C, 4) || misaligned(scale_a, 4) || misaligned(scale_b, 4) ||
            (ws_bytes > 0 && misaligned(ws, 16)))
            return hipErrorInvalidValue;
        if (K > 0) {
            if (!A || !B) return hipErrorInvalidValue;
            used[n++] = row_span(RowTensor{A, lda, 1}, M, K);
            used[n++] = row_span(RowTensor{B, ldb, 1}, N, K);
        }
        if (scale_a) used[n++] = row_span(RowTensor{scale_a, M, 4}, 1, M);
        if (scale_b) used[n++] = row_span(RowTensor{scale_b, N, 4}, 1, N);
        if (ws_bytes > 0) {
            const Span w{(uintptr_t)ws, (uintptr_t)ws + ws_bytes};
            if (overlaps_any(w, used, n)) return hipErrorInvalidValue;
            used[n++] = w;
        }
    }
    sgemm::Epi e = {};
    const sgemm_epilogue none = {};
    const hipError_t x = make_epi(epi ? *epi : none, c.p, C, 0, used, n, &e);
    if (x != hipSuccess) return x;
    if (empty) return hipSuccess;
    if (ws_bytes > 0 && !workspace_clear(used[n - 1], e, c.p)) return hipErrorInvalidValue;
    if (K > 0) {  // (a sum of nothing stays 0 whatever the scales hold)
        e.scale_a = scale_a;
        e.scale_b = scale_b;
    }
    c.epi = &e;
    if (K == 0) return launch_reduce(c, 0, 0.0f, stream);
    int cus = 0;
    hipError_t err = device_cus(&cus);
    if (err != hipSuccess) return err;
    const bool aligned = e4m3_aligned(A, lda, B, ldb);
    const sgemm::E4m3Plan plan = sgemm::e4m3_plan(
        M, N, K, cus, aligned, ws_bytes > (size_t)LLONG_MAX ? LLONG_MAX : (long long)ws_bytes);
    if (plan.kernel == sgemm::kE4m3None) return hipErrorInvalidValue;
    sgemm::E4m3Args g = {};
    g.A = static_cast<const float *>(A);
    g.B = static_cast<const float *>(B);
    g.ld_a = lda;
    g.ld_b = ldb;
    g.C = C;
    g.M = M;
    g.N = N;
    g.K = K;
    g.ldc = ldc;
    g.k_chunk = plan.k_chunk;
    g.splits = plan.splits;
    g.group_m = sgemm::kDefaultGroupM;
    g.xcd_remap = sgemm::kDefaultXcdRemap;
    g.alpha = 1.0f;
    g.e = e;
    if (plan.kernel < 0) {
        const E4m3SkinnyKernel &s = kE4m3SkinnyKernels[-1 - plan.kernel];
        const long long wgs = sgemm::ceil_div_ll(N, 16), cap = max_wgs_per_launch(s.threads);
        return launch1(s.fn, dim3((unsigned)(wgs < cap ? wgs : cap)), s.threads, &g, stream);
    }
    const E4m3TileKernel &v = kE4m3TileKernels[plan.kernel];
    g.tiles_m = (int)sgemm::ceil_div_ll(M, sgemm::kE4m3Tiles[plan.kernel].bm);
    g.tiles_n = (int)sgemm::ceil_div_ll(N, sgemm::kE4m3Tiles[plan.kernel].bn);
    if (plan.splits > 1) {
        g.e = sgemm::Epi{};
        g.C = static_cast<float *>(ws);
        g.ldc = (int)sgemm::partial_ld(N);
        g.split_c = (long long)M * g.ldc;
    }
    const long long grid = (long long)g.tiles_m * g.tiles_n * plan.splits, per = max_wgs_per_launch(v.threads);
    for (long long base = 0; base < grid; base += per) {
        g.wg_base = (int)base;
        err = launch1(aligned ? v.direct : v.reg, dim3((unsigned)(grid - base < per ? grid - base : per)), v.threads,
                      &g, stream);
        if (err != hipSuccess) return err;
    }
    return plan.splits > 1 ? launch_reduce(c, plan.splits, 1.0f, stream) : hipSuccess;
}
