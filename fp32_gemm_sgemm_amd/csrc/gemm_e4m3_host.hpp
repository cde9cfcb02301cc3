// Host side of the 8-bit product (gemm_e4m3.hpp): argument checks, the choice
// of a kernel, and the launches.  Included by sgemm.hip inside its anonymous
// namespace, after the helpers of the float32 product.

// A tile, and its cost for the selection: the time of 1024 codes of K with n
// tiles per compute unit is lat_ns + n * rate_ns, and fill_ns is the rest of a
// tile (its first fetch and its epilogue; the launch is left out, as every
// plan pays it).  Measured on MI355X, random codes, float32 output without an
// epilogue: K = 1024 and 4096 (microseconds, launch included) at
//                 1024x1024     2048x2048     4096x4096
//   256x256        25.7  78      29.7  81      39.9 109.5
//   128x128        12.1  29      16.1  36      43.3 115.9
//   64x128          9.1  20      14.7  35      41.6 125.7
//   64x64           7.9  18      16.7  43      51.9 150.6
struct E4m3Variant {
    int bm, bn, threads;
    const void *direct;  // rows 16-byte aligned
    const void *reg;     // any rows (null: not compiled)
    double lat_ns, rate_ns, fill_ns;
};

template <int BM, int BN, int BKF, int WM, int WN, int ST, int MB> const void *e4m3_fn()
{
    return reinterpret_cast<const void *>(&sgemm::gemm_e4m3_kernel<BM, BN, BKF, WM, WN, ST, MB, false>);
}
template <int BM, int BN, int BKF, int WM, int WN, int MB> const void *e4m3_reg_fn()
{
    return reinterpret_cast<const void *>(&sgemm::gemm_e4m3_kernel<BM, BN, BKF, WM, WN, 2, MB, true>);
}

const E4m3Variant kE4m3Variants[] = {
    {256, 256, 512, e4m3_fn<256, 256, 16, 4, 2, 4, 32>(), nullptr, 0.0, 22000.0, 5800.0},
    {128, 128, 256, e4m3_fn<128, 128, 32, 2, 2, 2, 32>(), e4m3_reg_fn<128, 128, 32, 2, 2, 32>(), 0.0, 5900.0, 3800.0},
    {64, 128, 256, e4m3_fn<64, 128, 32, 2, 2, 2, 32>(), e4m3_reg_fn<64, 128, 32, 2, 2, 32>(), 600.0, 3400.0, 2800.0},
    {64, 64, 256, e4m3_fn<64, 64, 32, 2, 2, 2, 16>(), e4m3_reg_fn<64, 64, 32, 2, 2, 16>(), 1500.0, 1900.0, 2500.0},
};
// Rows that are not 16-byte aligned go through registers: this much slower.
constexpr double kE4m3RegCost = 1.13;
// Rate at which the tiles' results reach memory, all compute units at once,
// and the second pass of a K split beyond its traffic.
constexpr double kE4m3StoreBytesPerNs = 6000.0;
constexpr double kE4m3ReduceNs = 5000.0;
constexpr int kE4m3VariantCount = (int)(sizeof(kE4m3Variants) / sizeof(kE4m3Variants[0]));

// The streaming kernel for few rows of A, by the rows it holds: its cost is
// fill_ns plus, per 1024 codes of K, wg_ns + row_ns * M for each workgroup (16
// columns) of the fullest compute unit, or the weights' time from memory if that is more.
// Measured (microseconds, launch included) at N x K of 512 x 4096, 1024 x
// 16384 and 8192 x 8192: 4.9, 11.8 and 13.7 (16 rows: 6.6, 17.1, 17.8) with 2
// waves; 8.9, 24.7 and 27.2 for 32 rows and 13.2, 39.4 and 43.4 for 64 with 4.
struct E4m3Skinny {
    int rows, threads;
    const void *fn;
    double wg_ns, row_ns, fill_ns;
};
const E4m3Skinny kE4m3Skinny[] = {
    {16, 128, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<2, 1>), 575.0, 23.0, 100.0},
    {32, 256, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<4, 2>), 1350.0, 0.0, 1100.0},
    {64, 256, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<4, 4>), 2200.0, 0.0, 2000.0},
};
constexpr int kE4m3SkinnyCount = (int)(sizeof(kE4m3Skinny) / sizeof(kE4m3Skinny[0]));
constexpr double kE4m3StreamBytesPerNs = 6000.0;
// Direct loads keep a tile's byte offsets (256 rows and a slice) below 2^31.
constexpr int kE4m3MaxLdDirect = 1 << 23;
constexpr int kE4m3SplitAlign = 128;  // codes: whole slices, and 16-byte aligned starts

constexpr int kE4m3None = kE4m3VariantCount;  // more tiles than a grid counts
struct E4m3Plan {
    int variant;  // a tile, or the streaming kernel -1 - i, or kE4m3None
    int splits, k_chunk;
    long long workspace_bytes;
};

E4m3Plan e4m3_plan(int M, int N, int K, int cus, bool aligned, long long ws)
{
    E4m3Plan best = {kE4m3None, 1, K > 0 ? K : 1, 0};
    double best_t = -1.0;
    for (int i = 0; i < kE4m3SkinnyCount; ++i) {
        const E4m3Skinny &s = kE4m3Skinny[i];
        if (M > s.rows) continue;
        const double per_cu = (double)sgemm::ceil_div_ll(sgemm::ceil_div_ll(N, 16), cus);
        const double work = (double)K / 1024.0 * per_cu * (s.wg_ns + s.row_ns * M),
                     stream = (double)N * K / kE4m3StreamBytesPerNs;
        best = {-1 - i, 1, K > 0 ? K : 1, 0};
        best_t = s.fill_ns + (work > stream ? work : stream);
        break;
    }
    for (int i = 0; i < kE4m3VariantCount; ++i) {
        const E4m3Variant &v = kE4m3Variants[i];
        if (!aligned && !v.reg) continue;
        const long long tiles = sgemm::ceil_div_ll(M, v.bm) * sgemm::ceil_div_ll(N, v.bn);
        int last = 0;
        for (int want : sgemm::kSplitCandidates) {
            const long long per = sgemm::ceil_div_ll(sgemm::ceil_div_ll(K, want), kE4m3SplitAlign) * kE4m3SplitAlign;
            const int splits = (int)sgemm::ceil_div_ll(K, per);
            if (splits <= last) continue;
            last = splits;
            const long long bytes = splits > 1 ? (long long)splits * M * sgemm::partial_ld(N) * 4 : 0;
            if (bytes > ws || tiles * splits > INT_MAX) break;
            const double per_cu = (double)sgemm::ceil_div_ll(tiles * splits, cus);
            const double k = (double)(splits > 1 ? per : K) / 1024.0 * (aligned ? 1.0 : kE4m3RegCost);
            double t = v.fill_ns + k * (v.lat_ns + per_cu * v.rate_ns) +
                       4.0 * splits * (double)M * (double)N / kE4m3StoreBytesPerNs;
            if (splits > 1)
                t += kE4m3ReduceNs + 4.0 * (splits + 1) * (double)M * (double)N / sgemm::kReduceBytesPerNs;
            if (best_t < 0.0 || t < best_t) {
                best = {i, splits, splits > 1 ? (int)per : K, bytes};
                best_t = t;
            }
        }
    }
    return best;
}

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
    const E4m3Plan plan = e4m3_plan(M, N, K, cus, aligned,
                                    ws_bytes > (size_t)LLONG_MAX ? LLONG_MAX : (long long)ws_bytes);
    if (plan.variant == kE4m3None) return hipErrorInvalidValue;
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
    if (plan.variant < 0) {
        const E4m3Skinny &s = kE4m3Skinny[-1 - plan.variant];
        const long long wgs = sgemm::ceil_div_ll(N, 16), cap = max_wgs_per_launch(s.threads);
        return launch1(s.fn, dim3((unsigned)(wgs < cap ? wgs : cap)), s.threads, &g, stream);
    }
    const E4m3Variant &v = kE4m3Variants[plan.variant];
    g.tiles_m = (int)sgemm::ceil_div_ll(M, v.bm);
    g.tiles_n = (int)sgemm::ceil_div_ll(N, v.bn);
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
