// Host side of the gated feed-forward block: argument checks, the choice of a
// form and the launches, in float32 (sgemm_gated.hpp, gated_rows.hpp) and for
// 8-bit operands (gemm_e4m3.hpp), and its elementwise gradient (gate.hpp).
// Included by sgemm.hip inside its anonymous namespace, after
// layernorm_host.hpp.

// ---- what both types share -----------------------------------------------------------

// Checks a gate against the M x N output and the `n` pieces of memory that the
// call reads besides; converts it for the kernels.  ws: the workspace (bytes 0:
// none), which the call writes.
hipError_t make_gate(const sgemm_gate &s, int M, int N, const Piece &c, const Piece *used, int n, void *ws,
                     size_t ws_bytes, sgemm::Gate *out)
{
    if (s.activation < SGEMM_ACT_NONE || s.activation > SGEMM_ACT_SILU) return hipErrorInvalidValue;
    sgemm::Gate e = {};
    e.act = s.activation;
    *out = e;
    if (M == 0 || N == 0) return hipSuccess;
    if (misaligned(s.bias_gate, 4) || misaligned(s.bias_up, 4)) return hipErrorInvalidValue;
    const RowTensor pg{s.pre_gate, s.ld_pre_gate, 4}, pu{s.pre_up, s.ld_pre_up, 4};
    if ((s.pre_gate && !row_tensor_ok(pg, N)) || (s.pre_up && !row_tensor_ok(pu, N))) return hipErrorInvalidValue;
    constexpr int kMost = 11;  // six inputs, two biases, three outputs
    Piece in[kMost];
    int m = 0;
    for (int i = 0; i < n; ++i) in[m++] = used[i];
    in[m++] = Piece{RowTensor{s.bias_gate, N, 4}, 1, N};
    in[m++] = Piece{RowTensor{s.bias_up, N, 4}, 1, N};
    const Piece written[3] = {c, Piece{pg, M, N}, Piece{pu, M, N}};
    for (int i = 0; i < 3; ++i) {
        if (pieces_overlap_any(written[i], in, m) || pieces_overlap_any(written[i], written + i + 1, 2 - i))
            return hipErrorInvalidValue;
        in[m + i] = written[i];
    }
    if (ws_bytes > 0) {
        const Span u{(uintptr_t)ws, (uintptr_t)ws + ws_bytes};
        for (int i = 0; i < m + 3; ++i)
            if (in[i].t.ptr && in[i].rows > 0 && in[i].cols > 0 &&
                overlap(u, row_span(in[i].t, in[i].rows, in[i].cols)))
                return hipErrorInvalidValue;
    }
    e.bias_gate = s.bias_gate;
    e.bias_up = s.bias_up;
    e.pre_gate = s.pre_gate;
    e.pre_up = s.pre_up;
    e.ld_pre_gate = s.ld_pre_gate;
    e.ld_pre_up = s.ld_pre_up;
    *out = e;
    return hipSuccess;
}

// C = gate of the two sums in the workspace, each `splits` partial ones (0: of
// nothing).
hipError_t launch_gate_reduce(const sgemm::Gate &e, int M, int N, int splits, const float *parts, float *C, int ldc,
                              hipStream_t stream)
{
    sgemm::GateReduceArgs r = {};
    r.ldp = (int)sgemm::partial_ld(N);
    r.P = parts;
    r.C = C;
    r.split_p = (int64_t)M * r.ldp;
    r.half_p = r.split_p * splits;
    r.quads = r.split_p / 4;
    r.M = M;
    r.N = N;
    r.ldc = ldc;
    r.splits = splits;
    r.e = e;
    const long long blocks = (r.quads + 255) / 256, per = max_wgs_per_launch(256);
    for (long long b0 = 0; b0 < blocks; b0 += per) {
        r.base = 256 * (int64_t)b0;
        const hipError_t x = launch1(reinterpret_cast<const void *>(&sgemm::gate_reduce_kernel),
                                     dim3((unsigned)(blocks - b0 < per ? blocks - b0 : per)), 256, &r, stream);
        if (x != hipSuccess) return x;
    }
    return hipSuccess;
}

// Bytes of both sums' partials.
long long gate_parts_bytes(int M, int N, int splits) { return 8ll * splits * M * sgemm::partial_ld(N); }

// ---- float32 ----------------------------------------------------------------------------

// The fused tiles: bm x bn of work, bm x bn / 2 outputs.  Their main loops are
// those of the plain product's tiles of the same size (kVariants 4, 7, 20 and
// with 4-byte loads 19, 13, 21), and so are the rates and fixed costs.  Two
// workgroups of the smaller ones share a compute unit and pay their fixed costs
// together (1472 x 1790 x 500, microseconds, launch included, model and measured: 60
// and 59 on 64x64 tiles, 66 and 66 on 128x128).
struct GatedTile {
    int bm, bn, bk;
    bool dword;  // 4-byte loads: rows that do not start 16-byte aligned
    int threads, eff_permille, eff_one_permille, fixed_ns, coresident;
    const void *fn[2];  // by transb
};
template <int BM, int BN, int BK, int WM, int WN, int ST, bool DW, int MB>
GatedTile gated_tile(int eff, int eff_one, int fixed_ns)
{
    return {BM, BN, BK, DW, WM * WN * 64, eff, eff_one, fixed_ns, BM < 256 ? 2 : 1,
            {reinterpret_cast<const void *>(&sgemm::sgemm_gated_kernel<BM, BN, BK, WM, WN, ST, false, DW, MB>),
             reinterpret_cast<const void *>(&sgemm::sgemm_gated_kernel<BM, BN, BK, WM, WN, ST, true, DW, MB>)}};
}
const GatedTile kGatedTiles[] = {
    gated_tile<256, 256, 32, 4, 2, 2, false, 32>(959, 954, 5000),
    gated_tile<128, 128, 32, 4, 2, 2, false, 32>(925, 928, 3500),
    gated_tile<64, 64, 32, 2, 2, 4, false, 16>(906, 868, 3900),
    gated_tile<256, 256, 16, 4, 2, 2, true, 32>(927, 950, 5000),
    gated_tile<128, 128, 32, 4, 2, 2, true, 32>(915, 888, 3500),
    gated_tile<64, 64, 32, 2, 2, 4, true, 16>(894, 770, 4455),
};
constexpr int kGatedTileCount = (int)(sizeof(kGatedTiles) / sizeof(kGatedTiles[0]));
static_assert(kGatedTileCount == SGEMM_GATED_TILES, "the header counts them");

struct GatedCall {
    int transb, M, N, K, lda, ldb[2], ldc;
    const float *A, *B[2];
    float *C;
    void *ws;
    size_t ws_bytes;
};

// The plain product of one half (or of both, as a batch of two), as the
// product's planner and launcher see it.
Call gated_product(const GatedCall &c, int half, int batch)
{
    const int ldp = (int)sgemm::partial_ld(c.N);
    return make_call(0, c.transb, c.M, c.N, c.K, 1.0f, c.A, c.lda, 0, c.B[half], c.ldb[half],
                     batch > 1 ? (long long)((intptr_t)c.B[1] - (intptr_t)c.B[0]) / 4 : 0, 0.0f, nullptr, ldp,
                     (long long)c.M * ldp, batch, nullptr, 0);
}

bool gated_aligned16(const GatedCall &c)
{
    return (((uintptr_t)c.A | (uintptr_t)c.B[0] | (uintptr_t)c.B[1]) & 15u) == 0 && c.lda % 4 == 0 &&
           c.ldb[0] % 4 == 0 && c.ldb[1] % 4 == 0;
}

// How a call runs: a tile's index, SGEMM_GATED_ROWS, or SGEMM_GATED_PRODUCTS
// with the plain product's plan.
struct GatedPlan {
    int form;
    sgemm::Choice choice;  // SGEMM_GATED_PRODUCTS
    long long workspace_bytes;
};

// Whether the two products can run as one batch of two.
bool gated_batch(const GatedCall &c) { return c.ldb[0] == c.ldb[1]; }

sgemm::Problem gated_problem(const GatedCall &c)
{
    return sgemm::Problem{0, c.transb, c.M, c.N, c.K, c.lda, c.ldb[0] > c.ldb[1] ? c.ldb[0] : c.ldb[1],
                          (int)sgemm::partial_ld(c.N), gated_batch(c) ? 2 : 1};
}

// The form for few rows, without the launch that every form pays: its cost beyond the
// stream, and the stream's rate over the chip, a share of it slower for each row past
// the first, and for weights stored (K, N) by the workgroups (32 columns each) there
// are.  Measured (microseconds, launch included), 1, 2 and 4 rows: 26.6, 28.0 and
// 30.0 for weights of 8192 x 2048 stored (N, K), 29.1 and 30.6 (1 and 4) stored
// (K, N); 65.6 for one row of 2048 x 8192 stored so, 64 workgroups, against 22.5.
// With more rows the fixed cost is paid by every round of workgroups: 45 rows of
// 2048 x 84, 11.4; 25 rows of 2371 x 163 stored (K, N), 25.1.
constexpr double kGatedRowsNs = 2000.0, kGatedRowsNsXc = 5000.0;
constexpr int kGatedRowsPerCu = 4, kGatedRowsPerCuXc = 1;  // workgroups that share a compute unit
constexpr double kGatedRowsBytesPerNs = 6300.0, kGatedRowsBytesPerNsXc = 5600.0, kGatedRowsWgBytesPerNsXc = 36.0;
constexpr double kGatedRowsPerRow = 0.05;
// The second pass that two products need (its launch, and the wait for the
// first ones).
constexpr double kGateReduceNs = 5000.0;

double gated_rows_ns(const GatedCall &c, int cus)
{
    const long long blocks = sgemm::ceil_div_ll(c.M, sgemm::kGatedRows);
    const double rows = c.M < sgemm::kGatedRows ? c.M : sgemm::kGatedRows;
    const long long wgs = blocks * sgemm::ceil_div_ll(c.N, c.transb ? 8 : 32);
    const double rate = c.transb ? kGatedRowsBytesPerNs
                                 : std::min(kGatedRowsBytesPerNsXc, kGatedRowsWgBytesPerNsXc * (double)wgs);
    const double fixed = c.transb ? kGatedRowsNs * (double)sgemm::ceil_div_ll(wgs, kGatedRowsPerCu * (long long)cus)
                                  : kGatedRowsNsXc * (double)sgemm::ceil_div_ll(wgs, kGatedRowsPerCuXc * (long long)cus);
    return fixed + (double)blocks * 8.0 * c.K * (double)c.N * (1.0 + kGatedRowsPerRow * (rows - 1.0)) / rate;
}

double gated_tile_ns(const GatedTile &v, const GatedCall &c, int cus)
{
    const long long tiles = sgemm::ceil_div_ll(c.M, v.bm) * sgemm::ceil_div_ll(c.N, v.bn / 2);
    const double eff = (tiles <= cus ? v.eff_one_permille : v.eff_permille) / 1000.0;
    const double slice_ns = 2.0 * v.bm * v.bn * v.bk / (sgemm::kCuFlopPerNs * eff);
    return (double)sgemm::ceil_div_ll(tiles, (long long)cus * v.coresident) * v.fixed_ns +
           (double)sgemm::ceil_div_ll(tiles, cus) * (double)sgemm::ceil_div_ll(c.K, v.bk) * slice_ns;
}

// Whether a tile can serve the call: offsets in 32 bits, and a grid that a launch counts.
bool gated_tile_serves(const GatedTile &v, const GatedCall &c)
{
    const int ldb = c.ldb[0] > c.ldb[1] ? c.ldb[0] : c.ldb[1];
    return c.lda <= sgemm::kMaxLdK && ldb <= (c.transb ? sgemm::kMaxLdK : sgemm::kMaxLdX) &&
           sgemm::ceil_div_ll(c.M, v.bm) * sgemm::ceil_div_ll(c.N, v.bn / 2) <= INT_MAX;
}

// The best two products into the workspace; their time to *ns (negative: none).
GatedPlan gated_products_plan(const GatedCall &c, int cus, long long ws, double *ns)
{
    GatedPlan plan = {SGEMM_GATED_PRODUCTS, {-1, 1, 0, 0}, 0};
    *ns = -1.0;
    const sgemm::Problem q = gated_problem(c);
    const long long one = gate_parts_bytes(c.M, c.N, 1);
    if (one > ws || !sgemm::sizes_ok(q)) return plan;
    // (the planner counts the partials of its own batch: here they are kept for
    // both products whether one launch makes them or two)
    const sgemm::Choice ch = sgemm::select_plan(kVariants, kNumVariants, q, cus, gated_aligned16(c),
                                                sgemm::direct_lds_ok(q), q.batch == 2 ? ws : ws / 2, false, false, ns);
    if (ch.id < 0) return plan;
    plan.choice = ch;
    plan.workspace_bytes = gate_parts_bytes(c.M, c.N, ch.splits);
    if (plan.workspace_bytes > ws) {
        *ns = -1.0;
        return plan;
    }
    if (q.batch == 1) *ns *= 2.0;
    if (ch.splits <= 1) *ns += kGateReduceNs + 12.0 * (double)c.M * (double)c.N / sgemm::kReduceBytesPerNs;
    return plan;
}

GatedPlan gated_plan(const GatedCall &c, int cus, long long ws)
{
    GatedPlan best = {SGEMM_GATED_ROWS, {-1, 1, 0, 0}, 0};
    double best_t = gated_rows_ns(c, cus);
    const bool aligned = gated_aligned16(c);
    for (int i = 0; i < kGatedTileCount; ++i) {
        const GatedTile &v = kGatedTiles[i];
        if (v.dword == aligned || !gated_tile_serves(v, c)) continue;
        const double t = gated_tile_ns(v, c, cus);
        if (t < best_t) {
            best = {i, {-1, 1, 0, 0}, 0};
            best_t = t;
        }
    }
    double t = -1.0;
    const GatedPlan p = gated_products_plan(c, cus, ws, &t);
    if (t >= 0.0 && t < best_t) best = p;
    return best;
}

// A call's plan, remembered per thread for the last few distinct ones as the
// plain product's is (cached_plan): the search costs about 5 us.
struct GatedPlanKey {
    sgemm::Problem p;
    int ldb_up, cus, aligned;
    long long ws;
};
struct GatedPlanEntry {
    GatedPlanKey key;
    GatedPlan plan;
    int valid;
};
thread_local GatedPlanEntry t_gated_plans[kPlanCacheEntries];
thread_local int t_gated_next;

GatedPlan cached_gated_plan(const GatedCall &c, int cus, long long ws)
{
    GatedPlanKey key;
    memset(&key, 0, sizeof(key));  // padding too: keys compare bytewise
    key.p = sgemm::Problem{0, c.transb, c.M, c.N, c.K, c.lda, c.ldb[0], 0, 1};
    key.ldb_up = c.ldb[1];
    key.cus = cus;
    key.aligned = gated_aligned16(c) ? 1 : 0;
    key.ws = ws;
    for (const GatedPlanEntry &e : t_gated_plans)
        if (e.valid && memcmp(&e.key, &key, sizeof(key)) == 0) return e.plan;
    const GatedPlan plan = gated_plan(c, cus, ws);
    GatedPlanEntry &e = t_gated_plans[t_gated_next];
    t_gated_next = (t_gated_next + 1) % kPlanCacheEntries;
    e.key = key;
    e.plan = plan;
    e.valid = 1;
    return plan;
}

hipError_t launch_gated_tile(const GatedTile &v, const GatedCall &c, const sgemm::Gate &e, hipStream_t stream)
{
    const sgemm::Problem q = gated_problem(c);
    sgemm::GatedArgs g = {};
    g.A = c.A;
    g.B = c.B[0];
    g.B_up = c.B[1];
    g.C = c.C;
    g.M = c.M;
    g.N = c.N;
    g.K = c.K;
    g.lda = c.lda;
    g.ldb = c.ldb[0];
    g.ldb_up = c.ldb[1];
    g.ldc = c.ldc;
    g.k_chunk = c.K;
    g.splits = 1;
    g.tiles_m = (int)sgemm::ceil_div_ll(c.M, v.bm);
    g.tiles_n = (int)sgemm::ceil_div_ll(c.N, v.bn / 2);
    g.group_m = sgemm::kDefaultGroupM;
    g.xcd_remap = sgemm::kDefaultXcdRemap;
    g.direct = sgemm::direct_lds_ok(q) && (v.dword || gated_aligned16(c)) ? 1 : 0;
    g.e = e;
    const long long grid = (long long)g.tiles_m * g.tiles_n, per = max_wgs_per_launch(v.threads);
    for (long long base = 0; base < grid; base += per) {
        g.wg_base = (int)base;
        const hipError_t x = launch1(v.fn[c.transb], dim3((unsigned)(grid - base < per ? grid - base : per)),
                                     v.threads, &g, stream);
        if (x != hipSuccess) return x;
    }
    return hipSuccess;
}

// Few rows: the form by the rows there are, and for weights stored (N, K) by
// whether two columns a wave fill the chip (else four waves split K).
hipError_t launch_gated_rows(const GatedCall &c, const sgemm::Gate &e, int cus, hipStream_t stream)
{
    sgemm::GatedRowsArgs g = {};
    g.A = c.A;
    g.B[0] = c.B[0];
    g.B[1] = c.B[1];
    g.C = c.C;
    g.lda = c.lda;
    g.ldb[0] = c.ldb[0];
    g.ldb[1] = c.ldb[1];
    g.ldc = c.ldc;
    g.M = c.M;
    g.N = c.N;
    g.K = c.K;
    g.e = e;
    const int mr = c.M >= 3 ? 2 : c.M - 1;  // index of 1, 2, 4 rows
    const void *fn;
    int threads, cols;
    if (c.transb) {
        static const void *const fns[2][3] = {
            {reinterpret_cast<const void *>(&sgemm::gated_rows_kc_kernel<1, 1>),
             reinterpret_cast<const void *>(&sgemm::gated_rows_kc_kernel<2, 1>),
             reinterpret_cast<const void *>(&sgemm::gated_rows_kc_kernel<4, 1>)},
            {reinterpret_cast<const void *>(&sgemm::gated_rows_kc_kernel<1, 4>),
             reinterpret_cast<const void *>(&sgemm::gated_rows_kc_kernel<2, 4>),
             reinterpret_cast<const void *>(&sgemm::gated_rows_kc_kernel<4, 4>)}};
        const bool split = sgemm::ceil_div_ll(c.N, 8) < 4 * cus && c.K >= 1024;
        fn = fns[split][mr];
        threads = 256;
        cols = split ? 2 : 8;
    } else {
        static const void *const fns[3] = {reinterpret_cast<const void *>(&sgemm::gated_rows_xc_kernel<1>),
                                           reinterpret_cast<const void *>(&sgemm::gated_rows_xc_kernel<2>),
                                           reinterpret_cast<const void *>(&sgemm::gated_rows_xc_kernel<4>)};
        fn = fns[mr];
        threads = sgemm::kRowsThreads;
        cols = 32;
    }
    const long long x = sgemm::ceil_div_ll(c.N, cols), y = sgemm::ceil_div_ll(c.M, sgemm::kGatedRows);
    // (the dispatch packet counts work-items in 32 bits, and a grid's second
    // dimension to 65535)
    const long long per_x = max_wgs_per_launch(threads) < x ? max_wgs_per_launch(threads) : x;
    long long per_y = max_wgs_per_launch(threads) / per_x;
    per_y = per_y < 1 ? 1 : per_y > 65535 ? 65535 : per_y;
    for (long long y0 = 0; y0 < y; y0 += per_y)
        for (long long x0 = 0; x0 < x; x0 += per_x) {
            g.m_base = (int)(y0 * sgemm::kGatedRows);
            g.n_base = x0 * cols;
            const hipError_t r = launch1(fn, dim3((unsigned)(x - x0 < per_x ? x - x0 : per_x),
                                                  (unsigned)(y - y0 < per_y ? y - y0 : per_y)),
                                         threads, &g, stream);
            if (r != hipSuccess) return r;
        }
    return hipSuccess;
}

hipError_t launch_gated_products(const GatedCall &c, const GatedPlan &plan, const sgemm::Gate &e, hipStream_t stream)
{
    const int batch = gated_batch(c) ? 2 : 1;
    const int ldp = (int)sgemm::partial_ld(c.N), splits = plan.choice.splits;
    float *const ws = static_cast<float *>(c.ws);
    for (int half = 0; half < (batch == 2 ? 1 : 2); ++half) {
        Call p = gated_product(c, half, batch);
        sgemm_cfg cfg;
        if (!sgemm::finish_cfg(kVariants[plan.choice.id], plan.choice.id, p.p, splits, 0, 0, &cfg))
            return hipErrorInvalidValue;
        // a split product leaves its partials in the workspace, a whole one its result
        p.ws = p.C = ws + (long long)half * splits * c.M * ldp;
        const hipError_t r = launch_gemm(kVariants[plan.choice.id], cfg, p, stream);
        if (r != hipSuccess) return r;
    }
    return launch_gate_reduce(e, c.M, c.N, splits, ws, c.C, c.ldc, stream);
}

bool gated_sizes_ok(int transb, int M, int N, int K, int lda, int ldb_gate, int ldb_up, int ldc)
{
    sgemm::Problem p{0, transb, M, N, K, lda, ldb_gate, ldc, 1};
    if (!sgemm::sizes_ok(p)) return false;
    p.ldb = ldb_up;
    return sgemm::sizes_ok(p);
}

hipError_t run_gated(int transb, int M, int N, int K, const float *A, int lda, const float *Bg, int ldg,
                     const float *Bu, int ldu, float *C, int ldc, const sgemm_gate *gate, void *ws, size_t ws_bytes,
                     int form, hipStream_t stream)
{
    if (!gated_sizes_ok(transb, M, N, K, lda, ldg, ldu, ldc) || !gate) return hipErrorInvalidValue;
    if (form < SGEMM_GATED_AUTO || form > SGEMM_GATED_PRODUCTS) return hipErrorInvalidValue;
    if (!ws) ws_bytes = 0;
    const bool empty = M == 0 || N == 0;
    Piece used[3];
    int n = 0;
    const Piece pc{RowTensor{C, ldc, 4}, M, N};
    if (!empty) {
        if (!row_tensor_ok(pc.t, N) || (ws_bytes > 0 && misaligned(ws, 16))) return hipErrorInvalidValue;
        if (K > 0) {
            const RowTensor a{A, lda, 4}, bg{Bg, ldg, 4}, bu{Bu, ldu, 4};
            const int rows = transb ? N : K, cols = transb ? K : N;
            if (!row_tensor_ok(a, K) || !row_tensor_ok(bg, cols) || !row_tensor_ok(bu, cols))
                return hipErrorInvalidValue;
            used[n++] = Piece{a, M, K};
            used[n++] = Piece{bg, rows, cols};
            used[n++] = Piece{bu, rows, cols};
        }
    }
    sgemm::Gate e;
    const hipError_t x = make_gate(*gate, M, N, pc, used, n, ws, ws_bytes, &e);
    if (x != hipSuccess) return x;
    if (empty) return hipSuccess;
    if (K == 0) return launch_gate_reduce(e, M, N, 0, nullptr, C, ldc, stream);
    const GatedCall c{transb, M, N, K, lda, {ldg, ldu}, ldc, A, {Bg, Bu}, C, ws, ws_bytes};
    const long long room = ws_bytes > (size_t)LLONG_MAX ? LLONG_MAX : (long long)ws_bytes;
    // (arguments are checked before the first HIP call)
    if (form >= 0 && form < kGatedTileCount && !gated_tile_serves(kGatedTiles[form], c)) return hipErrorInvalidValue;
    if (form == SGEMM_GATED_PRODUCTS && gate_parts_bytes(M, N, 1) > room) return hipErrorInvalidValue;
    int cus = 0;
    const hipError_t err = device_cus(&cus);
    if (err != hipSuccess) return err;
    GatedPlan plan = {form, {-1, 1, 0, 0}, 0};
    if (form == SGEMM_GATED_AUTO) {
        plan = cached_gated_plan(c, cus, room);
    } else if (form == SGEMM_GATED_PRODUCTS) {
        double ns;
        plan = gated_products_plan(c, cus, room, &ns);
        if (ns < 0.0) return hipErrorInvalidValue;
    }
    if (plan.form < kGatedTileCount) return launch_gated_tile(kGatedTiles[plan.form], c, e, stream);
    if (plan.form == SGEMM_GATED_ROWS) return launch_gated_rows(c, e, cus, stream);
    return launch_gated_products(c, plan, e, stream);
}

// ---- the sum of two products ------------------------------------------------------------

// C = A1 op(B1) + A2 op(B2): as one batch of two whose partial products (and
// those of a K split) are added by one reduction, or one product after the other,
// the second added to the first's result.  The batch has twice the tiles, which
// pays where one product does not fill the chip.
struct PairCall {
    Call c[2];  // as the product's entry takes them, the second with beta 1
};

struct PairPlan {
    bool batch;
    sgemm::Choice choice;  // of the batch
    long long workspace_bytes;
};

// The batch's problem (its partials as the workspace holds them).
sgemm::Problem pair_problem(const PairCall &p)
{
    sgemm::Problem q = p.c[0].p;
    q.batch = 2;
    q.ldc = (int)sgemm::partial_ld(q.N);
    return q;
}

PairPlan pair_plan(const PairCall &p, int cus, long long ws)
{
    const sgemm::Problem &one = p.c[0].p, two = pair_problem(p);
    const bool aligned = rows_aligned16(p.c[0]) && rows_aligned16(p.c[1]), lds_ok = sgemm::direct_lds_ok(one);
    double t1 = 0.0, t2 = 0.0;
    const sgemm::Choice ch = sgemm::select_plan(kVariants, kNumVariants, one, cus, aligned, lds_ok, ws, false, true, &t1);
    PairPlan plan = {false, {-1, 1, 0, 0}, ch.id < 0 ? 0 : sgemm::split_workspace_bytes(
                     sgemm::main_block(one, ch.strip_m, ch.strip_n), ch.splits)};
    if (gate_parts_bytes(one.M, one.N, 1) > ws || one.ldb != p.c[1].p.ldb || one.lda != p.c[1].p.lda) return plan;
    const sgemm::Choice both = sgemm::select_plan(kVariants, kNumVariants, two, cus, aligned, lds_ok, ws, false, false, &t2);
    const long long bytes = gate_parts_bytes(one.M, one.N, both.splits);
    if (both.id < 0 || bytes > ws) return plan;
    // (a split's reduction is in its time; it writes one sum here, not two)
    if (both.splits <= 1) t2 += sgemm::kReduceFixedNs + 12.0 * (double)one.M * (double)one.N / sgemm::kReduceBytesPerNs;
    if (ch.id < 0 || t2 < 2.0 * t1 + sgemm::kLaunchFloorNs) plan = {true, both, bytes};
    return plan;
}

hipError_t run_pair(PairCall &p, hipStream_t stream)
{
    for (const Call &c : p.c) {
        const hipError_t e = validate(c);
        if (e != hipSuccess) return e;
    }
    const sgemm::Problem &one = p.c[0].p;
    if (one.M == 0 || one.N == 0) return hipSuccess;
    if (one.K == 0) return (hipError_t)run(p.c[0], stream, nullptr);
    int cus = 0;
    hipError_t e = device_cus(&cus);
    if (e != hipSuccess) return e;
    const PairPlan plan =
        pair_plan(p, cus, p.c[0].ws_bytes > (size_t)LLONG_MAX ? LLONG_MAX : (long long)p.c[0].ws_bytes);
    if (!plan.batch) {
        for (const Call &c : p.c) {
            e = (hipError_t)run(c, stream, nullptr);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    Call both = p.c[0];
    both.p = pair_problem(p);
    both.sa = (long long)((intptr_t)p.c[1].A - (intptr_t)p.c[0].A) / 4;
    both.sb = (long long)((intptr_t)p.c[1].B - (intptr_t)p.c[0].B) / 4;
    both.C = static_cast<float *>(both.ws);
    both.sc = (long long)one.M * both.p.ldc;
    sgemm_cfg cfg;
    const Variant &v = kVariants[plan.choice.id];
    if (!sgemm::finish_cfg(v, plan.choice.id, both.p, plan.choice.splits, 0, 0, &cfg)) return hipErrorInvalidValue;
    e = launch_gemm(v, cfg, both, stream);
    // (the partial sums of both products lie one after the other)
    return e == hipSuccess ? launch_reduce(p.c[0], 2 * cfg.splits, 1.0f, stream) : e;
}

PairCall make_pair(int transb, int M, int N, int K, const float *A1, const float *A2, int lda, const float *B1, int ldb1,
                   const float *B2, int ldb2, float *C, int ldc, void *ws, size_t ws_bytes)
{
    return {{make_call(0, transb, M, N, K, 1.0f, A1, lda, 0, B1, ldb1, 0, 0.0f, C, ldc, 0, 1, ws, ws_bytes),
             make_call(0, transb, M, N, K, 1.0f, A2, lda, 0, B2, ldb2, 0, 1.0f, C, ldc, 0, 1, ws, ws_bytes)}};
}

// ---- 8 bits ---------------------------------------------------------------------------------

template <int BM, int BN, int BKF, int WM, int WN, int ST, int MB> const void *e4m3_gated_fn()
{
    return reinterpret_cast<const void *>(&sgemm::gemm_e4m3_kernel<BM, BN, BKF, WM, WN, ST, MB, false, true>);
}
template <int BM, int BN, int BKF, int WM, int WN, int MB> const void *e4m3_gated_reg_fn()
{
    return reinterpret_cast<const void *>(&sgemm::gemm_e4m3_kernel<BM, BN, BKF, WM, WN, 2, MB, true, true>);
}

// The gated forms of kE4m3TileKernels and kE4m3SkinnyKernels, in their order.
const E4m3TileKernel kE4m3GatedTiles[sgemm::kE4m3TileCount] = {
    {512, e4m3_gated_fn<256, 256, 16, 4, 2, 4, 32>(), nullptr},
    {256, e4m3_gated_fn<128, 128, 32, 2, 2, 2, 32>(), e4m3_gated_reg_fn<128, 128, 32, 2, 2, 32>()},
    {256, e4m3_gated_fn<64, 128, 32, 2, 2, 2, 32>(), e4m3_gated_reg_fn<64, 128, 32, 2, 2, 32>()},
    {256, e4m3_gated_fn<64, 64, 32, 2, 2, 2, 16>(), e4m3_gated_reg_fn<64, 64, 32, 2, 2, 16>()},
};
// Up to 16 rows where 16 columns a workgroup leave compute units idle: 8 columns of each
// weight (1 and 16 rows in a graph, microseconds, 16 and 8 columns: two weights of 1024 x
// 4096 8.2 and 6.5, 10.0 and 8.1; 2048 x 8192 13.9 and 12.2, 15.9 and 13.3; with as many
// workgroups as compute units, 4096 x 4096, 11.8 and 10.7, 12.0 and 13.0).  The rule
// goes by the columns alone, so a single row of just as many columns as that leaves
// those 10% for what 16 rows would lose.
const E4m3SkinnyKernel kE4m3GatedNarrow = {
    128, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<2, 1, true, true>)};
const E4m3SkinnyKernel kE4m3GatedSkinny[sgemm::kE4m3SkinnyCount] = {
    {128, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<2, 1, true>)},
    {256, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<4, 2, true>)},
    {256, reinterpret_cast<const void *>(&sgemm::gemm_e4m3_skinny_kernel<4, 4, true>)},
};

hipError_t run_e4m3_gated(int M, int N, int K, const void *A, int lda, const float *scale_a, const void *Bg, int ldg,
                          const float *scale_gate, const void *Bu, int ldu, const float *scale_up, float *C, int ldc,
                          const sgemm_gate *gate, void *ws, size_t ws_bytes, hipStream_t stream)
{
    const int kmin = K > 1 ? K : 1, nmin = N > 1 ? N : 1;
    if (!e4m3_sizes_ok(M, N, K) || !gate || lda < kmin || ldg < kmin || ldu < kmin || ldc < nmin ||
        lda > sgemm::kMaxDim || ldg > sgemm::kMaxDim || ldu > sgemm::kMaxDim || ldc > sgemm::kMaxDim)
        return hipErrorInvalidValue;
    if (!ws) ws_bytes = 0;
    const bool empty = M == 0 || N == 0;
    Piece used[6];
    int n = 0;
    const Piece pc{RowTensor{C, ldc, 4}, M, N};
    if (!empty) {
        if (!row_tensor_ok(pc.t, N) || misaligned(scale_a, 4) || misaligned(scale_gate, 4) || misaligned(scale_up, 4) ||
            (ws_bytes > 0 && misaligned(ws, 16)))
            return hipErrorInvalidValue;
        if (K > 0) {
            if (!A || !Bg || !Bu) return hipErrorInvalidValue;
            used[n++] = Piece{RowTensor{A, lda, 1}, M, K};
            used[n++] = Piece{RowTensor{Bg, ldg, 1}, N, K};
            used[n++] = Piece{RowTensor{Bu, ldu, 1}, N, K};
        }
        used[n++] = Piece{RowTensor{scale_a, M, 4}, 1, M};
        used[n++] = Piece{RowTensor{scale_gate, N, 4}, 1, N};
        used[n++] = Piece{RowTensor{scale_up, N, 4}, 1, N};
    }
    sgemm::Gate e;
    const hipError_t x = make_gate(*gate, M, N, pc, used, n, ws, ws_bytes, &e);
    if (x != hipSuccess) return x;
    if (empty) return hipSuccess;
    if (K == 0) return launch_gate_reduce(e, M, N, 0, nullptr, C, ldc, stream);
    // (a sum of nothing stays 0 whatever the scales hold)
    e.scale_a = scale_a;
    e.scale_gate = scale_gate;
    e.scale_up = scale_up;
    int cus = 0;
    hipError_t err = device_cus(&cus);
    if (err != hipSuccess) return err;
    const bool aligned = e4m3_aligned(A, lda, Bg, ldg) && e4m3_aligned(A, lda, Bu, ldu);
    const sgemm::E4m3Plan plan =
        sgemm::e4m3_gated_plan(M, N, K, cus, aligned, ws_bytes > (size_t)LLONG_MAX ? LLONG_MAX : (long long)ws_bytes);
    if (plan.kernel == sgemm::kE4m3None) return hipErrorInvalidValue;
    sgemm::E4m3GatedArgs g = {};
    g.A = static_cast<const float *>(A);
    g.B = static_cast<const float *>(Bg);
    g.B_up = static_cast<const unsigned char *>(Bu);
    g.ld_a = lda;
    g.ld_b = ldg;
    g.ld_b_up = ldu;
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
    g.gate = e;
    if (plan.kernel < 0) {
        const bool narrow = plan.kernel == -1 && sgemm::ceil_div_ll(N, 16) < cus;
        const E4m3SkinnyKernel &s = narrow ? kE4m3GatedNarrow : kE4m3GatedSkinny[-1 - plan.kernel];
        const long long wgs = sgemm::ceil_div_ll(N, narrow ? 8 : 16), cap = max_wgs_per_launch(s.threads);
        return launch1(s.fn, dim3((unsigned)(wgs < cap ? wgs : cap)), s.threads, &g, stream);
    }
    const sgemm::E4m3Tile &t = sgemm::kE4m3Tiles[plan.kernel];
    const E4m3TileKernel &v = kE4m3GatedTiles[plan.kernel];
    g.tiles_m = (int)sgemm::ceil_div_ll(M, t.bm);
    g.tiles_n = (int)sgemm::ceil_div_ll(N, t.bn / 2);
    if (plan.splits > 1) {
        const int ldp = (int)sgemm::partial_ld(N);
        g.split_c = (long long)M * ldp;
        g.gate = sgemm::Gate{};
        g.gate.pre_gate = static_cast<float *>(ws);
        g.gate.pre_up = g.gate.pre_gate + plan.splits * g.split_c;
        g.gate.ld_pre_gate = g.gate.ld_pre_up = ldp;
        g.C = nullptr;
    }
    const long long grid = (long long)g.tiles_m * g.tiles_n * plan.splits, per = max_wgs_per_launch(v.threads);
    for (long long base = 0; base < grid; base += per) {
        g.wg_base = (int)base;
        err = launch1(aligned ? v.direct : v.reg, dim3((unsigned)(grid - base < per ? grid - base : per)), v.threads,
                      &g, stream);
        if (err != hipSuccess) return err;
    }
    if (plan.splits <= 1) return hipSuccess;
    return launch_gate_reduce(e, M, N, plan.splits, static_cast<const float *>(ws), C, ldc, stream);
}

// ---- the elementwise gradient -------------------------------------------------------------------

size_t gate_grad_bytes(int M, int N)
{
    return M > 0 && N > 0 ? (size_t)col_plan(M, N).chunks * 8u * (size_t)N : 0;
}

hipError_t run_gate_grad(int M, int N, int act, const float *dY, int ldy, const float *G, int ldg, const float *U,
                         int ldu, float *dG, int lddg, float *dU, int lddu, float *dbg, float *dbu, void *ws,
                         size_t ws_bytes, hipStream_t stream)
{
    if (M < 0 || N < 0 || M > sgemm::kMaxDim || N > sgemm::kMaxDim || act < SGEMM_ACT_NONE ||
        act > SGEMM_ACT_SILU || misaligned(dbg, 4) || misaligned(dbu, 4))
        return hipErrorInvalidValue;
    if (N == 0) return hipSuccess;
    const Piece pbg{RowTensor{dbg, N, 4}, 1, N}, pbu{RowTensor{dbu, N, 4}, 1, N};
    if (pieces_overlap(pbg, pbu)) return hipErrorInvalidValue;
    if (M == 0) {
        const hipError_t e = dbg ? launch_zero(dbg, N, stream) : hipSuccess;
        return e == hipSuccess && dbu ? launch_zero(dbu, N, stream) : e;
    }
    const RowTensor y{dY, ldy, 4}, g{G, ldg, 4}, u{U, ldu, 4}, og{dG, lddg, 4}, ou{dU, lddu, 4};
    if (!row_tensor_ok(y, N) || !row_tensor_ok(g, N) || !row_tensor_ok(u, N) || (dG && !row_tensor_ok(og, N)) ||
        (dU && !row_tensor_ok(ou, N)))
        return hipErrorInvalidValue;
    const bool sums = dbg || dbu;
    if (!dG && !dU && !sums) return hipSuccess;
    const size_t need = sums ? gate_grad_bytes(M, N) : 0;
    if (need > 0 && (!ws || misaligned(ws, 16) || ws_bytes < need)) return hipErrorInvalidValue;
    const Piece in[3] = {Piece{y, M, N}, Piece{g, M, N}, Piece{u, M, N}};
    const RowTensor in_t[3] = {y, g, u};
    const Piece out[4] = {Piece{og, M, N}, Piece{ou, M, N}, pbg, pbu};
    for (int o = 0; o < 4; ++o) {
        // dG and dU may take an input's place
        for (int i = 0; i < 3; ++i)
            if (pieces_overlap(out[o], in[i]) && !(o < 2 && same_tensor(out[o].t, in_t[i])))
                return hipErrorInvalidValue;
        if (pieces_overlap_any(out[o], out + o + 1, 3 - o)) return hipErrorInvalidValue;
    }
    if (need > 0) {
        const Span w{(uintptr_t)ws, (uintptr_t)ws + need};
        const Piece all[7] = {in[0], in[1], in[2], out[0], out[1], out[2], out[3]};
        for (const Piece &p : all)
            if (p.t.ptr && overlap(w, row_span(p.t, p.rows, p.cols))) return hipErrorInvalidValue;
    }
    const ColPlan p = col_plan(M, N);
    sgemm::GateGradArgs a = {};
    a.dY = dY;
    a.G = G;
    a.U = U;
    a.dG = dG;
    a.dU = dU;
    a.part = sums ? static_cast<float *>(ws) : nullptr;
    a.ldy = ldy;
    a.ldg = ldg;
    a.ldu = ldu;
    a.lddg = lddg;
    a.lddu = lddu;
    a.M = M;
    a.N = N;
    a.act = act;
    a.rows_per_chunk = p.rows_per_chunk;
    const void *fn = p.tx == 16 ? reinterpret_cast<const void *>(&sgemm::gate_grad_kernel<16>)
                                : reinterpret_cast<const void *>(&sgemm::gate_grad_kernel<64>);
    const hipError_t e = launch1(fn, dim3((unsigned)p.wgs, (unsigned)p.chunks), 256, &a, stream);
    return e == hipSuccess && sums ? launch_pair_sum(a.part, p.chunks, N, dbg, dbu, stream) : e;
}
