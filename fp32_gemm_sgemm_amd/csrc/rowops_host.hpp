// Host side of the row and column operators (rowops.hpp): argument checks,
// the choice of a form by the row length, and the launches.  Included by
// sgemm.hip inside its anonymous namespace, after Span and its helpers.

// ---- row operators -----------------------------------------------------------------

// One row-major tensor of a row operator.
struct RowTensor {
    const void *ptr;
    int ld;
    int size;  // bytes per element
};

Span row_span(const RowTensor &t, int rows, int D)
{
    Span s;
    s.lo = (uintptr_t)t.ptr;
    s.hi = s.lo + ((uint64_t)(rows - 1) * (uint64_t)t.ld + (uint64_t)D) * (uint64_t)t.size;
    return s;
}

bool row_tensor_ok(const RowTensor &t, int D)
{
    return t.ptr && !misaligned(t.ptr, (uintptr_t)t.size) && t.ld >= D && t.ld <= sgemm::kMaxDim;
}

// The same memory with the same row stride.
bool same_tensor(const RowTensor &a, const RowTensor &b) { return a.ptr == b.ptr && a.ld == b.ld; }

bool row_sizes_ok(int rows, int D, float eps)
{
    return rows >= 0 && D >= 1 && rows <= sgemm::kMaxDim && D <= sgemm::kMaxDim && eps >= 0.0f &&
           eps <= 3.4028235e38f;
}

// A form of a row operator: threads per row, groups of 4 per thread (0: the
// form for any length).  Short rows go to one wave; from there on a workgroup
// of 256 threads, and of 1024 where 256 would hold more than 16 values a
// thread.
struct RowForm {
    int nt, v;
};
RowForm row_form(int D)
{
    if (D <= 256) return {64, 1};
    if (D <= 512) return {64, 2};
    if (D <= 1024) return {64, 4};
    if (D <= 2048) return {256, 2};
    if (D <= 4096) return {256, 4};
    if (D <= 8192) return {1024, 2};
    if (D <= sgemm::kRowCached) return {1024, 4};
    return {1024, 0};
}

// The form of a norm or quantisation.  Where a compute unit gets more than two
// rows, long ones go to workgroups of 512: four of them share a compute unit, and one's
// arithmetic overlaps another's memory (8192 x 8192: quantize 74 to 61 us, 8-bit
// norm with residual 182 to 166, norm 108 to 99; 2048 x 5120: 16 to 13, 36 to 31,
// 19 to 18; 600 x 8192: 9.3 to 8.3, 17.4 to 15.9, 10.9 to 10.3; at 512 rows they tie
// or lose up to 6%).  The norm with residual to float32, the one that moves 16
// bytes a value, gains so too while its tensors stay in the last-level cache (600 x
// 8192: 16.1 to 14.8, 2048 x 5120: 37 to 34) and loses 3% past it (8192 x 8192: 194
// to 200): it goes with the others.  Past 8192 values workgroups of 512 pay only
// where no residual is read too (4096 x 16384: quantize 77 to 69, norm with residual
// 208 to 214), but as soon as a compute unit gets more than one row (800 x 12000:
// quantize 17.0 to 13.8, 8-bit norm 23.3 to 19.0; 384 x 16384: 11.2 to 9.9 and 15.1
// to 13.0).  Fewer rows wait for one workgroup's latency, which more threads shorten
// (1 x 8192, norm with residual: 5.0 to 4.5 us; 256 x 16384, norm: 9.8 to 9.2).
RowForm row_form_forward(int D, int rows, bool residual)
{
    constexpr int kOneEach = 256, kTwoEach = 512;  // rows, on 256 compute units
    if (rows > kTwoEach && D > 4096 && D <= 8192) return {512, 4};
    if (rows > kOneEach && D > 8192 && D <= sgemm::kRowCached && !residual) return {512, 8};
    return row_form(D);
}

// Workgroups of a row operator: one per row (or four short ones), as many as
// the dispatch packet counts; the kernels loop over the rest.
unsigned row_grid(const RowForm &f, int rows, long long most)
{
    const int rpb = f.nt >= 256 ? 1 : 256 / f.nt;
    const long long n = ((long long)rows + rpb - 1) / rpb;
    const long long cap = max_wgs_per_launch(f.nt > 256 ? f.nt : 256);
    const long long lim = most > 0 && most < cap ? most : cap;
    return (unsigned)(n < lim ? n : lim);
}

hipError_t launch1(const void *fn, dim3 grid, int threads, void *args, hipStream_t stream)
{
    void *list[] = {args};
    return hipLaunchKernel(fn, grid, dim3((unsigned)threads), list, 0, stream);
}

template <bool NORM, bool Q8> const void *row_kernel_for(const RowForm &f)
{
    using sgemm::row_kernel;
    if (f.nt == 64) {
        if (f.v == 1) return reinterpret_cast<const void *>(&row_kernel<64, 1, NORM, Q8>);
        if (f.v == 2) return reinterpret_cast<const void *>(&row_kernel<64, 2, NORM, Q8>);
        return reinterpret_cast<const void *>(&row_kernel<64, 4, NORM, Q8>);
    }
    if (f.nt == 256) {
        if (f.v == 2) return reinterpret_cast<const void *>(&row_kernel<256, 2, NORM, Q8>);
        return reinterpret_cast<const void *>(&row_kernel<256, 4, NORM, Q8>);
    }
    if (f.nt == 512) {
        if (f.v == 4) return reinterpret_cast<const void *>(&row_kernel<512, 4, NORM, Q8>);
        return reinterpret_cast<const void *>(&row_kernel<512, 8, NORM, Q8>);
    }
    if (f.v == 2) return reinterpret_cast<const void *>(&row_kernel<1024, 2, NORM, Q8>);
    if (f.v == 4) return reinterpret_cast<const void *>(&row_kernel<1024, 4, NORM, Q8>);
    return reinterpret_cast<const void *>(&row_kernel<1024, 0, NORM, Q8>);
}

const void *row_grad_kernel_for(const RowForm &f)
{
    using sgemm::row_grad_kernel;
    if (f.nt == 64) {
        if (f.v == 1) return reinterpret_cast<const void *>(&row_grad_kernel<64, 1>);
        if (f.v == 2) return reinterpret_cast<const void *>(&row_grad_kernel<64, 2>);
        return reinterpret_cast<const void *>(&row_grad_kernel<64, 4>);
    }
    if (f.nt == 256) {
        if (f.v == 2) return reinterpret_cast<const void *>(&row_grad_kernel<256, 2>);
        return reinterpret_cast<const void *>(&row_grad_kernel<256, 4>);
    }
    if (f.nt == 512) return reinterpret_cast<const void *>(&row_grad_kernel<512, 4>);
    if (f.v == 2) return reinterpret_cast<const void *>(&row_grad_kernel<1024, 2>);
    if (f.v == 4) return reinterpret_cast<const void *>(&row_grad_kernel<1024, 4>);
    return reinterpret_cast<const void *>(&row_grad_kernel<1024, 0>);
}

// A norm or a quantisation.  norm: with the RMS scaling; q8: to codes.
hipError_t run_row(bool norm, bool q8, int rows, int D, const float *X, int ldx, const float *R, int ldr,
                   const float *w, float eps, float *S, int lds, float *Y, int ldy, void *Q, int ldq,
                   float *scale, hipStream_t stream)
{
    if (!row_sizes_ok(rows, D, eps)) return hipErrorInvalidValue;
    if (rows == 0) return hipSuccess;
    const RowTensor x{X, ldx, 4}, r{R, ldr, 4}, s{S, lds, 4};
    const RowTensor y = q8 ? RowTensor{Q, ldq, 1} : RowTensor{Y, ldy, 4};
    if (!row_tensor_ok(x, D) || (R && !row_tensor_ok(r, D)) || (S && !row_tensor_ok(s, D)) ||
        !row_tensor_ok(y, D) || misaligned(w, 4))
        return hipErrorInvalidValue;
    if (q8 && (!scale || misaligned(scale, 4))) return hipErrorInvalidValue;
    // outputs: S, Y or Q, scale
    const Span xs = row_span(x, rows, D), ys = row_span(y, rows, D);
    const Span rs = R ? row_span(r, rows, D) : Span{0, 0}, ss = S ? row_span(s, rows, D) : Span{0, 0};
    const Span ws = w ? row_span(RowTensor{w, D, 4}, 1, D) : Span{0, 0};
    const Span cs = q8 ? row_span(RowTensor{scale, rows, 4}, 1, rows) : Span{0, 0};
    const bool y_in_place = !q8;  // codes are of another size: no element keeps its place
    if ((overlap(ys, xs) && !(y_in_place && same_tensor(x, y))) ||
        (R && overlap(ys, rs) && !(y_in_place && same_tensor(r, y))) || overlap(ys, ws) || overlap(ys, cs))
        return hipErrorInvalidValue;
    if (S && ((overlap(ss, xs) && !same_tensor(s, x)) || (R && overlap(ss, rs) && !same_tensor(s, r)) ||
              overlap(ss, ys) || overlap(ss, ws) || overlap(ss, cs)))
        return hipErrorInvalidValue;
    if (overlap(cs, xs) || overlap(cs, rs) || overlap(cs, ws)) return hipErrorInvalidValue;
    sgemm::RowArgs a = {};
    a.X = X;
    a.R = R;
    a.w = w;
    a.S = S;
    a.Y = Y;
    a.Q = static_cast<unsigned char *>(Q);
    a.scale = scale;
    a.ldx = ldx;
    a.ldr = ldr;
    a.lds = lds;
    a.ldy = ldy;
    a.ldq = ldq;
    a.rows = rows;
    a.D = D;
    a.eps = eps;
    const RowForm f = row_form_forward(D, rows, R != nullptr);
    const void *fn = norm ? (q8 ? row_kernel_for<true, true>(f) : row_kernel_for<true, false>(f))
                          : row_kernel_for<false, true>(f);
    return launch1(fn, dim3(row_grid(f, rows, 0)), f.nt > 256 ? f.nt : 256, &a, stream);
}

// ---- column sums -----------------------------------------------------------------------

// How a column pass covers M x N: lanes along the columns, column workgroups,
// and chunks of rows, about kColWgs workgroups in all where the rows allow
// (four steps of a workgroup's rows at least).
constexpr long long kColWgs = 2048;
struct ColPlan {
    int tx, chunks, rows_per_chunk;
    long long wgs;
};
ColPlan col_plan(int M, int N)
{
    ColPlan p;
    p.tx = N > 128 ? 64 : 16;
    p.wgs = sgemm::ceil_div_ll(N, 4 * p.tx);
    const long long by_rows = sgemm::ceil_div_ll(M, 4 * (256 / p.tx));
    long long chunks = sgemm::ceil_div_ll(kColWgs, p.wgs);
    if (chunks > by_rows) chunks = by_rows;
    if (chunks < 1) chunks = 1;
    p.rows_per_chunk = (int)sgemm::ceil_div_ll(M > 0 ? M : 1, chunks);
    p.chunks = (int)sgemm::ceil_div_ll(M > 0 ? M : 1, p.rows_per_chunk);
    return p;
}

// Bytes of the chunks' sums (none where one chunk holds all rows: its sums
// are the result).
size_t parts_bytes(long long parts, int N) { return parts > 1 ? (size_t)parts * (size_t)N * 4u : 0; }

hipError_t launch_col_sum(const float *part, int parts, int N, float *out, hipStream_t stream)
{
    const float *p = part;
    int n = parts, w = N;
    void *list[] = {&p, &n, &w, &out};
    return hipLaunchKernel(reinterpret_cast<const void *>(&sgemm::col_sum_kernel),
                           dim3((unsigned)sgemm::ceil_div_ll(N, 32)), dim3(sgemm::kColSumThreads), list, 0, stream);
}

hipError_t launch_zero(float *p, int n, hipStream_t stream)
{
    void *list[] = {&p, &n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&sgemm::fill_zero_kernel),
                           dim3((unsigned)sgemm::ceil_div_ll(n, 256)), dim3(256), list, 0, stream);
}

// A column pass, and the sum of its chunks to `out` (null: no sums) through
// `parts` (used when there is more than one chunk).
template <int KIND>
hipError_t run_cols(sgemm::ColArgs a, float *out, float *parts, hipStream_t stream)
{
    const ColPlan p = col_plan(a.M, a.N);
    a.rows_per_chunk = p.rows_per_chunk;
    a.part = out ? (p.chunks > 1 ? parts : out) : nullptr;
    const void *fn = reinterpret_cast<const void *>(&sgemm::col_kernel<KIND, 64>);
    // (a norm's column pass is for rows past kRowCached values: never narrow)
    if constexpr (KIND == sgemm::kColAct)
        if (p.tx == 16) fn = reinterpret_cast<const void *>(&sgemm::col_kernel<KIND, 16>);
    const hipError_t e = launch1(fn, dim3((unsigned)p.wgs, (unsigned)p.chunks), 256, &a, stream);
    if (e != hipSuccess || !out || p.chunks <= 1) return e;
    return launch_col_sum(parts, p.chunks, a.N, out, stream);
}

// ---- the norm's gradient --------------------------------------------------------------------

// Workgroups of the one-pass form with a weight gradient.  Each adds up dw over
// its own rows, and its D sums are written and read once more: four rows or
// more each (times the four a workgroup of short rows holds at once) keep that
// to an eighth of the traffic, but for at least 256 workgroups where the rows
// allow, and at most 1024, which fill the chip.
long long row_grad_wgs(const RowForm &f, int rows)
{
    const long long at_once = f.nt >= 256 ? 1 : 256 / f.nt;
    const long long n = sgemm::ceil_div_ll(rows, 4 * at_once);
    return n < 256 ? 256 : n < 1024 ? n : 1024;
}

// Floats of workspace the weight gradient needs, and the parts they hold.
size_t row_grad_bytes(int rows, int D)
{
    const RowForm f = row_form(D);
    if (f.v > 0) return parts_bytes(row_grid(f, rows, row_grad_wgs(f, rows)), D);
    // r of every row (16-byte padded), then the column pass's sums
    return (((size_t)rows + 3) & ~(size_t)3) * 4u + parts_bytes(col_plan(rows, D).chunks, D);
}

hipError_t run_row_grad(int rows, int D, const float *dY, int ldy, const float *S, int lds, const float *w,
                        float eps, const float *dS, int ldds, float *dX, int lddx, float *dw, void *ws,
                        size_t ws_bytes, hipStream_t stream)
{
    if (!row_sizes_ok(rows, D, eps)) return hipErrorInvalidValue;
    if (misaligned(dw, 4)) return hipErrorInvalidValue;
    if (rows == 0) return dw ? launch_zero(dw, D, stream) : hipSuccess;
    const RowTensor y{dY, ldy, 4}, s{S, lds, 4}, g{dS, ldds, 4}, x{dX, lddx, 4};
    if (!row_tensor_ok(y, D) || !row_tensor_ok(s, D) || (dS && !row_tensor_ok(g, D)) || !row_tensor_ok(x, D) ||
        misaligned(w, 4))
        return hipErrorInvalidValue;
    const size_t need = dw ? row_grad_bytes(rows, D) : 0;
    if (need > 0 && (!ws || misaligned(ws, 16) || ws_bytes < need)) return hipErrorInvalidValue;
    const Span none{0, 0};
    const Span xs = row_span(x, rows, D), vs = w ? row_span(RowTensor{w, D, 4}, 1, D) : none;
    const Span ds = dw ? row_span(RowTensor{dw, D, 4}, 1, D) : none;
    const Span in[4] = {row_span(y, rows, D), row_span(s, rows, D), vs, dS ? row_span(g, rows, D) : none};
    const bool same = dS && same_tensor(x, g);
    if (overlaps_any(xs, in, same ? 3 : 4) || overlap(xs, ds) || overlaps_any(ds, in, 4)) return hipErrorInvalidValue;
    if (need > 0) {
        const Span u{(uintptr_t)ws, (uintptr_t)ws + need};
        if (overlaps_any(u, in, 4) || overlap(u, xs) || overlap(u, ds)) return hipErrorInvalidValue;
    }
    // Workgroups of 512 as for the forward norm, but only where no weight gradient
    // is kept in registers too (8192 x 8192: 153 to 144 us without it, 157 to 165
    // with; 4096 x 5120: 61 to 50).
    const RowForm f = !dw && rows > 512 && D > 4096 && D <= 8192 ? RowForm{512, 4} : row_form(D);
    sgemm::RowGradArgs a = {};
    a.dY = dY;
    a.S = S;
    a.w = w;
    a.dS = dS;
    a.dX = dX;
    a.ldy = ldy;
    a.lds = lds;
    a.ldds = ldds;
    a.lddx = lddx;
    a.rows = rows;
    a.D = D;
    a.eps = eps;
    const unsigned grid = row_grid(f, rows, dw && f.v > 0 ? row_grad_wgs(f, rows) : 0);
    float *fws = static_cast<float *>(ws);
    if (dw && f.v > 0) a.dw = grid > 1 ? fws : dw;
    if (dw && f.v == 0) a.inv_rms = fws;
    hipError_t e = launch1(row_grad_kernel_for(f), dim3(grid), f.nt > 256 ? f.nt : 256, &a, stream);
    if (e != hipSuccess || !dw) return e;
    if (f.v > 0) return grid > 1 ? launch_col_sum(fws, (int)grid, D, dw, stream) : hipSuccess;
    sgemm::ColArgs c = {};
    c.Y = dY;
    c.Z = S;
    c.r = fws;
    c.ldy = ldy;
    c.ldz = lds;
    c.M = rows;
    c.N = D;
    return run_cols<sgemm::kColNorm>(c, dw, fws + (((size_t)rows + 3) & ~(size_t)3), stream);
}

// ---- the elementwise gradient of a layer -----------------------------------------------------

hipError_t run_act_grad(int M, int N, int act, const float *dY, int ldy, const float *Z, int ldz, float *dZ,
                        int lddz, float *dbias, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (M < 0 || N < 0 || M > sgemm::kMaxDim || N > sgemm::kMaxDim || act < SGEMM_ACT_NONE ||
        act > SGEMM_ACT_SILU || misaligned(dbias, 4))
        return hipErrorInvalidValue;
    if (N == 0) return hipSuccess;
    if (M == 0) return dbias ? launch_zero(dbias, N, stream) : hipSuccess;
    const bool reads_z = act != SGEMM_ACT_NONE;
    const RowTensor y{dY, ldy, 4}, z{Z, ldz, 4}, o{dZ, lddz, 4};
    if (!row_tensor_ok(y, N) || (reads_z && !row_tensor_ok(z, N)) || (dZ && !row_tensor_ok(o, N)))
        return hipErrorInvalidValue;
    if (!dZ && !dbias) return hipSuccess;
    const ColPlan p = col_plan(M, N);
    const size_t need = dbias ? parts_bytes(p.chunks, N) : 0;
    if (need > 0 && (!ws || misaligned(ws, 16) || ws_bytes < need)) return hipErrorInvalidValue;
    const Span none{0, 0};
    const Span ys = row_span(y, M, N), zs = reads_z ? row_span(z, M, N) : none;
    const Span os = dZ ? row_span(o, M, N) : none, bs = dbias ? row_span(RowTensor{dbias, N, 4}, 1, N) : none;
    if ((overlap(os, ys) && !same_tensor(o, y)) || overlap(os, zs) || overlap(os, bs) || overlap(bs, ys) ||
        overlap(bs, zs))
        return hipErrorInvalidValue;
    if (need > 0) {
        const Span u{(uintptr_t)ws, (uintptr_t)ws + need};
        if (overlap(u, ys) || overlap(u, zs) || overlap(u, os) || overlap(u, bs)) return hipErrorInvalidValue;
    }
    sgemm::ColArgs a = {};
    a.Y = dY;
    a.Z = Z;
    a.out = dZ;
    a.ldy = ldy;
    a.ldz = ldz;
    a.ldo = lddz;
    a.M = M;
    a.N = N;
    a.act = act;
    return run_cols<sgemm::kColAct>(a, dbias, static_cast<float *>(ws), stream);
}
