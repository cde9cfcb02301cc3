// Host side of the layer norm (layernorm.hpp): argument checks, the choice of
// a form and the launches.  Included by sgemm.hip inside its anonymous
// namespace, after rowops_host.hpp.

// Memory that one call reads or writes.
struct Piece {
    RowTensor t;
    int rows, cols;
};

// Whether two tensors share memory.  Tensors with the same row stride whose
// spans overlap may still be apart, column ranges of one matrix (the two
// halves of a gated layer's weights, gradients or pre-activations).
bool pieces_overlap(const Piece &a, const Piece &b)
{
    if (!a.t.ptr || !b.t.ptr || a.rows <= 0 || b.rows <= 0 || a.cols <= 0 || b.cols <= 0) return false;
    const Span as = row_span(a.t, a.rows, a.cols), bs = row_span(b.t, b.rows, b.cols);
    if (!overlap(as, bs)) return false;
    if (a.t.size != b.t.size || a.t.ld != b.t.ld) return true;
    const uint64_t row = (uint64_t)a.t.ld * (uint64_t)a.t.size;
    const uint64_t off = as.lo >= bs.lo ? (as.lo - bs.lo) % row : (row - (bs.lo - as.lo) % row) % row;
    return off < (uint64_t)b.cols * b.t.size || off + (uint64_t)a.cols * a.t.size > row;
}

// Whether an output shares memory with any of the others.
bool pieces_overlap_any(const Piece &a, const Piece *others, int n)
{
    for (int i = 0; i < n; ++i)
        if (pieces_overlap(a, others[i])) return true;
    return false;
}

// The forms of a layer norm to 8 bits are row_form's: it holds w and b in
// registers too, so workgroups of 512 for long rows would hold 32 values a thread
// and be one to a compute unit as those of 1024 are (8192 x 8192 with residual:
// 204 us against 180).
RowForm layernorm_form(bool q8, int D, int rows, bool residual)
{
    return q8 ? row_form(D) : row_form_forward(D, rows, residual);
}

// Workgroups of a layer norm: to 8 bits as many as share the chip, which then
// loop over the rows with w and b in their registers (microseconds with
// residual, so many and one a row: 8192 x 4096 80 and 118, 8192 x 8192 180 and 202,
// 4096 x 16384 204 and 239).
long long layernorm_wgs(bool q8, const RowForm &f)
{
    if (!q8 || f.v == 0) return 0;
    if (f.nt == 1024) return f.v == 2 ? 512 : 256;
    return f.v == 4 ? 768 : 2048;
}

template <bool Q8> const void *layernorm_kernel_for(const RowForm &f)
{
    using sgemm::layernorm_kernel;
    if (f.nt == 64) {
        if (f.v == 1) return reinterpret_cast<const void *>(&layernorm_kernel<64, 1, Q8>);
        if (f.v == 2) return reinterpret_cast<const void *>(&layernorm_kernel<64, 2, Q8>);
        return reinterpret_cast<const void *>(&layernorm_kernel<64, 4, Q8>);
    }
    if (f.nt == 256) {
        if (f.v == 2) return reinterpret_cast<const void *>(&layernorm_kernel<256, 2, Q8>);
        return reinterpret_cast<const void *>(&layernorm_kernel<256, 4, Q8>);
    }
    if constexpr (!Q8)
        if (f.nt == 512) {
            if (f.v == 4) return reinterpret_cast<const void *>(&layernorm_kernel<512, 4, Q8>);
            return reinterpret_cast<const void *>(&layernorm_kernel<512, 8, Q8>);
        }
    if (f.v == 2) return reinterpret_cast<const void *>(&layernorm_kernel<1024, 2, Q8>);
    if (f.v == 4) return reinterpret_cast<const void *>(&layernorm_kernel<1024, 4, Q8>);
    return reinterpret_cast<const void *>(&layernorm_kernel<1024, 0, Q8>);
}

const void *layernorm_grad_kernel_for(const RowForm &f)
{
    using sgemm::layernorm_grad_kernel;
    if (f.nt == 64) {
        if (f.v == 1) return reinterpret_cast<const void *>(&layernorm_grad_kernel<64, 1>);
        if (f.v == 2) return reinterpret_cast<const void *>(&layernorm_grad_kernel<64, 2>);
        return reinterpret_cast<const void *>(&layernorm_grad_kernel<64, 4>);
    }
    if (f.nt == 256) {
        if (f.v == 2) return reinterpret_cast<const void *>(&layernorm_grad_kernel<256, 2>);
        return reinterpret_cast<const void *>(&layernorm_grad_kernel<256, 4>);
    }
    if (f.nt == 512) return reinterpret_cast<const void *>(&layernorm_grad_kernel<512, 4>);
    if (f.v == 2) return reinterpret_cast<const void *>(&layernorm_grad_kernel<1024, 2>);
    if (f.v == 4) return reinterpret_cast<const void *>(&layernorm_grad_kernel<1024, 4>);
    return reinterpret_cast<const void *>(&layernorm_grad_kernel<1024, 0>);
}

// A layer norm; q8: to codes.
hipError_t run_layernorm(bool q8, int rows, int D, const float *X, int ldx, const float *R, int ldr, const float *w,
                         const float *b, float eps, float *S, int lds, float *Y, int ldy, void *Q, int ldq,
                         float *scale, hipStream_t stream)
{
    if (!row_sizes_ok(rows, D, eps)) return hipErrorInvalidValue;
    if (rows == 0) return hipSuccess;
    const RowTensor x{X, ldx, 4}, r{R, ldr, 4}, s{S, lds, 4};
    const RowTensor y = q8 ? RowTensor{Q, ldq, 1} : RowTensor{Y, ldy, 4};
    if (!row_tensor_ok(x, D) || (R && !row_tensor_ok(r, D)) || (S && !row_tensor_ok(s, D)) ||
        !row_tensor_ok(y, D) || misaligned(w, 4) || misaligned(b, 4))
        return hipErrorInvalidValue;
    if (q8 && (!scale || misaligned(scale, 4))) return hipErrorInvalidValue;
    const Piece px{x, rows, D}, pr{r, rows, D}, ps{s, rows, D}, py{y, rows, D}, pw{RowTensor{w, D, 4}, 1, D},
        pb{RowTensor{b, D, 4}, 1, D}, pc{RowTensor{q8 ? scale : nullptr, rows, 4}, 1, rows};
    // outputs: S, Y or Q, scale.  (Codes are of another size: none keeps an
    // input's place.)
    const Piece fixed[3] = {pw, pb, pc};
    if (pieces_overlap_any(py, fixed, 3) || pieces_overlap_any(ps, fixed, 3) || pieces_overlap(ps, py) ||
        (pieces_overlap(py, px) && (q8 || !same_tensor(x, y))) ||
        (pieces_overlap(py, pr) && (q8 || !same_tensor(r, y))) || (pieces_overlap(ps, px) && !same_tensor(s, x)) ||
        (pieces_overlap(ps, pr) && !same_tensor(s, r)))
        return hipErrorInvalidValue;
    const Piece in[4] = {px, pr, pw, pb};
    if (pieces_overlap_any(pc, in, 4)) return hipErrorInvalidValue;
    sgemm::LnArgs a = {};
    a.X = X;
    a.R = R;
    a.w = w;
    a.b = b;
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
    const RowForm f = layernorm_form(q8, D, rows, R != nullptr);
    return launch1(q8 ? layernorm_kernel_for<true>(f) : layernorm_kernel_for<false>(f),
                   dim3(row_grid(f, rows, layernorm_wgs(q8, f))), f.nt > 256 ? f.nt : 256, &a, stream);
}

// ---- gradient --------------------------------------------------------------------------

// The sum of `parts` rows of 2 N partial sums to two vectors (either may be null).
hipError_t launch_pair_sum(const float *part, int parts, int N, float *first, float *second, hipStream_t stream)
{
    // (blocks of 32 columns; the dispatch packet counts work-items in 32 bits)
    const long long blocks = sgemm::ceil_div_ll(2ll * N, 32), per = max_wgs_per_launch(sgemm::kColSumThreads);
    for (long long b0 = 0; b0 < blocks; b0 += per) {
        const long long n = blocks - b0 < per ? blocks - b0 : per;
        int64_t base = 32 * (int64_t)b0;
        void *list[] = {&part, &parts, &N, &base, &first, &second};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&sgemm::pair_sum_kernel),
                                             dim3((unsigned)n), dim3(sgemm::kColSumThreads), list, 0, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Bytes of every row's mean and r (16-byte padded), for the column pass of long rows.
size_t layernorm_rows_bytes(int rows) { return ((size_t)rows * sizeof(sgemm::LnRow) + 15) & ~(size_t)15; }

// Workgroups of the one-pass form with sums: four rows or more each, as for the RMS
// norm's gradient, but at least 512 where there are so many rows, and at most as
// many as share the chip, since each writes 2 D sums (microseconds, without their
// sum: 8192 x 4096 with 768 and 1024 workgroups 100 and 105, 8192 x 8192 with
// 256 and 1024 143 and 155, 515 x 2052 with 256 and 515 9.8 and 7.6).  With their sum
// a row each past 512 workgroups costs more than the second row that some of 512
// take: calls of 600 x 2051 16.3 and 15.8, 768 x 4096 19.3 and 17.2, 1000 x 2051
// 19.3 and 16.4, 515 x 2051 the same.
long long layernorm_grad_wgs(const RowForm &f, int rows)
{
    const long long at_once = f.nt >= 256 ? 1 : 256 / f.nt;
    const long long n = sgemm::ceil_div_ll(rows, 4 * at_once), most = f.nt == 1024 ? 256 : f.v == 4 ? 768 : 1024;
    const long long least = most < 512 ? most : 512;
    return n < least ? least : n < most ? n : most;
}

// Workspace of the sums: each workgroup's (or chunk's) 2 D partial ones.
size_t layernorm_grad_bytes(int rows, int D)
{
    const RowForm f = row_form(D);
    if (f.v > 0) return (size_t)row_grid(f, rows, layernorm_grad_wgs(f, rows)) * 8u * (size_t)D;
    return layernorm_rows_bytes(rows) + (size_t)col_plan(rows, D).chunks * 8u * (size_t)D;
}

hipError_t run_layernorm_grad(int rows, int D, const float *dY, int ldy, const float *S, int lds, const float *w,
                              float eps, const float *dS, int ldds, float *dX, int lddx, float *dw, float *db,
                              void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!row_sizes_ok(rows, D, eps)) return hipErrorInvalidValue;
    if (misaligned(dw, 4) || misaligned(db, 4)) return hipErrorInvalidValue;
    const Piece pdw{RowTensor{dw, D, 4}, 1, D}, pdb{RowTensor{db, D, 4}, 1, D};
    if (pieces_overlap(pdw, pdb)) return hipErrorInvalidValue;
    if (rows == 0) {
        const hipError_t e = dw ? launch_zero(dw, D, stream) : hipSuccess;
        return e == hipSuccess && db ? launch_zero(db, D, stream) : e;
    }
    const RowTensor y{dY, ldy, 4}, s{S, lds, 4}, g{dS, ldds, 4}, x{dX, lddx, 4};
    if (!row_tensor_ok(y, D) || !row_tensor_ok(s, D) || (dS && !row_tensor_ok(g, D)) || !row_tensor_ok(x, D) ||
        misaligned(w, 4))
        return hipErrorInvalidValue;
    const bool sums = dw || db;
    const size_t need = sums ? layernorm_grad_bytes(rows, D) : 0;
    if (need > 0 && (!ws || misaligned(ws, 16) || ws_bytes < need)) return hipErrorInvalidValue;
    const Piece px{x, rows, D};
    // dX may be dS's own memory
    const Piece in[4] = {Piece{y, rows, D}, Piece{s, rows, D}, Piece{RowTensor{w, D, 4}, 1, D}, Piece{g, rows, D}};
    if (pieces_overlap_any(px, in, dS && same_tensor(x, g) ? 3 : 4) || pieces_overlap(px, pdw) ||
        pieces_overlap(px, pdb) || pieces_overlap_any(pdw, in, 4) || pieces_overlap_any(pdb, in, 4))
        return hipErrorInvalidValue;
    if (need > 0) {
        const Span u{(uintptr_t)ws, (uintptr_t)ws + need};
        const Piece all[7] = {in[0], in[1], in[2], in[3], px, pdw, pdb};
        for (const Piece &p : all)
            if (p.t.ptr && overlap(u, row_span(p.t, p.rows, p.cols))) return hipErrorInvalidValue;
    }
    const RowForm f = !sums && rows > 512 && D > 4096 && D <= 8192 ? RowForm{512, 4} : row_form(D);
    sgemm::LnGradArgs a = {};
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
    const unsigned grid = row_grid(f, rows, sums && f.v > 0 ? layernorm_grad_wgs(f, rows) : 0);
    char *const at = static_cast<char *>(ws);
    if (sums && f.v > 0) a.part = reinterpret_cast<float *>(at);
    if (sums && f.v == 0) a.rows3 = reinterpret_cast<sgemm::LnRow *>(at);
    hipError_t e = launch1(layernorm_grad_kernel_for(f), dim3(grid), f.nt > 256 ? f.nt : 256, &a, stream);
    if (e != hipSuccess || !sums) return e;
    if (f.v > 0) return launch_pair_sum(a.part, (int)grid, D, dw, db, stream);
    const ColPlan p = col_plan(rows, D);
    sgemm::LnColArgs c = {};
    c.dY = dY;
    c.S = S;
    c.rows3 = a.rows3;
    c.part = reinterpret_cast<float *>(at + layernorm_rows_bytes(rows));
    c.ldy = ldy;
    c.lds = lds;
    c.M = rows;
    c.N = D;
    c.rows_per_chunk = p.rows_per_chunk;
    e = launch1(reinterpret_cast<const void *>(&sgemm::layernorm_col_kernel),
                dim3((unsigned)p.wgs, (unsigned)p.chunks), 256, &c, stream);
    return e == hipSuccess ? launch_pair_sum(c.part, p.chunks, D, dw, db, stream) : e;
}
