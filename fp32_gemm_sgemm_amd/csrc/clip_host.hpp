// Host side of clip.hpp: argument checks and launches.  Included by sgemm.hip
// inside its anonymous namespace, after layernorm_host.hpp.

// Chunks that one workgroup does alone in one launch (16384 elements).  Above,
// two launches are quicker.
constexpr int kClipOneChunks = 4;
static_assert(kClipOneChunks <= sgemm::kClipInline, "their table travels with the launch");

struct ClipKernels {
    const void *norm, *scale;
};
template <bool HERE, bool WRITE> ClipKernels clip_kernels()
{
    return {reinterpret_cast<const void *>(&sgemm::clip_norm_kernel<HERE>),
            reinterpret_cast<const void *>(&sgemm::clip_scale_kernel<HERE, WRITE>)};
}
// by where the table is (the launch's arguments, memory) and whether y is written
const ClipKernels kClipKernels[2][2] = {{clip_kernels<true, false>(), clip_kernels<true, true>()},
                                        {clip_kernels<false, false>(), clip_kernels<false, true>()}};
const void *const kClipOne[2] = {reinterpret_cast<const void *>(&sgemm::clip_one_kernel<false>),
                                 reinterpret_cast<const void *>(&sgemm::clip_one_kernel<true>)};

size_t clip_table_bytes(int count)
{
    return count > sgemm::kClipInline ? ((size_t)count * sizeof(sgemm::ClipTensor) + 15) & ~(size_t)15 : 0;
}
size_t clip_bytes(int count) { return clip_table_bytes(count) + sgemm::kClipMaxWgs * sizeof(double); }

// Memory of one tensor in a call, with what it belongs to.
struct ClipPiece {
    uintptr_t lo, hi;
    uint64_t ld, cols;  // bytes
    bool written;
    int id;
};

// Whether two pieces whose spans overlap share memory (as pieces_overlap).
bool clip_pieces_meet(const ClipPiece &a, const ClipPiece &b)
{
    if (a.ld != b.ld) return true;
    const uint64_t off = a.lo >= b.lo ? (a.lo - b.lo) % a.ld : (a.ld - (b.lo - a.lo) % a.ld) % a.ld;
    return off < b.cols || off + a.cols > a.ld;
}

// Whether what one tensor writes is read or written through another one, or
// covers the `others` (the norm, the workspace); pieces in order of address.
// A tensor's own input and output may be the same memory.
bool clip_overlaps(std::vector<ClipPiece> &v)
{
    std::sort(v.begin(), v.end(), [](const ClipPiece &a, const ClipPiece &b) { return a.lo < b.lo; });
    std::vector<const ClipPiece *> open;  // pieces that may reach past the next one's start
    for (const ClipPiece &p : v) {
        size_t keep = 0;
        for (const ClipPiece *q : open) {
            if (q->hi <= p.lo) continue;
            open[keep++] = q;
            if ((p.written || q->written) && !(p.id == q->id && p.lo == q->lo && p.ld == q->ld) &&
                clip_pieces_meet(*q, p))
                return true;
        }
        open.resize(keep);
        open.push_back(&p);
    }
    return false;
}

// write: y = c x too.
hipError_t run_clip(bool write, int count, const sgemm_tensor *tensors, float max_norm, float eps, float *norm,
                    void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (count < 0 || (count > 0 && !tensors) || misaligned(norm, 4)) return hipErrorInvalidValue;
    if (!(max_norm >= 0.0f && max_norm <= 3.4028235e38f) || !(eps >= 0.0f && eps <= 3.4028235e38f))
        return hipErrorInvalidValue;
    if (!write && !norm) return hipErrorInvalidValue;
    const size_t need = clip_bytes(count);
    if (!ws || misaligned(ws, 16) || ws_bytes < need) return hipErrorInvalidValue;
    // (no allocation failure may leave a C entry as an exception)
    try {
        std::vector<sgemm::ClipTensor> table;
        std::vector<ClipPiece> pieces;
        table.reserve((size_t)count);
        pieces.reserve(2 * (size_t)count + 2);
        long long chunks = 0;
        bool in_place = true;
        for (int i = 0; i < count; ++i) {
            const sgemm_tensor &t = tensors[i];
            if (t.rows < 0 || t.cols < 0) return hipErrorInvalidValue;
            if (t.rows == 0 || t.cols == 0) continue;
            const bool one = t.rows == 1;
            if (t.rows > sgemm::kMaxDim || t.cols > (one ? 1ll << 40 : (long long)sgemm::kMaxDim) || !t.x ||
                misaligned(t.x, 4) || (!one && (t.ldx < t.cols || t.ldx > sgemm::kMaxDim)))
                return hipErrorInvalidValue;
            if (write && (!t.y || misaligned(t.y, 4) || (!one && (t.ldy < t.cols || t.ldy > sgemm::kMaxDim))))
                return hipErrorInvalidValue;
            sgemm::ClipTensor e;
            e.x = t.x;
            e.y = write ? t.y : nullptr;
            e.rows = (int)t.rows;
            e.cols = t.cols;
            e.ldx = one ? 0 : (int)t.ldx;
            e.ldy = one || !write ? 0 : (int)t.ldy;
            const uint64_t width = (uint64_t)t.cols * 4;
            auto piece = [&](const float *p, int ld, bool written) {
                const uint64_t step = one ? width : (uint64_t)ld * 4;
                const uintptr_t lo = (uintptr_t)p;
                pieces.push_back({lo, lo + (uint64_t)(t.rows - 1) * step + width, step, width, written, i});
            };
            if (write) {
                piece(t.x, e.ldx, false);
                piece(t.y, e.ldy, true);
                in_place = in_place && t.y == t.x && e.ldx == e.ldy;
            }
            // rows without a gap are one row
            if (!one && e.ldx == t.cols && (!write || e.ldy == t.cols)) {
                e.cols = t.rows * t.cols;
                e.rows = 1;
            }
            if (chunks > INT_MAX) return hipErrorInvalidValue;
            e.first = (int)chunks;
            const long long rpc = sgemm::clip_rows(e.cols);
            chunks += rpc > 1 ? (e.rows + rpc - 1) / rpc : e.rows * sgemm::clip_row_chunks(e.cols);
            table.push_back(e);
        }
        if (chunks > INT_MAX) return hipErrorInvalidValue;
        const int outside = -1;
        if (norm) pieces.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, 4, 4, true, outside});
        pieces.push_back({(uintptr_t)ws, (uintptr_t)ws + need, need, need, true, outside});
        if (!write)
            for (const sgemm::ClipTensor &e : table) {
                const uint64_t width = (uint64_t)e.cols * 4, step = e.rows == 1 ? width : (uint64_t)e.ldx * 4;
                const uintptr_t lo = (uintptr_t)e.x;
                pieces.push_back({lo, lo + (uint64_t)(e.rows - 1) * step + width, step, width, false, 0});
            }
        if (clip_overlaps(pieces)) return hipErrorInvalidValue;

        sgemm::ClipArgs a = {};
        const int n = (int)table.size();
        a.norm = norm;
        a.max_norm = max_norm;
        a.eps = eps;
        a.chunks = (int)chunks;
        a.in_place = in_place ? 1 : 0;
        a.part = reinterpret_cast<double *>(static_cast<char *>(ws) + clip_table_bytes(count));
        if (n > sgemm::kClipInline) {
            sgemm::ClipTensor *to = static_cast<sgemm::ClipTensor *>(ws);
            for (int i0 = 0; i0 < n; i0 += sgemm::kClipInline) {
                a.count = n - i0 < sgemm::kClipInline ? n - i0 : sgemm::kClipInline;
                for (int i = 0; i < a.count; ++i) a.here[i] = table[(size_t)(i0 + i)];
                sgemm::ClipTensor *at = to + i0;
                void *list[] = {&a, &at};
                const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&sgemm::clip_table_kernel), dim3(1),
                                                     dim3(128), list, 0, stream);
                if (e != hipSuccess) return e;
            }
            a.table = to;
        } else {
            for (int i = 0; i < n; ++i) a.here[i] = table[(size_t)i];
        }
        a.count = n;
        if (chunks <= kClipOneChunks) return launch1(kClipOne[write ? 1 : 0], dim3(1), sgemm::kClipOneThreads, &a, stream);
        const ClipKernels &k = kClipKernels[a.table ? 1 : 0][write ? 1 : 0];
        a.parts = chunks < sgemm::kClipMaxWgs ? (int)chunks : sgemm::kClipMaxWgs;
        const hipError_t e = launch1(k.norm, dim3((unsigned)a.parts), sgemm::kClipThreads, &a, stream);
        if (e != hipSuccess) return e;
        return launch1(k.scale, dim3(write ? (unsigned)a.parts : 1u), sgemm::kClipThreads, &a, stream);
    } catch (const std::bad_alloc &) {
        return hipErrorOutOfMemory;
    }
}
