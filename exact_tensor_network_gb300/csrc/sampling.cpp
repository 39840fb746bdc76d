// C ABI of the draws (include/tn_sampling.h): argument checks, workspace
// layout and launches.  Kernels are in sampling.cuh.  Nothing here allocates
// after tn_sampler_create, and nothing throws.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <new>

#include "sampling.h"

namespace {

using tn::Sampler;

thread_local char g_error[256] = {0};

tn_status fail(char (&buf)[256], tn_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return st;
}

tn_status cuda_fail(Sampler &s, cudaError_t e, const char *what) {
    return fail(s.error, TN_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

uint64_t align(uint64_t x) { return (x + 255) / 256 * 256; }

// Vectors of the longest row (its first may hold one entry only), and its pieces.
int64_t vectors(int32_t type, int64_t cols) {
    const int64_t E = tn::kOutVecBytes / tn::out_entry_bytes(type);
    return (cols + 2 * (E - 1)) / E;
}
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t pieces(int32_t type, int64_t cols) { return ceil_div(vectors(type, cols), tn::kPieceVecs); }

// CTAs for every SM where rows alone are too few, segments of a piece a warp at least.
int64_t segment(int64_t pieces, int64_t rows, int64_t *len) {
    int64_t want = tn::kDrawTarget / rows;
    const int64_t most = ceil_div(pieces, tn::kDrawWarps);
    if (want > most) want = most;
    if (want < 1) want = 1;
    *len = ceil_div(ceil_div(pieces, want), tn::kDrawWarps) * tn::kDrawWarps;
    return ceil_div(pieces, *len);
}

}  // namespace

extern "C" {

tn_status tn_sampler_create(int32_t type, int64_t cols, int64_t max_rows, float scale, tn_sampler_t **out) {
    if (!out) return fail(g_error, TN_EINVAL, "out is NULL");
    *out = nullptr;
    if (type < TN_TYPE_C64 || type > TN_TYPE_F16) return fail(g_error, TN_EINVAL, "unknown entry type %d", (int)type);
    if (cols < 1 || max_rows < 1) return fail(g_error, TN_EINVAL, "cols and max_rows must be >= 1");
    if (!(scale >= 0x1p-40f && scale <= 0x1p40f))
        return fail(g_error, TN_EINVAL, "scale must lie in 2^-40 .. 2^40");
    if (cols > 0x7fffffff) return fail(g_error, TN_EOVERFLOW, "more than 2^31 - 1 entries a row");
    int64_t n;
    if (__builtin_mul_overflow(max_rows, pieces(type, cols), &n) || n > (int64_t)1 << 48)
        return fail(g_error, TN_EOVERFLOW, "the workspace's size overflows");
    tn_sampler_s *h = new (std::nothrow) tn_sampler_s;
    if (!h) return fail(g_error, TN_ENOMEM, "host allocation failed");
    Sampler &s = h->s;
    s.type = type;
    s.cols = cols;
    s.max_rows = max_rows;
    s.scale = scale;
    const uint64_t at = 256;
    if (vectors(type, cols) > tn::kRowVecs) {
        // rows of several segments are at most half of kDrawTarget, their segments kDrawTarget
        const uint64_t cut = max_rows < tn::kDrawTarget / 2 ? max_rows : tn::kDrawTarget / 2;
        s.state_off = at;
        s.bins_off = align(s.state_off + static_cast<uint64_t>(max_rows) * tn::state_bytes());
        s.clear_bytes = s.partial_off = align(s.bins_off + cut * tn::bins_bytes());
        s.rest_off = align(s.partial_off + tn::kDrawTarget * sizeof(ulonglong2));
        s.list_off = align(s.rest_off + tn::kDrawTarget * sizeof(uint64_t));
        s.mass_off = align(s.list_off + cut * tn::kSorted * sizeof(uint64_t));
        s.tie_off = align(s.mass_off + static_cast<uint64_t>(n) * 8);
        s.ws_bytes = align(s.tie_off + static_cast<uint64_t>(n) * 4);
    } else {
        s.clear_bytes = s.ws_bytes = at;
    }
    g_error[0] = 0;
    *out = h;
    return TN_OK;
}

void tn_sampler_destroy(tn_sampler_t *h) { delete h; }

tn_status tn_sampler_workspace_bytes(const tn_sampler_t *h, uint64_t *bytes) {
    if (!h || !bytes) return TN_EINVAL;
    *bytes = h->s.ws_bytes;
    return TN_OK;
}

tn_status tn_sampler_set_workspace(tn_sampler_t *h, void *dev_ptr, uint64_t bytes) {
    if (!h) return TN_EINVAL;
    Sampler &s = h->s;
    if (!dev_ptr || reinterpret_cast<uintptr_t>(dev_ptr) % 256)
        return fail(s.error, TN_EINVAL, "workspace must be a non-NULL 256-byte aligned device pointer");
    if (bytes < s.ws_bytes)
        return fail(s.error, TN_ENOMEM, "workspace of %llu bytes is smaller than the %llu bytes needed",
                    (unsigned long long)bytes, (unsigned long long)s.ws_bytes);
    s.ws = nullptr;
    cudaError_t e = cudaMemset(dev_ptr, 0, s.clear_bytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(s, e, "clearing the workspace");
    s.ws = static_cast<char *>(dev_ptr);
    return TN_OK;
}

tn_status tn_sampler_draw(tn_sampler_t *h, const tn_rows *r, const tn_filters *filters, const void *u, int32_t wide,
                          int64_t draws, int64_t *ids, float *logp, int64_t *kept, tn_stream_t stream) {
    if (!h) return TN_EINVAL;
    Sampler &s = h->s;
    if (!r || (r->rows > 0 && !r->data)) return fail(s.error, TN_EINVAL, "rows and their data are required");
    if (r->rows < 0 || r->rows > s.max_rows)
        return fail(s.error, TN_EINVAL, "%lld rows: the handle was made for at most %lld", (long long)r->rows,
                    (long long)s.max_rows);
    if (reinterpret_cast<uintptr_t>(r->data) % tn::out_entry_bytes(s.type))
        return fail(s.error, TN_EINVAL, "rows are not aligned to their entry type");
    if (r->row_stride < 0 || r->col_stride < 0 || (r->col_stride == 0 && s.cols > 1))
        return fail(s.error, TN_EINVAL, "row_stride must be >= 0 and col_stride >= 1");
    if (r->mask && (r->mask_row_stride < 0 || r->mask_col_stride < 0))
        return fail(s.error, TN_EINVAL, "mask strides must be >= 0");
    if (draws < 0) return fail(s.error, TN_EINVAL, "draws must be >= 0");
    int64_t n;
    if (__builtin_mul_overflow(r->rows, draws, &n) || n > (int64_t)1 << 40)
        return fail(s.error, TN_EOVERFLOW, "more than 2^40 draws");
    if (r->rows > 0 && (!kept || (draws > 0 && (!u || !ids || !logp))))
        return fail(s.error, TN_EINVAL, "the random numbers or an output are missing");
    if (n > 0 && reinterpret_cast<uintptr_t>(u) % (wide ? 8 : 4))
        return fail(s.error, TN_EINVAL, "the random numbers are not aligned to their type");
    if (!s.ws) return fail(s.error, TN_ENOMEM, "no workspace bound (tn_sampler_set_workspace)");
    if (r->rows == 0) return TN_OK;
    tn::SampleArgs a = {};
    a.r.data = static_cast<const char *>(r->data);
    a.r.rows = r->rows;
    a.r.cols = s.cols;
    a.r.row_stride = r->row_stride;
    a.r.col_stride = s.cols == 1 ? 1 : r->col_stride;
    a.r.mask = r->mask;
    a.r.mask_row_stride = r->mask_row_stride;
    a.r.mask_col_stride = r->mask_col_stride;
    a.r.scale = s.scale;
    a.r.status = reinterpret_cast<tn::DevStatus *>(s.ws);
    if (filters) a.f = *filters;
    else a.f.temperature = a.f.top_p = 1.f;
    a.u = u;
    a.wide = wide;
    a.draws = draws;
    a.ids = ids;
    a.logp = logp;
    a.kept = kept;
    const tn_filters &f = a.f;
    a.filtered = f.top_ks || f.top_ps || f.top_k > 0 || f.top_p < 1.f;
    a.powers = f.temperatures || s.scale != f.temperature;      // (their quotient is 1 only where they are equal)
    a.pieces = pieces(s.type, s.cols);
    if (s.state_off) {
        a.segs = segment(a.pieces, r->rows, &a.seg_pieces);
        a.state = reinterpret_cast<tn::RowState *>(s.ws + s.state_off);
        a.bins = reinterpret_cast<tn::RowBins *>(s.ws + s.bins_off);
        a.partials = reinterpret_cast<ulonglong2 *>(s.ws + s.partial_off);
        a.alls = reinterpret_cast<uint64_t *>(s.ws + s.rest_off);
        a.lists = reinterpret_cast<uint64_t *>(s.ws + s.list_off);
        a.masses = reinterpret_cast<uint64_t *>(s.ws + s.mass_off);
        a.ties = reinterpret_cast<uint32_t *>(s.ws + s.tie_off);
    }
    if (r->rows * (a.segs + ceil_div(draws, tn::kDrawWarps)) > 0x7fffffff)
        return fail(s.error, TN_EOVERFLOW, "too many draws or rows for one call");
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (s.type) {
        case TN_TYPE_C64: e = tn::sample_of<TN_TYPE_C64>(a, st); break;
        case TN_TYPE_F32: e = tn::sample_of<TN_TYPE_F32>(a, st); break;
        case TN_TYPE_BF16: e = tn::sample_of<TN_TYPE_BF16>(a, st); break;
        default: e = tn::sample_of<TN_TYPE_F16>(a, st); break;
    }
    return e == cudaSuccess ? TN_OK : cuda_fail(s, e, "launching the draws");
}

tn_status tn_sampler_check(tn_sampler_t *h) {
    if (!h) return TN_EINVAL;
    Sampler &s = h->s;
    if (!s.ws) return TN_OK;
    tn::DevStatus d{0, 0};
    cudaError_t e = cudaMemcpy(&d, s.ws, sizeof(d), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(s, e, "reading the status word");
    if (d.code == tn::ERR_NONE) return TN_OK;
    e = cudaMemset(s.ws, 0, sizeof(d));
    if (e != cudaSuccess) return cuda_fail(s, e, "clearing the status word");
    return fail(s.error, TN_EDEVICE, "an invalid parameter or random number in row %d", (int)d.where);
}

const char *tn_sampler_last_error(const tn_sampler_t *h) { return h ? h->s.error : g_error; }

}  // extern "C"
