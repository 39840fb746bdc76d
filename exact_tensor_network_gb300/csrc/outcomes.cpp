// C ABI of the operators on outcome distributions (include/tn_outcomes.h):
// argument checks, workspace layout and launches.  Kernels are in
// k_outcomes*.cu.  Nothing here allocates after tn_outcomes_create, and
// nothing throws.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "outcomes.h"

namespace tn {

OutSplit out_split(int32_t type, int64_t cols, int64_t rows, bool aligned, int64_t warp_vecs) {
    const int64_t E = kOutVecBytes / out_entry_bytes(type);
    OutSplit s;
    s.vecs = (cols + E - 1 + (aligned ? 0 : E - 1)) / E;   // its first may hold one entry only
    s.warp_rows = s.vecs <= warp_vecs;
    s.segs = 1;
    s.seg_vecs = s.vecs;
    if (s.warp_rows) return s;
    // One wave of CTAs where whole segments fill five sixths of it, else up to two
    // (64x131072 bf16 one 8.0 us, half of one 10.1, two 8.2, four 10.1; 700x50001
    // bf16 one, 58 % full, 22.7, two 16.7; 1024x50001 amplitudes one, 84 % full, 67,
    // two 71).  A CTA of less than two vectors a thread gains nothing.
    const int64_t target = kOutTarget;
    int64_t want = rows >= target ? 1 : target / rows;
    if (rows < target && rows * want * 6 < target * 5) want = 2 * target / rows;
    const int64_t most = (s.vecs + 2 * kOutThreads - 1) / (2 * kOutThreads);
    if (want > most) want = most;
    const int64_t least = (s.vecs + kOutSegVecs - 1) / kOutSegVecs;
    if (want < least) want = least;
    int64_t sv = (s.vecs + want - 1) / want;
    if (want > 1) sv = (sv + kOutThreads - 1) / kOutThreads * kOutThreads;
    if (sv > kOutSegVecs) sv = kOutSegVecs;
    s.seg_vecs = sv;
    s.segs = (s.vecs + sv - 1) / sv;
    return s;
}

}  // namespace tn

namespace {

using tn::Outcomes;

thread_local char g_error[256] = {0};

tn_status fail(char (&buf)[256], tn_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return st;
}

tn_status cuda_fail(Outcomes &o, cudaError_t e, const char *what) {
    return fail(o.error, TN_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Rows of how many vectors are one warp's.  Short ones always are: a CTA would
// have less than two vectors a thread.  Longer ones cost fewer instructions as
// a warp's (what a row costs besides its vectors is paid once, not once for
// each of four or eight warps), if there are rows enough for all warps.
// Measured, CTA against warp a row: scores of 20000 rows of 6 KB 44 against
// 28 us (with five alternatives 92 against 61), of 10 KB 58 against 41, of 10000
// rows of 16 KB 35 against 32 (66 against 53), but of 1300 rows 6.2 against 7.6 (15.5
// against 15.6), of 10000 rows of 24 KB 45 against 44; gradients of 20000 rows of 6 KB 65 against 45 us, of
// 10 KB 85 against 70, but of 10000 rows of 16 KB 56 against 59 and of 2500
// rows 10.9 against 15.5; training steps of 20000 rows of 4 KB 173 against 41 us,
// of 8 KB 181 against 64, of 10000 rows of 16 KB 101 against 73, but of 100
// rows of 16 KB 5.5 against 7.7 and of 10000 rows of 32 KB 132 against 218.
// None of these is below the limit that the workspace is made for.
int64_t warp_vecs(int64_t rows) { return rows > 2 * tn::kOutTarget ? 1024 : tn::kOutWarpVecs; }
int64_t grad_warp_vecs(int64_t rows) { return rows > 4 * tn::kOutTarget ? 640 : tn::kOutWarpVecs; }
int64_t step_warp_vecs(int64_t rows) { return rows > 3 * tn::kOutSms ? 1024 : tn::kOutWarpVecs; }

bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

// How the maxima of k alternatives lie.  Chunks are as large as leaves twice as
// many of them as alternatives (a cut well inside) and at most 1024 vectors to
// read again (4096 for the larger groups that few rows have), but no more of
// them in a segment than kOutKeys.  32 vectors, a warp's load, are the last that
// one reduction finds the largest of; they stay for up to three tenths of a row
// to read again.  Measured, chunks of 64, 32, 16, 8, 4 vectors: 2048x50001 bf16
// with 20 alternatives 73, 65, 86, 84, 84 us, with 128 (three quarters of a row's
// vectors read again at 32) 3285, 253, 125, 113, 109; 300x65536 f32 with 64 28.5,
// 27.7, 31.6, 30.3, 46.2; 32, 16, 8 vectors: 400x65536 f32 with 64 35, 38, 51,
// 2000x30001 with 64 (31 % of a row at 32) 100, 97, 92.
struct Chunks {
    int log;
    int64_t seg_chunks;     // of a segment
    bool tree;
};

Chunks chunks_of(const tn::OutSplit &s, int64_t rows, int64_t k) {
    Chunks c;
    const int64_t again = rows >= tn::kOutTarget / 4 ? 1024 : 4096;
    if (s.warp_rows) {      // what a warp has registers for
        c.log = 0;
        while ((s.vecs + (1 << c.log) - 1) >> c.log > tn::kOutWarpVecs) ++c.log;
        c.seg_chunks = (s.vecs + (1 << c.log) - 1) >> c.log;
        c.tree = false;
        return c;
    }
    c.log = tn::kOutChunkLog;
    while (c.log > 0 && s.seg_vecs <= (int64_t)tn::kOutKeys << (c.log - 1)) {
        const int64_t most = (int64_t)tn::out_most((int)k) << c.log;
        if (s.vecs >> c.log >= 2 * k && (most <= again || (c.log == 5 && most * 10 <= s.vecs * 3))) break;
        --c.log;
    }
    c.seg_chunks = (s.seg_vecs + (1 << c.log) - 1) >> c.log;
    c.tree = c.seg_chunks * s.segs > tn::kOutTree;
    return c;
}

// What calls of up to max_rows rows need at most: segments, and maxima.
struct Need {
    uint64_t slots = 0, maxima = 0, supers = 0;
};

void add_need(const Outcomes &o, int64_t rows, bool aligned, Need *n) {
    const tn::OutSplit s = tn::out_split(o.type, o.cols, rows, aligned, tn::kOutWarpVecs);
    if (s.warp_rows || (s.segs == 1 && o.max_top == 0)) return;
    const uint64_t slots = (uint64_t)rows * s.segs;
    if (slots > n->slots) n->slots = slots;
    // fewer alternatives have larger chunks
    for (int k = 1; k <= o.max_top; k *= 2) {
        const Chunks c = chunks_of(s, rows, k * 2 > o.max_top ? o.max_top : k);
        if (slots * c.seg_chunks > n->maxima) n->maxima = slots * c.seg_chunks;
        if (c.tree && slots * 33 > n->supers) n->supers = slots * 33;
    }
}

Need workspace_need(const Outcomes &o) {
    Need n;
    // the number of segments a row falls to its lowest value once the rows
    // alone fill the GPU
    const int64_t last = o.max_rows < tn::kOutTarget ? o.max_rows : tn::kOutTarget;
    for (int aligned = 0; aligned < 2; ++aligned) {
        for (int64_t r = 1; r <= last; ++r) add_need(o, r, aligned, &n);
        add_need(o, o.max_rows, aligned, &n);
    }
    return n;
}

uint64_t align(uint64_t x) { return (x + 255) / 256 * 256; }

// Whether every row starts at a 16-byte boundary (strided rows have no
// vectors that could be cut short).
bool aligned(const Outcomes &o, const tn_rows *r) {
    const int64_t size = tn::out_entry_bytes(o.type);
    if (r->col_stride != 1 && o.cols > 1) return true;
    return reinterpret_cast<uintptr_t>(r->data) % tn::kOutVecBytes == 0 &&
           (r->rows == 1 || r->row_stride * size % tn::kOutVecBytes == 0);
}

// Checks of the rows and the arguments that every call shares.
tn_status common(Outcomes &o, const tn_rows *r) {
    if (!r || (r->rows > 0 && !r->data)) return fail(o.error, TN_EINVAL, "rows and their data are required");
    if (r->rows < 0 || r->rows > o.max_rows)
        return fail(o.error, TN_EINVAL, "%lld rows: the handle was made for at most %lld",
                    (long long)r->rows, (long long)o.max_rows);
    if (reinterpret_cast<uintptr_t>(r->data) % tn::out_entry_bytes(o.type))
        return fail(o.error, TN_EINVAL, "rows are not aligned to their entry type");
    if (r->row_stride < 0 || r->col_stride < 0 || (r->col_stride == 0 && o.cols > 1))
        return fail(o.error, TN_EINVAL, "row_stride must be >= 0 and col_stride >= 1");
    if (r->mask && (r->mask_row_stride < 0 || r->mask_col_stride < 0))
        return fail(o.error, TN_EINVAL, "mask strides must be >= 0");
    if (!o.ws) return fail(o.error, TN_ENOMEM, "no workspace bound (tn_outcomes_set_workspace)");
    return TN_OK;
}

tn_status check_teacher(Outcomes &o, const tn_rows *r, const tn_teacher *t) {
    if (!t || (r->rows > 0 && (!t->ids || !t->logits)))
        return fail(o.error, TN_EINVAL, "the teacher's ids and logits are required");
    if (t->count < 1 || t->count > TN_OUTCOMES_MAX_IDS)
        return fail(o.error, TN_EINVAL, "teacher count %d outside 1 .. %d", (int)t->count,
                    (int)TN_OUTCOMES_MAX_IDS);
    if (t->type != TN_TYPE_F32 && t->type != TN_TYPE_BF16 && t->type != TN_TYPE_F16)
        return fail(o.error, TN_EINVAL, "the teacher's logits must be f32, bf16 or f16");
    if (!(t->scale > 0.f) || std::isinf(t->scale))
        return fail(o.error, TN_EINVAL, "the teacher's scale must be finite and > 0");
    return TN_OK;
}

tn_status check_grad(Outcomes &o, const tn_rows *r, const void *grad, int64_t rs, int64_t cs) {
    if (r->rows > 0 && !grad) return fail(o.error, TN_EINVAL, "grad is required");
    if (reinterpret_cast<uintptr_t>(grad) % tn::out_entry_bytes(o.type))
        return fail(o.error, TN_EINVAL, "grad is not aligned to its entry type");
    if (rs < 0 || cs < 0 || (cs == 0 && o.cols > 1) || (rs == 0 && r->rows > 1))
        return fail(o.error, TN_EINVAL, "grad strides must be >= 1");
    return TN_OK;
}

tn::OutRows rows_of(const Outcomes &o, const tn_rows *r, const tn::OutSplit &s) {
    tn::OutRows a = {};
    a.data = static_cast<const char *>(r->data);
    a.rows = r->rows;
    a.cols = o.cols;
    a.row_stride = r->row_stride;
    a.col_stride = o.cols == 1 ? 1 : r->col_stride;
    a.mask = r->mask;
    a.mask_row_stride = r->mask_row_stride;
    a.mask_col_stride = r->mask_col_stride;
    a.scale = o.scale;
    a.c2 = o.type == TN_TYPE_C64 ? o.scale : static_cast<float>(o.scale * 1.4426950408889634);
    int x;
    std::frexp(a.c2, &x);                       // c2 <= 2^x
    a.floor = -std::ldexp(1.f, x > 0 ? 126 - x : 126);   // a bf16 number as well
    a.lag = a.c2 <= 0.25f ? 0x1p127f : a.c2 <= 1.f ? 256.f : std::exp2(8.f / a.c2);
    a.seg_vecs = s.seg_vecs;
    a.segs = s.segs;
    a.status = reinterpret_cast<tn::DevStatus *>(o.ws);
    return a;
}

tn::OutTeacher teacher_of(const tn_teacher *t) {
    return tn::OutTeacher{t->ids, t->logits, t->type, t->count, t->scale};
}

// The kernel of the rows' type.
template <class Args, class C64, class F32, class BF16, class F16>
cudaError_t by_type(int32_t type, C64 c64, F32 f32, BF16 bf16, F16 f16, const Args &a, bool warp_rows,
                    cudaStream_t stream) {
    switch (type) {
        case TN_TYPE_C64: return c64(a, warp_rows, stream);
        case TN_TYPE_F32: return f32(a, warp_rows, stream);
        case TN_TYPE_BF16: return bf16(a, warp_rows, stream);
        default: return f16(a, warp_rows, stream);
    }
}

tn_status forward(Outcomes &o, tn::OutForward &a, const tn::OutSplit &s, cudaStream_t stream) {
    const int64_t k = a.n_top;
    a.finish = !s.warp_rows && (s.segs > 1 || k > 0);
    if (k > 0) {
        const Chunks c = chunks_of(s, a.r.rows, k);
        a.chunk_log = c.log;
        a.seg_chunks = static_cast<int32_t>(c.seg_chunks);
        a.tree = c.tree;
        int64_t words = c.seg_chunks * s.segs;
        if (c.tree) words = tn::kOutTree;
        words = (words + 3) / 4 * 4;
        // room for the entries of k vectors; as words, for the maxima of k
        // chunks' vectors and the 256 bins of the cut
        int64_t cand = 8 * k;
        if (cand < (k << c.log) / 2) cand = (k << c.log) / 2;
        if (cand < 128) cand = 128;
        cand = (cand + 1) / 2 * 2;
        a.key_words = static_cast<int32_t>(words);
        a.cand_len = static_cast<int32_t>(cand);
        const int64_t kk = (k + 3) / 4 * 4, pp = ((c.tree ? tn::out_room((int)k) : tn::out_most((int)k)) + 3) / 4 * 4;
        a.group_bytes = static_cast<int32_t>(words * 4 + cand * 8 + kk * 8 + pp * 8 + 16 +
                                             (c.tree ? 2 * tn::kOutList * 4 : 0));
    }
    a.partials = reinterpret_cast<tn::OutPartial *>(o.ws + o.partial_off);
    a.maxima = reinterpret_cast<uint32_t *>(o.ws + o.maxima_off);
    a.supers = reinterpret_cast<uint32_t *>(o.ws + o.super_off);
    const cudaError_t e = by_type(o.type, tn::outcomes_forward_of<TN_TYPE_C64>, tn::outcomes_forward_of<TN_TYPE_F32>,
                                  tn::outcomes_forward_of<TN_TYPE_BF16>, tn::outcomes_forward_of<TN_TYPE_F16>, a,
                                  s.warp_rows, stream);
    return e == cudaSuccess ? TN_OK : cuda_fail(o, e, "launching the forward pass");
}

tn_status gradient(Outcomes &o, const tn::OutGrad &a, const tn::OutSplit &s, cudaStream_t stream) {
    const cudaError_t e = by_type(o.type, tn::outcomes_grad_of<TN_TYPE_C64>, tn::outcomes_grad_of<TN_TYPE_F32>,
                                  tn::outcomes_grad_of<TN_TYPE_BF16>, tn::outcomes_grad_of<TN_TYPE_F16>, a,
                                  s.warp_rows, stream);
    return e == cudaSuccess ? TN_OK : cuda_fail(o, e, "launching the gradient");
}

// CTAs of a cluster that hold a row in shared memory: a power of two, as others
// pack badly (2048x100001 bf16 by three 265 us, by four 205; 300x100001 f32 by six
// 69, by eight 62).  segs 0: better by a forward pass and a gradient, which read
// the row twice.  That is so
//  - for slices that leave one or two CTAs an SM: 200x800003 bf16 167 against
//    227 us, 500x100001 amplitudes 204 against 336, 300x200001 f32 130 against 142;
//  - for many rows by eight that could almost be by four: 2048x160001 bf16 318
//    against 375 (but 500x250001 135 against 127);
//  - for many rows of amplitudes by four or more: 500x25001 62 against 73, 500x60001
//    127 against 142 (by two 2000x16384 135 against 120).
tn::OutSplit step_split(int32_t type, int64_t cols, int64_t rows, bool aligned, int32_t count, tn::OutStep *a) {
    tn::OutSplit s = tn::out_split(type, cols, rows, aligned, step_warp_vecs(rows));
    if (s.warp_rows) return s;
    const int64_t bytes = s.vecs * tn::kOutVecBytes, teachers = tn::step_lists(count);
    int64_t c = (bytes + tn::kStepSlice - teachers - 1) / (tn::kStepSlice - teachers);
    // few rows: more CTAs a row, of two vectors a thread at least
    while (c < tn::kStepCluster && rows * c < 2 * tn::kOutSms && s.vecs >= 2 * (c + 1) * tn::kStepThreads) ++c;
    c = c <= 2 ? c : c <= 4 ? 4 : tn::kStepCluster;
    s.segs = c;
    s.seg_vecs = (s.vecs + c - 1) / c;
    const int64_t slice = s.seg_vecs * tn::kOutVecBytes;
    // Twice the threads where a CTA waits for others that hold as much: half
    // the work between two barriers (500x32003 f32 by two CTAs 36 against 39 us,
    // 1000x50000 f32 by four 95 against 105).  Otherwise what a row costs a
    // warp besides its vectors counts for more (4096x32000 bf16 by one 99
    // against 96, 2048x50001 bf16 by two 105 against 95, 2000x16384 amplitudes
    // by two 125 against 118).  And where the teacher's outcomes need them.
    a->wide = count > tn::kStepThreads || (slice > (32 << 10) && c >= (type == TN_TYPE_F32 ? 2 : 3));
    const bool many = rows * c > 3 * tn::kOutSms;
    if (slice + teachers > tn::kStepSlice) s.segs = 0;
    if (many && (type == TN_TYPE_C64 ? c >= 4 : type != TN_TYPE_F32 && c == 8 && slice < (48 << 10))) s.segs = 0;
    return s;
}

}  // namespace

extern "C" {

tn_status tn_outcomes_create(int32_t type, int64_t cols, int64_t max_rows, int32_t max_top, float scale,
                             tn_outcomes_t **out) {
    if (!out) return fail(g_error, TN_EINVAL, "out is NULL");
    *out = nullptr;
    if (type < TN_TYPE_C64 || type > TN_TYPE_F16) return fail(g_error, TN_EINVAL, "unknown entry type %d", (int)type);
    if (cols < 1 || max_rows < 1) return fail(g_error, TN_EINVAL, "cols and max_rows must be >= 1");
    if (max_top < 0 || max_top > TN_OUTCOMES_MAX_TOP)
        return fail(g_error, TN_EINVAL, "max_top %d outside 0 .. %d", (int)max_top, (int)TN_OUTCOMES_MAX_TOP);
    if (!(scale >= 0x1p-40f && scale <= 0x1p40f))
        return fail(g_error, TN_EINVAL, "scale must lie in 2^-40 .. 2^40");
    if (cols > (int64_t)1 << 40) return fail(g_error, TN_EOVERFLOW, "more than 2^40 entries a row");
    int64_t items;
    if (!mul_ok(max_rows, tn::out_split(type, cols, max_rows, false, tn::kOutWarpVecs).segs, &items) || items > 0x7fffffff)
        return fail(g_error, TN_EOVERFLOW, "more than 2^31 - 1 row segments");
    tn_outcomes_s *h = new (std::nothrow) tn_outcomes_s;
    if (!h) return fail(g_error, TN_ENOMEM, "host allocation failed");
    Outcomes &o = h->o;
    o.type = type;
    o.cols = cols;
    o.max_rows = max_rows;
    o.max_top = max_top;
    o.scale = scale;
    const Need n = workspace_need(o);
    o.partial_off = 256;
    o.maxima_off = align(o.partial_off + n.slots * sizeof(tn::OutPartial));
    o.super_off = align(o.maxima_off + n.maxima * sizeof(uint32_t));
    o.ws_bytes = align(o.super_off + n.supers * sizeof(uint32_t));
    g_error[0] = 0;
    *out = h;
    return TN_OK;
}

void tn_outcomes_destroy(tn_outcomes_t *h) { delete h; }

tn_status tn_outcomes_workspace_bytes(const tn_outcomes_t *h, uint64_t *bytes) {
    if (!h || !bytes) return TN_EINVAL;
    *bytes = h->o.ws_bytes;
    return TN_OK;
}

tn_status tn_outcomes_set_workspace(tn_outcomes_t *h, void *dev_ptr, uint64_t bytes) {
    if (!h) return TN_EINVAL;
    Outcomes &o = h->o;
    if (!dev_ptr || reinterpret_cast<uintptr_t>(dev_ptr) % 256)
        return fail(o.error, TN_EINVAL, "workspace must be a non-NULL 256-byte aligned device pointer");
    if (bytes < o.ws_bytes)
        return fail(o.error, TN_ENOMEM, "workspace of %llu bytes is smaller than the %llu bytes needed",
                    (unsigned long long)bytes, (unsigned long long)o.ws_bytes);
    o.ws = nullptr;
    // the status word; the rest is written before it is read
    cudaError_t e = cudaMemset(dev_ptr, 0, o.partial_off);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(o, e, "clearing the workspace");
    o.ws = static_cast<char *>(dev_ptr);
    return TN_OK;
}

tn_status tn_outcomes_score(tn_outcomes_t *h, const tn_rows *rows, const int64_t *given, int32_t n_given,
                            float *logp, float *logz, float *entropy, int32_t n_top, int64_t *top_ids,
                            float *top_logp, tn_stream_t stream) {
    if (!h) return TN_EINVAL;
    Outcomes &o = h->o;
    tn_status st = common(o, rows);
    if (st != TN_OK) return st;
    if (n_given < 0 || n_given > TN_OUTCOMES_MAX_IDS)
        return fail(o.error, TN_EINVAL, "n_given %d outside 0 .. %d", (int)n_given, (int)TN_OUTCOMES_MAX_IDS);
    if (n_top < 0 || n_top > o.max_top)
        return fail(o.error, TN_EINVAL, "n_top %d outside 0 .. %d", (int)n_top, (int)o.max_top);
    if (rows->rows == 0) return TN_OK;
    if (!logz || !entropy || (n_given > 0 && (!given || !logp)) || (n_top > 0 && (!top_ids || !top_logp)))
        return fail(o.error, TN_EINVAL, "an output or the given outcomes are missing");
    const tn::OutSplit s = tn::out_split(o.type, o.cols, rows->rows, aligned(o, rows),
                                         warp_vecs(rows->rows));
    tn::OutForward a = {};
    a.r = rows_of(o, rows, s);
    a.given = given;
    a.n_given = n_given;
    a.logp = logp;
    a.logz = logz;
    a.entropy = entropy;
    a.n_top = n_top;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    return forward(o, a, s, reinterpret_cast<cudaStream_t>(stream));
}

tn_status tn_outcomes_score_grad(tn_outcomes_t *h, const tn_rows *rows, const int64_t *given, int32_t n_given,
                                 const float *logz, const float *entropy, const float *g_logp,
                                 const float *g_entropy, void *grad, int64_t grad_row_stride,
                                 int64_t grad_col_stride, tn_stream_t stream) {
    if (!h) return TN_EINVAL;
    Outcomes &o = h->o;
    tn_status st = common(o, rows);
    if (st == TN_OK) st = check_grad(o, rows, grad, grad_row_stride, grad_col_stride);
    if (st != TN_OK) return st;
    if (n_given < 0 || n_given > TN_OUTCOMES_MAX_IDS)
        return fail(o.error, TN_EINVAL, "n_given %d outside 0 .. %d", (int)n_given, (int)TN_OUTCOMES_MAX_IDS);
    if (rows->rows == 0) return TN_OK;
    if (!logz || (n_given > 0 && (!given || !g_logp)) || (g_entropy && !entropy))
        return fail(o.error, TN_EINVAL, "logz, the given outcomes with g_logp, or entropy are missing");
    const tn::OutSplit s = tn::out_split(o.type, o.cols, rows->rows, aligned(o, rows),
                                         grad_warp_vecs(rows->rows));
    tn::OutGrad a = {};
    a.r = rows_of(o, rows, s);
    a.logz = logz;
    a.given = given;
    a.n_given = n_given;
    a.entropy = entropy;
    a.g_logp = g_logp;
    a.g_entropy = g_entropy;
    a.grad = static_cast<char *>(grad);
    a.grad_row_stride = grad_row_stride;
    a.grad_col_stride = o.cols == 1 ? 1 : grad_col_stride;
    return gradient(o, a, s, reinterpret_cast<cudaStream_t>(stream));
}

tn_status tn_outcomes_distill(tn_outcomes_t *h, const tn_rows *rows, const tn_teacher *teacher, float *loss,
                              float *logz, tn_stream_t stream) {
    if (!h) return TN_EINVAL;
    Outcomes &o = h->o;
    tn_status st = common(o, rows);
    if (st == TN_OK) st = check_teacher(o, rows, teacher);
    if (st != TN_OK) return st;
    if (rows->rows == 0) return TN_OK;
    if (!loss || !logz) return fail(o.error, TN_EINVAL, "loss and logz are required");
    const tn::OutSplit s = tn::out_split(o.type, o.cols, rows->rows, aligned(o, rows),
                                         warp_vecs(rows->rows));
    tn::OutForward a = {};
    a.r = rows_of(o, rows, s);
    a.logz = logz;
    a.loss = loss;
    a.teacher = teacher_of(teacher);
    return forward(o, a, s, reinterpret_cast<cudaStream_t>(stream));
}

tn_status tn_outcomes_distill_grad(tn_outcomes_t *h, const tn_rows *rows, const tn_teacher *teacher,
                                   const float *logz, const float *g_loss, void *grad,
                                   int64_t grad_row_stride, int64_t grad_col_stride, tn_stream_t stream) {
    if (!h) return TN_EINVAL;
    Outcomes &o = h->o;
    tn_status st = common(o, rows);
    if (st == TN_OK) st = check_teacher(o, rows, teacher);
    if (st == TN_OK) st = check_grad(o, rows, grad, grad_row_stride, grad_col_stride);
    if (st != TN_OK) return st;
    if (rows->rows == 0) return TN_OK;
    if (!logz || !g_loss) return fail(o.error, TN_EINVAL, "logz and g_loss are required");
    const tn::OutSplit s = tn::out_split(o.type, o.cols, rows->rows, aligned(o, rows),
                                         grad_warp_vecs(rows->rows));
    tn::OutGrad a = {};
    a.r = rows_of(o, rows, s);
    a.logz = logz;
    a.g_loss = g_loss;
    a.teacher = teacher_of(teacher);
    a.grad = static_cast<char *>(grad);
    a.grad_row_stride = grad_row_stride;
    a.grad_col_stride = o.cols == 1 ? 1 : grad_col_stride;
    return gradient(o, a, s, reinterpret_cast<cudaStream_t>(stream));
}

tn_status tn_outcomes_distill_step(tn_outcomes_t *h, const tn_rows *rows, const tn_teacher *teacher,
                                   const float *g_loss, float *loss, float *logz, void *grad,
                                   int64_t grad_row_stride, int64_t grad_col_stride, tn_stream_t stream) {
    if (!h) return TN_EINVAL;
    if (rows && rows->rows > 0 && !g_loss) return fail(h->o.error, TN_EINVAL, "g_loss is required");
    if (rows) {
        const tn_status st = check_grad(h->o, rows, grad, grad_row_stride, grad_col_stride);
        if (st != TN_OK) return st;
    }
    Outcomes &o = h->o;
    tn_status st = common(o, rows);
    if (st == TN_OK) st = check_teacher(o, rows, teacher);
    if (st != TN_OK) return st;
    if (rows->rows == 0) return TN_OK;
    if (!loss || !logz) return fail(o.error, TN_EINVAL, "loss and logz are required");
    tn::OutStep a = {};
    const tn::OutSplit s = step_split(o.type, o.cols, rows->rows, aligned(o, rows), teacher->count, &a);
    if (s.segs == 0) {      // rows that no cluster holds: two passes
        st = tn_outcomes_distill(h, rows, teacher, loss, logz, stream);
        if (st != TN_OK) return st;
        return tn_outcomes_distill_grad(h, rows, teacher, logz, g_loss, grad, grad_row_stride, grad_col_stride,
                                        stream);
    }
    a.r = rows_of(o, rows, s);
    a.teacher = teacher_of(teacher);
    a.g_loss = g_loss;
    a.loss = loss;
    a.logz = logz;
    a.grad = static_cast<char *>(grad);
    a.grad_row_stride = grad_row_stride;
    a.grad_col_stride = o.cols == 1 ? 1 : grad_col_stride;
    const cudaError_t e = by_type(o.type, tn::outcomes_step_of<TN_TYPE_C64>, tn::outcomes_step_of<TN_TYPE_F32>,
                                  tn::outcomes_step_of<TN_TYPE_BF16>, tn::outcomes_step_of<TN_TYPE_F16>, a,
                                  s.warp_rows, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TN_OK : cuda_fail(o, e, "launching the training step");
}

tn_status tn_outcomes_check(tn_outcomes_t *h) {
    if (!h) return TN_EINVAL;
    Outcomes &o = h->o;
    if (!o.ws) return TN_OK;
    tn::DevStatus d{0, 0};
    cudaError_t e = cudaMemcpy(&d, o.ws, sizeof(d), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(o, e, "reading the status word");
    if (d.code == tn::ERR_NONE) return TN_OK;
    e = cudaMemset(o.ws, 0, sizeof(d));
    if (e != cudaSuccess) return cuda_fail(o, e, "clearing the status word");
    return fail(o.error, TN_EDEVICE, "an outcome's id is outside [-1, cols) in row %d", (int)d.where);
}

const char *tn_outcomes_last_error(const tn_outcomes_t *h) { return h ? h->o.error : g_error; }

}  // extern "C"
