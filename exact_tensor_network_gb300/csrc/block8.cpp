// C ABI of the 8-bit matrices and their products (include/tn_block8.h):
// argument checks, choice of tiles and launches.  Kernels are in
// k_block8_*.cu.  Nothing here allocates or throws.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "block8.h"

namespace {

thread_local char g_error[256] = {0};

tn_status fail(tn_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return st;
}

tn_status cuda_fail(cudaError_t e, const char *what) {
    return fail(TN_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMost = 0x7fffffff - 1024;    // rows or columns: TMA coordinates are 32-bit

int entry_bytes(int32_t type) { return type == TN_TYPE_F32 ? 4 : 2; }

// A quantised matrix of that shape.
tn_status check(const tn_block8 *m, const char *name) {
    if (!m) return fail(TN_EINVAL, "%s is required", name);
    if (m->rows < 0 || m->cols < 0) return fail(TN_EINVAL, "%s has a negative size", name);
    if (m->rows > kMost || m->cols > kMost) return fail(TN_EOVERFLOW, "%s has a side of 2^31 or more", name);
    if (m->block_rows != 1 && m->block_rows != TN_BLOCK8)
        return fail(TN_EINVAL, "block_rows of %s must be 1 or %d", name, (int)TN_BLOCK8);
    if (m->row_stride < m->cols || m->row_stride % 16)
        return fail(TN_EINVAL, "the row stride of %s must be a multiple of 16 and at least its columns", name);
    if (m->scale_stride < 1 || m->scale_block < 1) return fail(TN_EINVAL, "strides of the scales of %s must be > 0", name);
    if (m->rows > 0 && m->cols > 0) {
        if (!m->codes || !m->scales) return fail(TN_EINVAL, "codes and scales of %s are required", name);
        if (reinterpret_cast<uintptr_t>(m->codes) % 16)
            return fail(TN_EINVAL, "codes of %s must be 16-byte aligned", name);
        if (reinterpret_cast<uintptr_t>(m->scales) % 4) return fail(TN_EINVAL, "scales of %s are not aligned", name);
    }
    return TN_OK;
}

// What TMA reads of an operand: boxes of `box` rows by 128 codes.
tn_status encode(CUtensorMap *map, const tn_block8 *m, int box) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn_encode = nullptr;
    auto fn = __atomic_load_n(&fn_encode, __ATOMIC_RELAXED);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return cuda_fail(e, "looking up cuTensorMapEncodeTiled");
        if (q != cudaDriverEntryPointSuccess || !p) return fail(TN_ECUDA, "cuTensorMapEncodeTiled is unavailable");
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        __atomic_store_n(&fn_encode, fn, __ATOMIC_RELAXED);
    }
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(m->cols), static_cast<cuuint64_t>(m->rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m->row_stride)};
    const cuuint32_t boxes[2] = {TN_BLOCK8, static_cast<cuuint32_t>(box)};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r =
        fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m->codes, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? TN_OK : fail(TN_ECUDA, "cuTensorMapEncodeTiled failed with %d", (int)r);
}

// Rows of Q a tile, and the CTAs that share a tile's blocks of k.
struct Tiles {
    bool swapped;       // P is the product's b
    int bn, split;
};

// By rounds of CTAs times what one takes: its blocks of k, and what a tile costs besides
// (in blocks of 240 columns, some 0.4 us: launch, first loads and outputs 6, sums that meet in a
// cluster 4 more).  1000 x 1112 x 5003: 72 tiles of 128 in two parts each 14 us, 40 of 240 43;
// 500 x 500 x 8192: 16 tiles of 128 in eight parts 18 us, in one 40.
Tiles choose(int64_t m, int64_t n, int64_t kbs, int most) {
    Tiles t = {};
    t.swapped = m <= 128;
    const int64_t p = t.swapped ? n : m, q = t.swapped ? m : n;
    double best = 0;
    for (const int bn : {most, 128, 64, 32, 16}) {
        // the narrowest that holds q, or one of the two for many
        if (q > 128 ? bn < 128 : bn > 128 || bn < q || (bn > 16 && bn / 2 >= q)) continue;
        const int64_t tiles = ceil_div(p, tn::kB8Tile) * ceil_div(q, bn);
        const int64_t room = bn >= 128 ? tn::kB8Sms : 2 * tn::kB8Sms;
        const double block = bn >= 240 ? 1.0 : bn == 128 ? 0.6 : 0.5;
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (bn > 128 || kbs < 4 * split)) break;
            const double cost = static_cast<double>(ceil_div(tiles * split, room)) *
                                (static_cast<double>(ceil_div(kbs, split)) * block + (split > 1 ? 10 : 6));
            if (best > 0 && cost >= best) continue;
            best = cost;
            t.bn = bn;
            t.split = split;
        }
    }
    return t;
}

}  // namespace

extern "C" {

tn_status tn_block8_quantize(const tn_matrix *x, const tn_block8 *rows, const tn_block8 *columns, tn_stream_t stream) {
    if (!x || (!rows && !columns)) return fail(TN_EINVAL, "x and an output are required");
    if (x->type != TN_TYPE_F32 && x->type != TN_TYPE_BF16 && x->type != TN_TYPE_F16)
        return fail(TN_EINVAL, "x must be f32, bf16 or f16");
    if (x->rows < 0 || x->cols < 0) return fail(TN_EINVAL, "x has a negative size");
    if (x->rows > kMost || x->cols > kMost) return fail(TN_EOVERFLOW, "x has a side of 2^31 or more");
    if (x->row_stride < 0 || x->col_stride < 0) return fail(TN_EINVAL, "strides of x must be >= 0");
    tn_status st = TN_OK;
    if (rows) {
        st = check(rows, "rows");
        if (st == TN_OK && (rows->rows != x->rows || rows->cols != x->cols))
            st = fail(TN_EINVAL, "rows must have x's shape");
    }
    if (st == TN_OK && columns) {
        st = check(columns, "columns");
        if (st == TN_OK && (columns->rows != x->cols || columns->cols != x->rows))
            st = fail(TN_EINVAL, "columns must have the shape of x transposed");
        if (st == TN_OK && rows && rows->block_rows != columns->block_rows)
            st = fail(TN_EINVAL, "rows and columns must have the same block_rows");
    }
    if (st != TN_OK) return st;
    if (x->rows == 0 || x->cols == 0) return TN_OK;
    const int size = entry_bytes(x->type);
    if (!x->data || reinterpret_cast<uintptr_t>(x->data) % size)
        return fail(TN_EINVAL, "x is missing or not aligned to its entry type");
    tn::QuantArgs a = {};
    a.x = x->data;
    a.rows = x->rows;
    a.cols = x->cols;
    a.row_stride = x->row_stride;
    a.col_stride = x->col_stride;
    if (rows) a.r = {rows->codes, rows->scales, rows->row_stride, rows->scale_stride, rows->scale_block};
    if (columns) a.c = {columns->codes, columns->scales, columns->row_stride, columns->scale_stride,
                        columns->scale_block};
    if (a.row_stride == 1 && a.col_stride != 1) {       // x transposed is read along its rows
        const tn::Block8Out r = a.r;
        a.r = a.c;
        a.c = r;
        a.rows = x->cols;
        a.cols = x->rows;
        a.row_stride = x->col_stride;
        a.col_stride = 1;
    }
    a.row_tiles = ceil_div(a.rows, tn::kB8Tile);
    a.col_tiles = ceil_div(a.cols, tn::kB8Tile);
    if (a.row_tiles > 0x7fffffff / a.col_tiles) return fail(TN_EOVERFLOW, "more than 2^31 - 1 blocks of 128 x 128");
    const bool square = (rows ? rows : columns)->block_rows == TN_BLOCK8;
    a.few = !a.c.codes && !square && a.rows < 256;
    const int vec = a.few ? 16 / size : 4;      // entries at once: 16 bytes, or a lane's of a tile
    a.vec = a.col_stride == 1 && reinterpret_cast<uintptr_t>(a.x) % (vec * size) == 0 &&
            (a.row_stride % vec == 0 || a.rows == 1);
    const cudaError_t e = tn::launch_quantize(a, x->type, square, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TN_OK : cuda_fail(e, "launching the quantisation");
}

tn_status tn_block8_product(const tn_block8 *a, const tn_block8 *b, void *out, int32_t type, int64_t out_stride,
                            tn_stream_t stream) {
    tn_status st = check(a, "a");
    if (st == TN_OK) st = check(b, "b");
    if (st != TN_OK) return st;
    if (a->cols != b->cols) return fail(TN_EINVAL, "a has %lld columns, b %lld", (long long)a->cols, (long long)b->cols);
    if (type != TN_TYPE_F32 && type != TN_TYPE_BF16 && type != TN_TYPE_F16)
        return fail(TN_EINVAL, "the output must be f32, bf16 or f16");
    if (out_stride < b->rows) return fail(TN_EINVAL, "the output's stride is less than its columns");
    const int64_t m = a->rows, n = b->rows;
    if (m == 0 || n == 0) return TN_OK;
    if (!out || reinterpret_cast<uintptr_t>(out) % entry_bytes(type))
        return fail(TN_EINVAL, "the output is missing or not aligned to its entry type");
    tn::ProductArgs g = {};
    g.kbs = static_cast<int32_t>(ceil_div(a->cols, TN_BLOCK8));
    const bool powers = a->powers && b->powers;
    const Tiles t = choose(m, n, g.kbs, powers ? 240 : 256);
    const tn_block8 *p = t.swapped ? b : a, *q = t.swapped ? a : b;
    if (g.kbs > 0) {
        st = encode(&g.tmP, p, tn::kB8Tile);
        if (st == TN_OK) st = encode(&g.tmQ, q, t.bn);
        if (st != TN_OK) return st;
    }
    g.scaleP = p->scales;
    g.scaleQ = q->scales;
    g.strideP = p->scale_stride;
    g.strideQ = q->scale_stride;
    g.blockP = p->scale_block;
    g.blockQ = q->scale_block;
    g.shiftP = p->block_rows == TN_BLOCK8 ? 7 : 0;
    g.shiftQ = q->block_rows == TN_BLOCK8 ? 7 : 0;
    g.p = p->rows;
    g.q = q->rows;
    g.sp = t.swapped ? 1 : out_stride;
    g.sq = t.swapped ? out_stride : 1;
    g.out = out;
    g.type = type;
    g.split = t.split;
    g.ptiles = ceil_div(g.p, tn::kB8Tile);
    g.qtiles = ceil_div(g.q, t.bn);
    if (g.ptiles > 0x7fffffff / 8 / g.qtiles) return fail(TN_EOVERFLOW, "too many tiles");
    const bool each = g.shiftQ == 0 || t.bn < 128;
    cudaError_t e = tn::block8_status(&g.status);
    if (e != cudaSuccess) return cuda_fail(e, "looking up the status");
    const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
    e = powers ? tn::launch_scaled(g, t.bn, on) : tn::launch_product(g, t.bn, each, on);
    return e == cudaSuccess ? TN_OK : cuda_fail(e, "launching the product");
}

tn_status tn_block8_check(void) {
    // what this thread has been told of each device's counts
    thread_local tn::Block8Status told[64] = {};
    tn::Block8Status d = {}, *at = nullptr;
    int device;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = tn::block8_status(&at);
    if (e == cudaSuccess) e = cudaMemcpy(&d, at, sizeof(d), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "reading the status");
    tn::Block8Status &seen = told[device & 63];
    if (d.timeouts != seen.timeouts) {
        seen.timeouts = d.timeouts;
        return fail(TN_ETIMEOUT, "a product gave up waiting: its outputs are not valid");
    }
    if (d.scales != seen.scales) {
        seen.scales = d.scales;
        return fail(TN_EDEVICE, "a scale is no power of two: it counted as NaN");
    }
    return TN_OK;
}

const char *tn_block8_last_error(void) { return g_error; }

}  // extern "C"
