// Gradients of the scores and of the loss against a teacher: one pass over
// the rows, from the saved log Z.  Included by the translation unit of each
// entry type.
//
// Both have the form
//     dL/dz_v = mult (p_v (alpha + beta (log p_v + H)) + sum_j add_j [id_j = v])
// with, for scores, mult = scale, alpha = - sum g, beta = - h, add = g, and,
// for the loss, mult = g_loss scale, alpha = 1 (0 where the teacher has
// nothing left), beta = 0, add = - q.  A CTA writes the dense part of its
// segment and then, after a barrier, overwrites the few entries with ids: the
// first of equal ids adds up all of them in order, so no atomics are needed.
//
// Bound by memory, one read and one write: 1024x50001 bf16 38.8 us (5.3 TB/s, at
// 45 % of the issue slots), f32 75 us (5.5 TB/s), 64x2^18 amplitudes 46 us (5.8
// TB/s), 2^20 amplitudes 5.6 us (of which launch and one pass of the ids'
// corrections after the last store).
#pragma once

#include "outcomes.cuh"

namespace tn {

namespace {

constexpr int kGradU = 4;           // vectors of a thread's step

struct RowGrad {
    float mult, alpha, beta, logz, entropy;
    float shift;      // log p = scale (z - shift) - log Z of the shifted row
    float inv_z;      // amplitudes at scale 1: p = w inv_z (0: not used)
    float scale;
    bool plain;       // log Z is a number: no entry needs a second look
};

// shift: 0, or the logit that c.logz is relative to; logz: as it is.
template <int TYPE>
__device__ __forceinline__ void finish_row_grad(RowGrad &c, float shift, float logz) {
    c.shift = shift;
    c.plain = fabsf(c.logz) < __builtin_huge_valf();
    c.inv_z = !Entry<TYPE>::kReal && c.scale == 1.f && fabsf(logz) < 80.f ? expf(-logz) : 0.f;
}

// log p of a weight; the roundings of scale ln w and log Z may leave it above 0,
// and far above where scale is large
__device__ __forceinline__ float amplitude_log_prob(const RowGrad &c, float w) {
    return min_nan(__fadd_rn(__fmul_rn(c.scale, logf(w) - c.shift), -c.logz), 0.f);
}

// Gradient of a real logit v that is present.
__device__ __forceinline__ float logit_grad(const RowGrad &c, float v, float add) {
    const float lp = max_nan(__fadd_rn(__fmul_rn(v - c.shift, c.scale), -c.logz), -1e30f);
    const float f = fmaf(c.beta, lp + c.entropy, c.alpha);
    if (lp < -80.f) {       // p may underflow where its multiple does not
        const float q = ex2(lp * (0.5f * kLog2E));
        return add == 0.f ? c.mult * q * (q * f) : c.mult * fmaf(q, q * f, add);
    }
    return c.mult * fmaf(ex2(lp * kLog2E), f, add);
}

// Gradient at an amplitude a of weight w that is present: 2 a / w dL/dz.  The
// quotients by w meet a first: 1 / w itself, and more so with what else there is
// to multiply, may be beyond fp32 where the gradient, of the size of 1 / |a|, is
// not.  p is the square of q, whose factors are multiplied in turn, as p may be
// below 2^-126 where p / |a| is not.
__device__ __forceinline__ float2 amplitude_grad(const RowGrad &c, float w, float2 a) {
    float lp = 0.f, q = 1.f, t = c.inv_z;
    if (c.beta != 0.f || c.inv_z == 0.f) {
        lp = amplitude_log_prob(c, w);
        if (c.inv_z == 0.f) {
            q = ex2(lp * (0.5f * kLog2E));
            t = q / w;
        }
    }
    const float n = 2.f * c.mult * fmaf(c.beta, lp + c.entropy, c.alpha) * q;
    return make_float2(t * a.x * n, t * a.y * n);
}
// and with what is added there: over one denominator, so that nothing is left
// where p f = -add (p = 1)
__device__ __forceinline__ float2 amplitude_grad(const RowGrad &c, float w, float2 a, float add) {
    if (add == 0.f) return amplitude_grad(c, w, a);
    const float lp = amplitude_log_prob(c, w), q = ex2(lp * (0.5f * kLog2E));
    const float n = 2.f * c.mult * fmaf(q, q * fmaf(c.beta, lp + c.entropy, c.alpha), add);
    return make_float2(a.x / w * n, a.y / w * n);
}

// The same for entry x of order value v, rounded to the rows' type.
template <int TYPE>
__device__ __forceinline__ typename Entry<TYPE>::T entry_grad(const RowGrad &c, float v,
                                                              typename Entry<TYPE>::T x, float add) {
    if constexpr (TYPE == TN_TYPE_F32) return logit_grad(c, v, add);
    else if constexpr (TYPE == TN_TYPE_BF16) return __float2bfloat16_rn(logit_grad(c, v, add));
    else if constexpr (TYPE == TN_TYPE_F16) return __float2half_rn(logit_grad(c, v, add));
    else return amplitude_grad(c, v, x, add);
}

// g[i] of the vector's real entries as 16 bytes of the rows' type
template <int TYPE>
__device__ __forceinline__ uint4 pack(const float (&g)[Entry<TYPE>::E]) {
    uint4 o;
    if constexpr (TYPE == TN_TYPE_F32) {
        o = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                       __float_as_uint(g[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == TN_TYPE_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(g[2 * i], g[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return o;
}

// The dense part of a vector of a row with a plain log Z (absent entries, at
// -inf or 0, come out as 0: their p is 0 and its factor finite).
template <int TYPE, bool BETA>
__device__ __forceinline__ uint4 dense_grad(const RowGrad &c, const uint4 &raw) {
    constexpr int E = Entry<TYPE>::E;
    float v[E];
    Entry<TYPE>::values(raw, v);
    if constexpr (Entry<TYPE>::kReal) {
        const float2 lz = make_float2(-c.logz, -c.logz);
        // bf16 reaches below the least p that ex2 gives: p is the square of
        // ex2(d / 2) there, multiplied in turn.  (f16 does not reach that far;
        // f32 rows keep the better p, and p < 2^-126 counts as 0.)
        constexpr bool kSquare = TYPE == TN_TYPE_BF16;
        constexpr float kL2 = kSquare ? 0.5f * kLog2E : kLog2E;
        const float2 l2 = make_float2(kL2, kL2);
        const float ma = c.mult * c.alpha;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            // (scalar products: they are rounded as log Z's is.  A packed product and a
            // packed sum become one fused operation, whose lp is the product's
            // rounding where both are large: p = inf for logits of 1e10.)
            float2 lp = add2(make_float2(__fmul_rn(v[i], c.scale), __fmul_rn(v[i + 1], c.scale)), lz);
            if constexpr (BETA) lp = make_float2(fmaxf(lp.x, -1e30f), fmaxf(lp.y, -1e30f));
            const float2 d = mul2(lp, l2);
            const float2 p = make_float2(ex2(d.x), ex2(d.y));
            float2 o;
            if constexpr (BETA) {
                const float2 h = make_float2(c.entropy, c.entropy), b = make_float2(c.beta, c.beta);
                const float2 f = fma2(b, add2(lp, h), make_float2(c.alpha, c.alpha));
                o = mul2(mul2(p, f), make_float2(c.mult, c.mult));
            } else {
                o = mul2(p, make_float2(ma, ma));
            }
            if constexpr (kSquare) o = mul2(o, p);
            v[i] = o.x;
            v[i + 1] = o.y;
        }
        return pack<TYPE>(v);
    } else {
        const float2 a = make_float2(__uint_as_float(raw.x), __uint_as_float(raw.y));
        const float2 b = make_float2(__uint_as_float(raw.z), __uint_as_float(raw.w));
        const float2 none = make_float2(0.f, 0.f);
        const float2 ga = v[0] == 0.f ? none : amplitude_grad(c, v[0], a);
        const float2 gb = v[1] == 0.f ? none : amplitude_grad(c, v[1], b);
        return make_uint4(__float_as_uint(ga.x), __float_as_uint(ga.y), __float_as_uint(gb.x),
                          __float_as_uint(gb.y));
    }
}

// Where a row's gradient goes.
template <int TYPE>
struct Out {
    using T = typename Entry<TYPE>::T;
    T *p;
    int64_t cs;
    bool wide;     // vectors of the row are vectors of the gradient

    __device__ __forceinline__ Out(char *grad, int64_t row_stride, int64_t col_stride, const Row<TYPE> &r,
                                   int64_t row)
        : p(reinterpret_cast<T *>(grad) + row * row_stride), cs(col_stride) {
        wide = cs == 1 && (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(r.p)) % kOutVecBytes == 0;
    }
    __device__ __forceinline__ void put(int64_t e0, const uint4 &o) const {
        if (wide) {
            *reinterpret_cast<uint4 *>(p + e0) = o;
        } else {
            union {
                uint4 q;
                T t[Entry<TYPE>::E];
            } u;
            u.q = o;
#pragma unroll
            for (int i = 0; i < Entry<TYPE>::E; ++i) p[(e0 + i) * cs] = u.t[i];
        }
    }
};

// Vector j entry by entry, with everything looked at.
template <int TYPE>
__device__ __noinline__ void grad_vector(const Row<TYPE> r, const RowGrad c, const Out<TYPE> out, int64_t j) {
    constexpr int E = Entry<TYPE>::E;
    const int64_t e0 = j * E - r.head;
#pragma unroll 1
    for (int64_t e = e0 < 0 ? 0 : e0; e < e0 + E && e < r.cols; ++e) {
        const float v = r.value(e);
        typename Entry<TYPE>::T o = typename Entry<TYPE>::T();
        if (v != absent<TYPE>()) o = entry_grad<TYPE>(c, v, r.p[e * r.cs], 0.f);
        out.p[e * out.cs] = o;
    }
}

// Ids that stand in a list more than once, without comparing all with all:
// every id leaves its place in two tables, at two hashes of it; one that finds
// another place there with its own id, or its own place in neither, is marked
// (with whom it found).  A mark may be wrong, the absence of one is not: equal
// ids meet at the same places, and whoever of them a table kept is found by
// the others.  put() for all, a barrier, look() for all, a barrier.
struct Repeats {
    uint8_t *a, *b, *mark;
    int slots;

    __device__ __forceinline__ Repeats(void *tables, void *marks, int n)
        : a(static_cast<uint8_t *>(tables)), b(a + repeat_slots(n)), mark(static_cast<uint8_t *>(marks)),
          slots(repeat_slots(n)) {}
    __device__ __forceinline__ uint32_t second(int64_t id) const {
        return ((uint32_t)id * 2654435769u) >> (__clz(slots) + 1);     // Fibonacci hashing
    }
    __device__ __forceinline__ void put(int j, int64_t id) const {
        mark[j] = 0;
        a[(uint32_t)id & (slots - 1)] = (uint8_t)j;
        b[second(id)] = (uint8_t)j;
    }
    __device__ __forceinline__ void look(const int64_t *ids, int j, int64_t id) const {
        const int x = a[(uint32_t)id & (slots - 1)], y = b[second(id)];
        const bool ex = ids[x] == id, ey = ids[y] == id;
        if (ex && x != j) mark[x] = mark[j] = 1;
        if (ey && y != j) mark[y] = mark[j] = 1;
        if (!ex && !ey) mark[j] = 1;
    }
};

// What the outcomes equal to ids[j] add up to, in order, for a warp's j's;
// false where ids[j] is not the first of them.  The warp looks through the
// list once for each marked one.
__device__ __forceinline__ bool sum_of_equal(const int64_t *ids, const float *adds, int n, int j, int64_t id,
                                             bool marked, float &sum) {
    const int lane = threadIdx.x % 32;
    bool first = true;
#pragma unroll 1
    for (uint32_t m = __ballot_sync(0xffffffffu, marked); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int64_t x = __shfl_sync(0xffffffffu, id, src);
        const int at = __shfl_sync(0xffffffffu, j, src);
        float total = 0.f;
        bool lead = true;
#pragma unroll 1
        for (int i = 0; i < n; i += 32) {
            uint32_t e = __ballot_sync(0xffffffffu, i + lane < n && ids[i + lane] == x);
            if (e && i + __ffs(e) - 1 < at) {
                lead = false;
                break;
            }
#pragma unroll 1
            for (; e; e &= e - 1) total += adds[i + __ffs(e) - 1];
        }
        if (lane == src) {
            sum = total;
            first = lead;
        }
    }
    return first;
}

// The same for a whole list at once, by a warp and whatever it costs with few
// repeats: sum[j] for each id, the same for equal ones.  The list is taken 32
// at a time; the first lane of equal ids adds up theirs in order, finds their
// place in a table (2 n places or more, by linear probing: the index, plus one,
// of the first with that id) and adds to what came before.  Lists of up to 32
// need no table.
__device__ __noinline__ void sums_of_equal(const int64_t *ids, const float *adds, int n, float *sum, uint32_t *table,
                                           uint8_t *first) {
    const int lane = threadIdx.x % 32;
    int slots = 64;
    while (slots < 2 * n) slots *= 2;
    if (n > 32) {
#pragma unroll 1
        for (int i = lane; i < slots / 4; i += 32) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int j = i0 + lane;
        const int64_t id = j < n ? ids[j] : -1;
        const uint32_t peers = __match_any_sync(0xffffffffu, (unsigned long long)id);
        const int lead = __ffs(peers) - 1;
        float total = 0.f;
        int at = j;
        if (lane == lead && id >= 0) {
#pragma unroll 1
            for (uint32_t m = peers; m; m &= m - 1) total += adds[i0 + __ffs(m) - 1];
            if (n > 32) {
                uint32_t place = ((uint32_t)id * 2654435769u) >> (__clz(slots) + 1);
#pragma unroll 1
                while (true) {       // (at most n places are ever taken)
                    const uint32_t old = atomicCAS(table + place, 0u, (uint32_t)j + 1);
                    if (old == 0) break;
                    if (ids[old - 1] == id) {
                        at = (int)old - 1;
                        break;
                    }
                    place = (place + 1) & (slots - 1);
                }
                if (at != j) total += sum[at];
                sum[at] = total;
            }
        }
        if (n > 32) {
            at = __shfl_sync(0xffffffffu, at, lead);
            if (id >= 0) first[j] = (uint8_t)at;
        } else {
            total = __shfl_sync(0xffffffffu, total, lead);
            if (id >= 0) sum[j] = total;
        }
        __syncwarp();
    }
    if (n > 32) {
#pragma unroll 1
        for (int j = lane; j < n; j += 32)
            if (ids[j] >= 0 && first[j] != j) sum[j] = sum[first[j]];
        __syncwarp();
    }
}

// The entries with ids among entries [lo, hi), after the dense part; entries
// [held_lo, held_hi) of the row are at held[entry - lo], masked ones absent.
// scratch: the tables and marks of n ids.
template <int TYPE, int G>
__device__ __forceinline__ void grad_ids(const Group<G> &g, const Row<TYPE> &r, const RowGrad &c,
                                         const Out<TYPE> &out, const int64_t *ids, const float *adds, float sign,
                                         int n, int64_t lo, int64_t hi, unsigned char *scratch,
                                         const typename Entry<TYPE>::T *held = nullptr, int64_t held_lo = 0,
                                         int64_t held_hi = 0) {
    const Repeats rp(scratch + repeat_marks(n), scratch, n);
    const auto mine = [&](int j) { return j < n && ids[j] >= 0 && ids[j] >= lo && ids[j] < hi; };
    const float *sums = nullptr;       // where all are added up
    const bool marks = n > (G == 32 ? 32 : 1);
    if (marks) {
        g.sync();
#pragma unroll 1
        for (int j = g.t; j < n; j += G)
            if (mine(j)) rp.put(j, ids[j]);
        g.sync();
#pragma unroll 1
        for (int j = g.t; j < n; j += G)
            if (mine(j)) rp.look(ids, j, ids[j]);
        g.sync();
    }
    if constexpr (G == 32) {
        // One marked id costs about a sixteenth of all added up: 20000 rows of 1000
        // entries with 64 ids (a few of them repeated) take 53 us by the marks and
        // 72 all added up, with 256 (57 marked) 466 and 231; 60375 of 32 entries
        // with 64 305 and 100.
        int marked = 0;
        if (marks) {
#pragma unroll 1
            for (int j0 = 0; j0 < n; j0 += 32)
                marked += __popc(__ballot_sync(0xffffffffu, mine(j0 + g.t) && rp.mark[j0 + g.t]));
        }
        if (n > 1 && (!marks || marked > 16)) {
            float *to = reinterpret_cast<float *>(scratch + repeat_bytes(n));
            g.sync();
            sums_of_equal(ids, adds, n, to, reinterpret_cast<uint32_t *>(scratch + repeat_marks(n)), scratch);
            sums = to;
        }
    }
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += G) {
        const int j = j0 + g.t;
        const bool in = mine(j);
        const int64_t id = in ? ids[j] : -1;
        float add = in ? (sums ? sums[j] : adds[j]) : 0.f;
        const bool first = sums || n == 1 || sum_of_equal(ids, adds, n, j, id, in && rp.mark[j], add);
        if (!in || !first) continue;
        typename Entry<TYPE>::T x;
        float v;
        if (held && id >= held_lo && id < held_hi) {
            x = held[id - lo];
            v = Entry<TYPE>::value(x);
        } else {
            x = r.p[id * r.cs];
            v = row_value<TYPE>(r, id);
        }
        if (v != absent<TYPE>()) out.p[id * out.cs] = entry_grad<TYPE>(c, v, x, sign * add);
    }
}

template <int TYPE, int G, bool MASK, bool BETA>
__device__ __forceinline__ void grad_dense(const Group<G> &g, const Row<TYPE> &r, const RowGrad &c,
                                           const Out<TYPE> &out, int64_t v0, int nv) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    int64_t in0, in1;
    r.inside_range(in0, in1);
    const int lo = (int)max((int64_t)0, min((int64_t)nv, in0 - v0));
    const int hi = c.plain ? max(lo, (int)max((int64_t)0, min((int64_t)nv, in1 - v0))) : lo;
    const uint4 *vecs = r.vectors() + v0;
    const bool words = !MASK || r.mask_words();
    const int64_t first = v0 * E - r.head;
#pragma unroll 1
    for (int b = 0; b < nv; b += kGradU * G) {
        uint4 raw[kGradU];
        if (words && out.wide && b >= lo && b + kGradU * G <= hi) {
#pragma unroll
            for (int u = 0; u < kGradU; ++u) raw[u] = __ldcg(vecs + b + u * G + g.t);
            if (MASK) {
                typename Row<TYPE>::Keep keep[kGradU];
#pragma unroll
                for (int u = 0; u < kGradU; ++u) keep[u] = r.keep_word(first + (int64_t)(b + u * G + g.t) * E);
#pragma unroll
                for (int u = 0; u < kGradU; ++u) En::blank(raw[u], keep[u]);
            }
            uint4 *to = reinterpret_cast<uint4 *>(out.p + first) + b + g.t;
#pragma unroll
            for (int u = 0; u < kGradU; ++u) to[u * G] = dense_grad<TYPE, BETA>(c, raw[u]);
            continue;
        }
        uint32_t odd = 0;
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
            const int j = b + u * G + g.t;
            if (j >= lo && j < hi && words) {
                raw[u] = __ldcg(vecs + j);
                if (MASK) En::blank(raw[u], r.keep_word(first + (int64_t)j * E));
            } else if (j < nv) {
                odd |= 1u << u;
            }
        }
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
            const int j = b + u * G + g.t;
            if (j >= lo && j < hi && words) out.put(first + (int64_t)j * E, dense_grad<TYPE, BETA>(c, raw[u]));
        }
#pragma unroll 1
        for (; odd; odd &= odd - 1) grad_vector<TYPE>(r, c, out, v0 + b + (__ffs(odd) - 1) * G + g.t);
    }
}

template <int TYPE, int G, bool MASK>
__global__ void __launch_bounds__(kOutThreads) outcomes_grad(const __grid_constant__ OutGrad a) {
    constexpr int E = Entry<TYPE>::E;
    constexpr int kGroups = kOutThreads / G;
    extern __shared__ __align__(16) unsigned char lists[];
    __shared__ uint32_t red[4 * kOutThreads / 32];
    pdl_trigger();
    Group<G> g(red);
    const uint32_t item = blockIdx.x * kGroups + threadIdx.x / G, segs = (uint32_t)a.r.segs;
    const int64_t row = G == 32 ? item : item / segs;
    const int64_t seg = G == 32 ? 0 : item % segs;
    const int n = a.teacher.count ? a.teacher.count : a.n_given;
    Teacher te(lists + threadIdx.x / G * teacher_bytes(n), n);
    int64_t *ids = te.id;
    float *adds = te.q;
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;

    const Row<TYPE> r(a.r, row);
    const int64_t v0 = seg * a.r.seg_vecs;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    const int64_t v1 = min(all, v0 + a.r.seg_vecs);
    const int nv = static_cast<int>(max((int64_t)0, v1 - v0));

    RowGrad c;
    c.scale = a.r.scale;
    c.logz = __ldcg(a.logz + row);
    c.beta = 0.f;
    c.entropy = 0.f;
    if (a.teacher.count) {
        te.read(g, a.teacher, a.r, r, row, false);
        g.sync();
        if (g.warp == 0) te.normalise(a.teacher);
        g.sync();
        c.alpha = *te.used;
        c.mult = a.g_loss[row] * a.r.scale;
    } else {
        float total = 0.f;
#pragma unroll 1
        for (int j = g.t; j < n; j += G) {
            int64_t id = a.given[row * n + j];
            if (id < -1 || id >= r.cols) {
                flag_bad_id(a.r, row);
                id = -1;
            }
            if (id >= 0 && row_value<TYPE>(r, id) == absent<TYPE>()) id = -1;
            const float x = id >= 0 ? a.g_logp[row * n + j] : 0.f;
            ids[j] = id;
            adds[j] = x;
            total += x;
        }
        c.alpha = -g.sum(total);
        if (a.g_entropy) {
            c.beta = -a.g_entropy[row];
            c.entropy = __ldcg(a.entropy + row);
        }
        c.mult = a.r.scale;
    }
    finish_row_grad<TYPE>(c, 0.f, c.logz);
    const Out<TYPE> out(a.grad, a.grad_row_stride, a.grad_col_stride, r, row);
    if (c.beta != 0.f) grad_dense<TYPE, G, MASK, true>(g, r, c, out, v0, nv);
    else grad_dense<TYPE, G, MASK, false>(g, r, c, out, v0, nv);
    if (n == 0) return;
    g.sync();
    grad_ids<TYPE>(g, r, c, out, ids, adds, a.teacher.count ? -1.f : 1.f, n, v0 * E - r.head, v1 * E - r.head,
                   lists + kGroups * teacher_bytes(n) + threadIdx.x / G * (repeat_bytes(n) + repeat_sums(n)));
}

template <int TYPE, int G, bool MASK>
cudaError_t launch_grad(const OutGrad &a, cudaStream_t stream) {
    const int64_t items = a.r.rows * a.r.segs;
    const int groups = kOutThreads / G;
    const int n = a.teacher.count ? a.teacher.count : a.n_given;
    const size_t smem = n ? groups * (teacher_bytes(n) + repeat_bytes(n) + repeat_sums(n)) : 0;
    return launch_pdl(outcomes_grad<TYPE, G, MASK>, dim3((unsigned)((items + groups - 1) / groups)),
                      dim3(kOutThreads), smem, stream, a);
}

}  // namespace

template <int TYPE>
cudaError_t outcomes_grad_of(const OutGrad &a, bool warp_rows, cudaStream_t stream) {
    if (warp_rows)
        return a.r.mask ? launch_grad<TYPE, 32, true>(a, stream) : launch_grad<TYPE, 32, false>(a, stream);
    return a.r.mask ? launch_grad<TYPE, kOutThreads, true>(a, stream)
                    : launch_grad<TYPE, kOutThreads, false>(a, stream);
}

}  // namespace tn
