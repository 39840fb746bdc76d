// Scores of outcome distributions, and the loss against a teacher: one pass
// over the rows.  Included by the translation unit of each entry type.
//
// Per row: log Z = ln sum exp(scale z), H = log Z - scale sum p z, and the k
// largest entries with their indices.  A thread keeps a reference entry z0
// and, with d = scale log2(e) (z - z0),
//     s = sum 2^d,   t = sum 2^d d;
// then log Z = scale z0 + ln s and H = ln s - ln2 t / s.  z0 follows the
// largest entry seen only once that is more than 2^8 above it: any reference
// near the maximum will do, and a rescale on every new maximum would be a
// divergent branch in most steps.
//
// Alternatives cost the pass one maximum per vector of 16 bytes, kept in
// shared memory (per 32 vectors in segments of more than 16 KiB).  Ordered by
// (value, lowest index first), the k best entries lie in the k best groups of
// any division into contiguous index ranges ordered by (largest entry, lowest
// range first): k groups that come before a group each hold an entry that
// comes before all of that group's.  So the k best chunks, then the k best of
// their vectors, then the k best of those vectors' entries are selected, and
// only those chunks are read again (from L2).
//
// A row of more than kOutSegVecs vectors, or one of a few rows, is cut into
// segments of one CTA each; the last CTA of a row to finish (a ticket)
// combines the segments' sums in segment order and selects among their lists
// in the same way.
#pragma once

#include "outcomes.cuh"

namespace tn {

namespace {

constexpr int kU = 4;               // vectors of a thread's step
constexpr float kLag = 8.f;         // of the reference, in powers of two
constexpr float kFar = 4.253529586511730e37f;   // 2^125
constexpr float kTiny = 7.888609052210118e-31f; // 2^-100

// ---- running sums -----------------------------------------------------------

// Distance of order value v from reference z in powers of two (amplitudes:
// of the weights' quotient, so that the reference itself is at 0 exactly).
template <int TYPE>
__device__ __forceinline__ float distance(float v, float z, float c2) {
    if constexpr (Entry<TYPE>::kReal) return (v - z) * c2;
    else return c2 * lg2(__fdiv_rn(v, z));
}

// z0: reference, an order value that was seen (absent until then).
template <int TYPE>
struct Sums {
    float z0 = absent<TYPE>(), s = 0.f, t = 0.f;

    __device__ __forceinline__ void move_by(float d) {
        d = max_nan(d, -1e4f);       // nothing is left below; not 0 times -inf
        const float f = ex2(d);
        t = s == 0.f ? 0.f : f * (t + s * d);
        s = s == 0.f ? 0.f : f * s;
    }
    __device__ __forceinline__ void move_to(float z, float c2) {
        move_by(distance<TYPE>(z0, z, c2));
        z0 = z;
    }
};

// largest order value of a vector's 16 bytes
template <int TYPE>
__device__ __forceinline__ float vector_max(const uint4 &q) {
    if constexpr (TYPE == TN_TYPE_BF16) {
        const uint32_t m = max_bf16x2(max_bf16x2(q.x, q.y), max_bf16x2(q.z, q.w));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        float v[Entry<TYPE>::E];
        Entry<TYPE>::values(q, v);
        float m = v[0];
#pragma unroll
        for (int i = 1; i < Entry<TYPE>::E; ++i) m = max_nan(m, v[i]);
        return m;
    }
}

// A thread's sums while it streams, in two halves for the packed arithmetic.
//
// Real logits: d = c2 v - ref with ref = c2 z0 rounded, one fused operation;
// done() takes the rounding of ref out again.  Absent entries become `floor`,
// about -2^126 / c2, so that they add 0 to both sums instead of 0 times -inf.
// Logits beyond 2^125 / c2 either way (masks written as the type's lowest
// value) would overflow there: ref = -inf then sends every vector through
// far(), which works with differences of logits.
//
// Amplitudes: the quotient w / z0 as q = w (1 / z0) with one Newton correction
// q + (w - q z0) / z0 (Markstein 1990), which makes z0 / z0 exactly 1.  z0 is
// at least 2^-100, for a finite reciprocal.
template <int TYPE, bool ENT, bool UNIT>
struct Stream {
    using En = Entry<TYPE>;
    static constexpr int E = En::E;
    float z0 = absent<TYPE>();
    float ref = -__builtin_huge_valf();      // real
    float inv = __builtin_huge_valf();       // amplitudes
    float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);

    __device__ __forceinline__ void move_by(float d) {
        d = max_nan(d, -1e4f);
        const float f = ex2(d);
        const bool any = s.x != 0.f || s.y != 0.f;     // true for NaN
        if constexpr (ENT) {
            t.x = any ? f * (t.x + s.x * d) : 0.f;
            t.y = any ? f * (t.y + s.y * d) : 0.f;
        }
        s.x = any ? f * s.x : 0.f;
        s.y = any ? f * s.y : 0.f;
    }
    // Add a vector: v its order values, for real logits not below `floor`, lm
    // their largest before that.  False if it is one for far().
    __device__ __forceinline__ bool add(const float (&v)[E], float lm, float c2) {
        if constexpr (En::kReal) {
            if (!(fmaf(lm, c2, -ref) <= kLag)) {
                if (lm == absent<TYPE>()) return true;
                const float r = lm * c2;
                if (fabsf(r) > kFar || (ref == -__builtin_huge_valf() && s.x != 0.f && z0 > 0.f)) return false;
                move_by(ref - r);
                ref = r;
                z0 = lm;
            }
            const float2 cc = make_float2(c2, c2), rr = make_float2(-ref, -ref);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 d = fma2(make_float2(v[i], v[i + 1]), cc, rr);
                const float2 e = make_float2(ex2(d.x), ex2(d.y));
                s = add2(s, e);
                if constexpr (ENT) t = fma2(e, d, t);
            }
        } else {
            if (!(lm * inv <= 256.f)) {
                if (lm == 0.f) return true;
                const float z = lm < kTiny ? kTiny : lm;
                move_by(z0 == 0.f ? 0.f : distance<TYPE>(z0, z, c2));
                z0 = z;
                inv = __fdiv_rn(1.f, z);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float q = v[i] * inv;
                q = fmaf(fmaf(-q, z0, v[i]), inv, q);
                float d = 0.f, e = q;
                // at scale 1 the weight may be below what lg2 takes, not 0
                if (ENT || !UNIT) d = max_nan(UNIT ? lg2(q) : c2 * lg2(q), UNIT ? -200.f : -1e30f);
                if (!UNIT) e = ex2(d);
                if (i & 1) {
                    s.y += e;
                    if constexpr (ENT) t.y = fmaf(e, d, t.y);
                } else {
                    s.x += e;
                    if constexpr (ENT) t.x = fmaf(e, d, t.x);
                }
            }
        }
        return true;
    }
    // Add a step of vectors without a look at each one's maximum (sums alone,
    // no entropy).  The reference comes from the first step; later ones may
    // exceed it by far before a sum overflows, and the sums are as good either
    // way.  False: nothing was added, take the vectors one by one.
    __device__ __forceinline__ bool add_step(const uint4 (&raw)[kU], float c2) {
        static_assert(!ENT, "the entropy's sum needs a near reference");
        constexpr float kBig = 1.2379400392853803e27f;    // 2^90
        constexpr float kInf = __builtin_huge_valf();
        if (En::kReal ? ref == -kInf : z0 == 0.f) {
            if (s.x != 0.f || s.y != 0.f) return false;   // (far out)
            float lm = vector_max<TYPE>(raw[0]);
#pragma unroll
            for (int u = 1; u < kU; ++u) lm = max_nan(lm, vector_max<TYPE>(raw[u]));
            if (lm == absent<TYPE>()) return true;
            if constexpr (En::kReal) {
                const float r = lm * c2;
                if (!(fabsf(r) <= kFar)) return false;
                ref = r;
                z0 = lm;
            } else {
                if (!(lm < kInf)) return false;
                z0 = lm < kTiny ? kTiny : lm;
                inv = __fdiv_rn(1.f, z0);
            }
        }
        const float2 before = s;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float v[E];
            En::values(raw[u], v);
            if constexpr (En::kReal) {
                const float2 cc = make_float2(c2, c2), rr = make_float2(-ref, -ref);
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    const float2 d = fma2(make_float2(v[i], v[i + 1]), cc, rr);
                    s = add2(s, make_float2(ex2(d.x), ex2(d.y)));
                }
            } else {
                float e[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float q = v[i] * inv;
                    e[i] = fmaf(fmaf(-q, z0, v[i]), inv, q);
                    if (!UNIT) e[i] = ex2(c2 * lg2(e[i]));
                }
                s = add2(s, make_float2(e[0], e[1]));
            }
        }
        if (s.x + s.y < kBig) return true;
        s = before;
        return false;
    }
    // the same for logits far out: v as they are
    __device__ __forceinline__ void far(const float (&v)[E], float lm, float c2) {
        if (!(lm <= z0)) {
            move_by((z0 - lm) * c2);
            z0 = lm;
        }
        ref = -__builtin_huge_valf();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = (v[i] - z0) * c2;
            const float e = ex2(d);
            s.x += e;
            if (ENT && e != 0.f) t.x = fmaf(e, d, t.x);
        }
    }
    __device__ __forceinline__ Sums<TYPE> done(float c2) const {
        Sums<TYPE> a;
        a.z0 = z0;
        a.s = s.x + s.y;
        a.t = t.x + t.y;
        if (En::kReal && ref != -__builtin_huge_valf()) a.move_by(-fmaf(z0, c2, -ref));
        return a;
    }
};

// Order values of a vector, cut off at `floor` (real logits), and their
// largest before that.
template <int TYPE>
__device__ __forceinline__ float largest(float (&v)[Entry<TYPE>::E], float floor) {
    float lm = v[0];
#pragma unroll
    for (int i = 1; i < Entry<TYPE>::E; ++i) lm = max_nan(lm, v[i]);
    if constexpr (Entry<TYPE>::kReal) {
#pragma unroll
        for (int i = 0; i < Entry<TYPE>::E; ++i) v[i] = max_nan(v[i], floor);
    }
    return lm;
}

// The same from a vector's 16 bytes; bf16 in its own type, two at a time.
template <int TYPE>
__device__ __forceinline__ float decode(const uint4 &raw, float (&v)[Entry<TYPE>::E], float floor) {
    if constexpr (TYPE == TN_TYPE_BF16) {
        const uint32_t m = max_bf16x2(max_bf16x2(raw.x, raw.y), max_bf16x2(raw.z, raw.w));
        const uint32_t f1 = __float_as_uint(floor) >> 16, f2 = f1 | f1 << 16;
        const uint4 c = make_uint4(max_bf16x2(raw.x, f2), max_bf16x2(raw.y, f2), max_bf16x2(raw.z, f2),
                                   max_bf16x2(raw.w, f2));
        Entry<TYPE>::values(c, v);
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        Entry<TYPE>::values(raw, v);
        return largest<TYPE>(v, floor);
    }
}

// The group's sums, relative to its largest reference, in every thread.
template <int TYPE, int G>
__device__ __forceinline__ void combine(Group<G> &g, Sums<TYPE> &a, float c2) {
    const float z = g.max(a.z0);
    // a thread that saw nothing has s = 0 and an absent reference
    if (z != a.z0) a.move_to(z, c2);
    g.sum2(a.s, a.t);
}

// ---- selection --------------------------------------------------------------

// A cut of n keys in the order (key descending, position ascending), keys of 0
// left out: keys above `thr`, and the first `ties` of those equal to it.
struct Cut {
    uint32_t thr, ties, count;
};

// A cut after at least k and at most `most` keys (all of them if they are no
// more than k), by bisection.  Ties are cut at k.
template <class CountFrom>
__device__ __forceinline__ Cut bisect(CountFrom count_from, uint32_t lo, uint32_t mx, uint32_t nz, int k,
                                      int most) {
    Cut c = {1u, 0xffffffffu, nz};
    if (nz <= (uint32_t)k) return c;
    if (k == 1) {
        c.thr = mx;
        c.ties = c.count = 1;
        return c;
    }
    uint32_t hi = mx + 1, above = 0;   // keys >= lo: k or more; keys >= hi: `above`, fewer than k
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const uint32_t m = count_from(mid);
        if (m >= (uint32_t)k && m <= (uint32_t)most) {
            c.thr = mid;
            c.count = m;
            return c;
        }
        if (m > (uint32_t)k) lo = mid;
        else {
            hi = mid;
            above = m;
        }
    }
    c.thr = lo;
    c.ties = k - above;
    c.count = k;
    return c;
}

// One warp: positions of the keys before a cut, of n keys in shared memory
// (readable and zero up to a multiple of four), in ascending order.
__device__ __noinline__ Cut warp_select(const uint32_t *keys, int n, int k, int most, uint32_t *out) {
    const int lane = threadIdx.x % 32;
    const uint4 *k4 = reinterpret_cast<const uint4 *>(keys);
    const int n4 = (n + 3) / 4;
    uint32_t mx = 0, nz = 0, mn = 0xffffffffu;     // mn: smallest but 0
#pragma unroll 1
    for (int i = lane; i < n4; i += 32) {
        const uint4 q = k4[i];
        mx = max(max(mx, q.x), max(max(q.y, q.z), q.w));
        mn = min(min(mn, q.x - 1), min(min(q.y - 1, q.z - 1), q.w - 1));
        nz += (q.x != 0) + (q.y != 0) + (q.z != 0) + (q.w != 0);
    }
    // each lane has a key of at least the smallest of the lanes' largest
    uint32_t low = __reduce_min_sync(0xffffffffu, mx);
    mn = __reduce_min_sync(0xffffffffu, mn);
    if (k > 32 || low == 0) low = mn + 1;
    mx = __reduce_max_sync(0xffffffffu, mx);
    nz = __reduce_add_sync(0xffffffffu, nz);
    const Cut c = bisect([=](uint32_t mid) {
        uint32_t m = 0;
    #pragma unroll 1
    for (int i = lane; i < n4; i += 32) {
            const uint4 q = k4[i];
            m += (q.x >= mid) + (q.y >= mid) + (q.z >= mid) + (q.w >= mid);
        }
        return __reduce_add_sync(0xffffffffu, m);
    }, low, mx, nz, k, most);
    uint32_t at = 0, tied = 0;
    const uint32_t before = (1u << lane) - 1;
#pragma unroll 1
    for (int b = 0; b < n && at < c.count; b += 32) {
        const uint32_t x = b + lane < n ? keys[b + lane] : 0u;
        const uint32_t te = __ballot_sync(0xffffffffu, x == c.thr);
        const bool take = x > c.thr || (x == c.thr && tied + __popc(te & before) < c.ties);
        const uint32_t ms = __ballot_sync(0xffffffffu, take);
        if (take) out[at + __popc(ms & before)] = b + lane;
        at += __popc(ms);
        tied += __popc(te);
    }
    return c;
}

// The same by a group, cut at k, for any keys.
template <int G, class KeyAt>
__device__ int select(Group<G> &g, KeyAt key, int n, int k, uint32_t *out) {
    uint32_t mx = 0, nz = 0;
#pragma unroll 1
    for (int i = g.t; i < n; i += G) {
        const uint32_t x = key(i);
        mx = max(mx, x);
        nz += x != 0;
    }
    mx = g.max(mx);
    nz = g.sum(nz);
    const Cut c = bisect([&](uint32_t mid) {
        uint32_t m = 0;
#pragma unroll 1
        for (int i = g.t; i < n; i += G) m += key(i) >= mid;
        return g.sum(m);
    }, 1u, mx, nz, k, k);
    const int per = (n + G - 1) / G;
    const int i0 = min(n, g.t * per), i1 = min(n, i0 + per);
    uint32_t gt = 0, eq = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = key(i);
        gt += x > c.thr;
        eq += x == c.thr;
    }
    uint32_t pg = gt, pe = eq;
    g.scan2(pg, pe);
    uint32_t at = pg + min(pe, c.ties);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = key(i);
        if (x > c.thr) out[at++] = i;
        else if (x == c.thr) {
            if (pe < c.ties) out[at++] = i;
            ++pe;
        }
    }
    g.sync();
    return (int)c.count;
}

// Candidates as one number: larger is better, equal keys by lowest index.
__device__ __forceinline__ uint64_t candidate(uint32_t key, uint32_t index) {
    return (uint64_t)key << 32 | (0xffffffffu - index);
}
__device__ __forceinline__ int rank_of(const uint64_t *c, int n, uint64_t x) {
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += c[j] > x;
    return r;
}

// Shared memory of a group (all offsets multiples of 16 bytes).
struct Scratch {
    uint32_t *keys;       // maxima of vectors or of chunks
    uint64_t *cand;       // candidates
    uint64_t *best;       // the k best, in order
    uint32_t *pos, *pos2; // out_most(k) positions each
    uint32_t *n;          // number of candidates, of positions, threshold, number of vectors
    __device__ __forceinline__ Scratch(unsigned char *base, const OutForward &a) {
        const int kk = (a.n_top + 3) / 4 * 4, pp = (out_most(a.n_top) + 3) / 4 * 4;
        keys = reinterpret_cast<uint32_t *>(base);
        cand = reinterpret_cast<uint64_t *>(keys + a.key_words);
        best = cand + a.cand_len;
        pos = reinterpret_cast<uint32_t *>(best + kk);
        pos2 = pos + pp;
        n = pos2 + pp;
    }
    // First k (up to `most`) of keys[0 .. n) by the group's first warp, into
    // pos; returns their number, `least` a lower bound of the k best entries.
    template <int G>
    __device__ __forceinline__ int cut(Group<G> &g, int nk, int k, int most, uint32_t &least) const {
        if (g.t < 32) {
            if (g.t < 4 && nk + g.t < (nk + 3) / 4 * 4) keys[nk + g.t] = 0;
            __syncwarp();
            const Cut c = warp_select(keys, nk, k, most, pos);
            if (g.t == 0) {
                n[0] = n[3] = 0;
                n[1] = c.count;
                n[2] = c.thr;
            }
        }
        g.sync();
        least = n[2];
        return (int)n[1];
    }
    __device__ __forceinline__ void offer(uint32_t key, uint32_t index, int cand_len) const {
        const uint32_t at = atomicAdd(n, 1u);
        if (at < (uint32_t)cand_len) cand[at] = candidate(key, index);
    }
};

// The k best of the candidates (0: none), in order, into sm.best.  Returns
// their number.
template <int G>
__device__ __forceinline__ int rank_candidates(Group<G> &g, const Scratch &sm, int n, int k) {
    uint32_t found = 0;
#pragma unroll 1
    for (int i = g.t; i < n; i += G) {
        const uint64_t x = sm.cand[i];
        if (x == 0) continue;
        const int r = rank_of(sm.cand, n, x);
        if (r < k) {
            sm.best[r] = x;
            ++found;
        }
    }
    found = g.sum(found);
    g.sync();
    return (int)found;
}

// The k best entries of `nv` vectors from v0 on into sm.best, as candidates
// with indices (vector - v0) E + entry, from the maxima in sm.keys, each that
// of 2^log vectors.  Returns their number.
template <int TYPE, bool MASK, int G>
__device__ __noinline__ int best_entries(Group<G> g, const Scratch sm, const Row<TYPE> r, int64_t v0,
                                         int nv, int k, int log, int cand_len) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    const int nk = (nv + (1 << log) - 1) >> log, low = (1 << log) - 1;
    uint32_t least;
    int nc = sm.cut(g, nk, k, log ? out_most(k) : k, least);
    // vectors with an entry of at least `bar` (the lowest present value at the
    // lowest), then those entries
    const float bar = fmaxf(key_value(least), En::kReal ? -3.402823466e38f : 1.401298464e-45f);
    uint32_t *list = reinterpret_cast<uint32_t *>(sm.cand + cand_len / 2);   // cand_len positions
    const int work = nc << log;
    const bool words = MASK && r.mask_words();
#pragma unroll 1
    for (int b = g.t; b < work; b += kU * G) {
        int j[kU];
        uint4 q[kU];
        uint32_t odd = 0;       // vectors to be read entry by entry
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = b + u * G;
            j[u] = i < work ? ((int)sm.pos[i >> log] << log) + (i & low) : nv;
            const int64_t e0 = (v0 + j[u]) * E - r.head;
            const bool in = j[u] < nv && r.inside(e0) && (!MASK || words);
            q[u] = En::absent_vector();
            if (in) q[u] = r.raw(e0);
            if (MASK && in) En::blank(q[u], r.keep_word(e0));
            if (!in && j[u] < nv) odd |= 1u << u;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (vector_max<TYPE>(q[u]) >= bar) {
                const uint32_t at = atomicAdd(sm.n + 3, 1u);
                if (at < (uint32_t)cand_len) list[at] = j[u];
            }
#pragma unroll 1
        for (; odd; odd &= odd - 1) {
            const int i = b + (__ffs(odd) - 1) * G;
            const int jj = ((int)sm.pos[i >> log] << log) + (i & low);
            const auto x = row_vector<TYPE>(r, v0 + jj);
            float lm = absent<TYPE>();
#pragma unroll
            for (int e = 0; e < E; ++e) lm = fmaxf(lm, x.v[e]);
            if (lm >= bar) {
                const uint32_t at = atomicAdd(sm.n + 3, 1u);
                if (at < (uint32_t)cand_len) list[at] = jj;
            }
        }
    }
    g.sync();
    int nl = (int)sm.n[3];
    if (nl <= cand_len) {
#pragma unroll 1
        for (int i = g.t; i < nl * E; i += G) {
            const int jj = (int)list[i / E], e = i % E;
            const int64_t at = (v0 + jj) * E - r.head + e;
            const float v = at >= 0 && at < r.cols ? row_value<TYPE>(r, at) : absent<TYPE>();
            if (v >= bar) sm.offer(order_key<TYPE>(v), jj * E + e, cand_len / 2);
        }
        g.sync();
    }
    int n = (int)sm.n[0];
    if (nl > cand_len || n > cand_len / 2) {
        // Too many entries at the cut (long runs of equal or of sorted
        // entries): exactly k chunks, then the k best of their vectors, whose
        // entries fit (log > 0 here: the entries of k vectors always do).
        g.sync();
        nc = sm.cut(g, nk, k, k, least);
        uint32_t *sub = reinterpret_cast<uint32_t *>(sm.cand);
#pragma unroll 1
        for (int i = g.t; i < nc << log; i += G) {
            const int j = ((int)sm.pos[i >> log] << log) + (i & low);
            uint32_t key = 0;
            if (j < nv) {
                const auto x = row_vector<TYPE>(r, v0 + j);
                float lm = absent<TYPE>();
#pragma unroll
                for (int e = 0; e < E; ++e) lm = fmaxf(lm, x.v[e]);
                key = order_key<TYPE>(lm);
            }
            sub[i] = key;
        }
        g.sync();
        const int nsel = select(g, [=](int i) { return sub[i]; }, nc << log, k, sm.pos2);
#pragma unroll 1
        for (int i = g.t; i < nsel; i += G) {
            const uint32_t x = sm.pos2[i];
            sm.pos2[i] = (sm.pos[x >> log] << log) + (x & low);
        }
        g.sync();
#pragma unroll 1
        for (int i = g.t; i < nsel * E; i += G) {
            const int j = (int)sm.pos2[i / E], e = i % E;
            const int64_t at = (v0 + j) * E - r.head + e;
            const float v = at >= 0 && at < r.cols ? row_value<TYPE>(r, at) : absent<TYPE>();
            const uint32_t key = order_key<TYPE>(v);
            sm.cand[i] = key ? candidate(key, j * E + e) : 0;
        }
        g.sync();
        n = nsel * E;
    }
    // (ends with a barrier: the caller's g may use any slot again)
    return rank_candidates(g, sm, n, k);
}

// The k best of a split row among its segments' sorted lists, as candidates
// with positions in the row's lists.
template <int G>
__device__ __noinline__ int join_lists(Group<G> g, const Scratch sm, const OutForward &a, int64_t row) {
    const int k = a.n_top, segs = (int)a.r.segs;
    const uint64_t *lists = a.lists + row * a.r.segs * k;
    const auto key_at = [=](uint32_t i) { return (uint32_t)(__ldcg(lists + i) >> 32); };
    int nc;
    uint32_t least;
    if (segs <= a.key_words) {
#pragma unroll 1
        for (int i = g.t; i < segs; i += G) sm.keys[i] = key_at(i * k);
        g.sync();
        nc = sm.cut(g, segs, k, k, least);
    } else {
        nc = select(g, [=](int i) { return key_at((uint32_t)i * k); }, segs, k, sm.pos);
        uint32_t inv = 0;
#pragma unroll 1
        for (int i = g.t; i < nc; i += G) inv = max(inv, ~key_at(sm.pos[i] * k));
        inv = g.max(inv);
        least = nc ? ~inv : 1u;
        if (g.t == 0) sm.n[0] = 0;
        g.sync();
    }
#pragma unroll 1
    for (int i = g.t; i < nc * 4; i += G)      // sorted: few go past their first entries
#pragma unroll 1
        for (int e = i & 3; e < k; e += 4) {
            const uint32_t at = sm.pos[i >> 2] * k + e, key = key_at(at);
            if (key < least) break;
            sm.offer(key, at, a.cand_len);
        }
    g.sync();
    int n = (int)sm.n[0];
    if (n > a.cand_len) {
        // the first of eight consecutive keys of a list is their largest
        uint32_t *sub = reinterpret_cast<uint32_t *>(sm.cand);
        const int oct = (k + 7) / 8;
        g.sync();
#pragma unroll 1
        for (int i = g.t; i < nc * oct; i += G) sub[i] = key_at(sm.pos[i / oct] * k + i % oct * 8);
        g.sync();
        const int no = select(g, [=](int i) { return sub[i]; }, nc * oct, k, sm.pos2);
#pragma unroll 1
        for (int i = g.t; i < no; i += G) {
            const uint32_t x = sm.pos2[i];
            sm.pos2[i] = sm.pos[x / oct] * k + x % oct * 8;
        }
        g.sync();
#pragma unroll 1
        for (int i = g.t; i < no * 8; i += G) {
            const uint32_t first = sm.pos2[i / 8], at = first + i % 8;
            // the last octet of a list may be short
            const uint32_t key = at / k == first / k ? key_at(at) : 0u;
            sm.cand[i] = key ? candidate(key, at) : 0;
        }
        g.sync();
        n = no * 8;
    }
    return rank_candidates(g, sm, n, k);
}

// ---- the end of a row -------------------------------------------------------

template <int TYPE>
__device__ __forceinline__ float log_prob(const OutRows &r, float v, float logz) {
    // not fused, as log Z is not: a row's only entry has log p = 0 exactly
    return __fadd_rn(__fmul_rn(r.scale, Entry<TYPE>::kReal ? v : logf(v)), -logz);
}

// The loss of a row by one warp.
template <int TYPE>
__device__ __forceinline__ float teacher_loss(int count, const OutRows &r, const Teacher &te, float logz) {
    constexpr float kInf = __builtin_huge_valf();
    float loss = 0.f, bad = 0.f;
#pragma unroll 1
    for (int j = threadIdx.x % 32; j < count; j += 32) {
        if (te.id[j] == -2) bad = __int_as_float(0x7fffffff);
        if (te.id[j] >= 0 && te.q[j] != 0.f) {
            const float v = te.value[j];
            const float lp = v == absent<TYPE>() ? -kInf : log_prob<TYPE>(r, v, logz);
            loss += te.q[j] * (te.logq[j] - lp);
        }
    }
    if (logz == -kInf) loss = 0.f;
    loss += bad;
#pragma unroll
    for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    return loss;
}

template <int TYPE, bool ENT, int G>
__device__ __forceinline__ void finish_row(Group<G> &g, const OutForward &a, const Row<TYPE> &r,
                                           Teacher &te, int64_t row, float logz, float entropy) {
    constexpr float kInf = __builtin_huge_valf();
    if (g.t == 0) a.logz[row] = logz;
    if constexpr (ENT) {
        if (g.t == 0) a.entropy[row] = entropy;
#pragma unroll 1
        for (int j = g.t; j < a.n_given; j += G) {
            const int64_t id = a.given[row * a.n_given + j];
            float lp;
            if (id == -1) {
                lp = 0.f;
            } else if (id < 0 || id >= r.cols) {
                lp = __int_as_float(0x7fffffff);
                flag_bad_id(a.r, row);
            } else {
                const float v = row_value<TYPE>(r, id);
                lp = v == absent<TYPE>() ? -kInf : log_prob<TYPE>(a.r, v, logz);
            }
            a.logp[row * a.n_given + j] = lp;
        }
    } else {
        if (g.warp == 0) {
            te.normalise(a.teacher.count);
            const float loss = teacher_loss<TYPE>(a.teacher.count, a.r, te, logz);
            if (g.t == 0) a.loss[row] = loss;
        }
    }
}

// log Z and H of the sums; NaN where an entry was NaN or +inf.
template <int TYPE>
__device__ __forceinline__ void normaliser(const OutRows &r, const Sums<TYPE> &a, float &logz, float &entropy) {
    constexpr float kInf = __builtin_huge_valf();
    if (a.s == 0.f) {
        logz = -kInf;
        entropy = 0.f;
    } else if (a.s < kInf) {
        const float ls = logf(a.s);
        logz = __fadd_rn(__fmul_rn(r.scale, Entry<TYPE>::kReal ? a.z0 : logf(a.z0)), ls);
        entropy = ls - kLn2 * (a.t / a.s);
    } else {
        logz = entropy = __int_as_float(0x7fffffff);
    }
}

// ---- the kernel -------------------------------------------------------------

template <int TYPE, int G, bool MASK, bool ENT, bool UNIT>
__global__ void __launch_bounds__(kOutThreads, G == 32 ? 6 : kOutCtas)
outcomes_forward(const __grid_constant__ OutForward a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr int kGroups = kOutThreads / G;
    constexpr float kInf = __builtin_huge_valf();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t red[4 * kOutThreads / 32];
    __shared__ bool last;
    constexpr int kTeacher = ENT ? 16 : TN_OUTCOMES_MAX_IDS * 20 + 16;
    __shared__ __align__(16) unsigned char teachers[kGroups * kTeacher];
    Teacher te(teachers + threadIdx.x / G * kTeacher, ENT ? 0 : a.teacher.count);
    pdl_trigger();
    Group<G> g(red);
    const uint32_t item = blockIdx.x * kGroups + threadIdx.x / G, segs = (uint32_t)a.r.segs;
    const int64_t row = G == 32 ? item : item / segs;
    const int64_t seg = G == 32 ? 0 : item % segs;
    const Scratch sm(smem + (size_t)(threadIdx.x / G) * a.group_bytes, a);
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;

    const Row<TYPE> r(a.r, row);
    const int64_t v0 = seg * a.r.seg_vecs;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    const int64_t v1 = min(all, v0 + a.r.seg_vecs);
    const int nv = static_cast<int>(max((int64_t)0, v1 - v0));   // may be 0 in a row's last segment
    const int k = ENT ? a.n_top : 0;
    const int log = G > 32 ? a.chunk_log : 0;   // one maximum per 2^log vectors
    // vectors [lo, hi) of the segment lie inside the row
    int64_t in0, in1;
    r.inside_range(in0, in1);
    const int lo = (int)max((int64_t)0, min((int64_t)nv, in0 - v0));
    const int hi = max(lo, (int)max((int64_t)0, min((int64_t)nv, in1 - v0)));
    const uint4 *vecs = r.vectors() + v0;

    // A warp takes kU * 32 consecutive vectors a step (a chunk of them at most).
    constexpr int kStep = kU * 32;
    const bool words = MASK && r.mask_words();
    using Keep = typename Row<TYPE>::Keep;
    Stream<TYPE, ENT, UNIT> st;
    if (!ENT) te.read(g, a.teacher, a.r, r, row, true);

    // the largest of each of the step's kU rows of 32 vectors, into the maxima
    const auto put_maxima = [&](int b, float (&lm)[kU]) {
        if (G > 32 && log >= 5) {
            const int rows = (1 << log) >> 5;     // of 32 vectors in a chunk: 1, 2 or 4
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (u & (rows - 1)) lm[u] = fmaxf(lm[u], lm[u - 1]);
                if (((u + 1) & (rows - 1)) == 0) {
                    const uint32_t x = __reduce_max_sync(0xffffffffu, order_key<TYPE>(lm[u]));
                    const int at = (b + u * 32) >> log;
                    if (g.lane == 0 && at << log < nv) sm.keys[at] = x;
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = b + u * 32 + g.lane;
                uint32_t x = order_key<TYPE>(lm[u]);
#pragma unroll 1
                for (int o = 1; o < 1 << log; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
                if ((g.lane & ((1 << log) - 1)) == 0 && j < nv) sm.keys[j >> log] = x;
            }
        }
    };
    // a whole step inside the row
    const auto whole = [&](int b) { return b >= lo && b + kStep <= hi; };
#pragma unroll 1
    for (int b = g.warp * kStep; b < nv; b += kU * G) {
        [[maybe_unused]] float lm[kU];
        uint32_t later = 0;         // vectors that the straight way cannot do
        uint4 raw[kU];
        if (whole(b)) {
            if (MASK) {
                Keep keep[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int64_t e0 = (v0 + b + u * 32 + g.lane) * E - r.head;
                    keep[u] = words ? r.keep_word(e0) : row_keep<TYPE>(r, e0);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    raw[u] = __ldg(vecs + b + u * 32 + g.lane);
                    En::blank(raw[u], keep[u]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    raw[u] = __ldg(vecs + b + u * 32 + g.lane);
            }
        } else {
            // the row's first or last vectors, or a strided row
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = b + u * 32 + g.lane;
                raw[u] = En::absent_vector();
                if (j >= lo && j < hi && (!MASK || words)) {
                    raw[u] = __ldg(vecs + j);
                    if (MASK) En::blank(raw[u], r.keep_word((v0 + j) * E - r.head));
                } else if (j < nv) {
                    later |= 1u << u;
                }
            }
        }
        if constexpr (!ENT) {
            if (!st.add_step(raw, a.r.c2)) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (b + u * 32 + g.lane < nv) later |= 1u << u;
            }
        } else {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                float v[E];
                lm[u] = decode<TYPE>(raw[u], v, a.r.floor);
                if (!st.add(v, lm[u], a.r.c2)) later |= 1u << u;
            }
        }
        if (ENT && k > 0) put_maxima(b, lm);
        if (__any_sync(0xffffffffu, later)) {
            __syncwarp();
#pragma unroll 1
            while (later) {
                const int u = __ffs(later) - 1;
                later &= later - 1;
                const int j = b + u * 32 + g.lane;
                const auto x = row_vector<TYPE>(r, v0 + j);
                float v[E];
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = x.v[i];
                const float m = largest<TYPE>(v, a.r.floor);
                if (!st.add(v, m, a.r.c2)) st.far(x.v, m, a.r.c2);
                if (ENT && k > 0) atomicMax(sm.keys + (j >> log), order_key<TYPE>(m));
            }
            __syncwarp();
        }
    }
    Sums<TYPE> sum = st.done(a.r.c2);
    combine(g, sum, a.r.c2);     // its barriers also publish the maxima
    g.sync();
    bool valid = sum.s < kInf;

    float logz, entropy;
    int found = 0;
    bool lists = false;
    if (G > 32 && a.r.segs > 1) {
        lists = !a.flat;
        // leave the segment's part in the workspace; the last one joins
        const int64_t slot0 = row * a.r.segs;
        if (k > 0 && lists) {
            if (valid) found = best_entries<TYPE, MASK>(g, sm, r, v0, nv, k, log, a.cand_len);
            for (int i = g.t; i < k; i += G) a.lists[(slot0 + seg) * k + i] = i < found ? sm.best[i] : 0;
        } else if (k > 0) {
            uint32_t *to = a.maxima + row * a.row_chunks + (v0 >> log);
            for (int i = g.t; i < (nv + (1 << log) - 1) >> log; i += G) to[i] = sm.keys[i];
        }
        if (g.t == 0) {
            OutPartial p;
            p.z0 = sum.z0;
            p.s = sum.s;
            p.t = sum.t;
            p.pad = 0;
            a.partials[slot0 + seg] = p;
        }
        __threadfence();
        __syncthreads();
        if (g.t == 0) last = atomicAdd(a.tickets + row, 1u) == (uint32_t)a.r.segs - 1;
        __syncthreads();
        if (!last) return;
        __threadfence();
        if (g.t == 0) a.tickets[row] = 0;    // ready for the next call
        if (k > 0 && !lists)
            for (int i = g.t; i < (int)((all + (1 << log) - 1) >> log); i += G)
                sm.keys[i] = __ldcg(a.maxima + row * a.row_chunks + i);
        sum = Sums<TYPE>();
        for (int i = g.t; i < (int)segs; i += G) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(a.partials + slot0 + i));
            Sums<TYPE> o;
            o.z0 = f.x;
            o.s = f.y;
            o.t = f.z;
            const float z = max_nan(sum.z0, o.z0);
            if (sum.z0 != z) sum.move_to(z, a.r.c2);
            if (o.z0 != z) o.move_to(z, a.r.c2);
            sum.s += o.s;
            sum.t += o.t;
        }
        combine(g, sum, a.r.c2);
        g.sync();
        valid = sum.s < kInf;
    }
    normaliser<TYPE>(a.r, sum, logz, entropy);
    finish_row<TYPE, ENT>(g, a, r, te, row, logz, entropy);
    if constexpr (!ENT) return;
    if (k == 0) return;
    int64_t *ids = a.top_ids + row * k;
    float *lps = a.top_logp + row * k;
    found = 0;
    if (G == 32 && nv <= 32) {
        // one vector a lane: take the largest k times
        const auto x = row_vector<TYPE>(r, g.lane);
        uint32_t key[E];
#pragma unroll
        for (int i = 0; i < E; ++i) key[i] = valid ? order_key<TYPE>(x.v[i]) : 0u;
        for (; found < k; ++found) {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < E; ++i) m = max(m, key[i]);
            const uint32_t mx = __reduce_max_sync(0xffffffffu, m);
            if (mx == 0) break;
            const int src = __ffs(__ballot_sync(0xffffffffu, m == mx)) - 1;
            if (g.lane == src) {
                int at = E;
#pragma unroll
                for (int i = E - 1; i >= 0; --i) at = key[i] == mx ? i : at;
#pragma unroll
                for (int i = 0; i < E; ++i) key[i] = i == at ? 0u : key[i];
                ids[found] = g.lane * E + at - r.head;
                lps[found] = log_prob<TYPE>(a.r, key_value(mx), logz);
            }
        }
    } else if (valid) {
        if (lists) found = join_lists(g, sm, a, row);
        else found = best_entries<TYPE, MASK>(g, sm, r, 0, (int)all, k, log, a.cand_len);
        for (int i = g.t; i < found; i += G) {
            const uint64_t x = sm.best[i];
            const uint32_t at = 0xffffffffu - (uint32_t)x;
            int64_t id = at;
            if (lists) {     // a position in the row's lists
                const uint32_t local = 0xffffffffu - (uint32_t)__ldcg(a.lists + row * a.r.segs * k + at);
                id = (int64_t)(at / (uint32_t)k) * a.r.seg_vecs * E + local;
            }
            ids[i] = id - r.head;
            lps[i] = log_prob<TYPE>(a.r, key_value((uint32_t)(x >> 32)), logz);
        }
    }
    for (int i = found + g.t; i < k; i += G) {
        ids[i] = -1;
        lps[i] = valid ? -kInf : logz;
    }
}

template <int TYPE, int G, bool MASK, bool ENT, bool UNIT>
cudaError_t launch_forward(const OutForward &a, cudaStream_t stream) {
    const int64_t items = a.r.rows * a.r.segs;
    const int groups = kOutThreads / G;
    const size_t smem = (size_t)groups * a.group_bytes;
    auto *kernel = outcomes_forward<TYPE, G, MASK, ENT, UNIT>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3((unsigned)((items + groups - 1) / groups)), dim3(kOutThreads), smem,
                      stream, a);
}

template <int TYPE, int G, bool ENT, bool UNIT>
cudaError_t forward_mask(const OutForward &a, cudaStream_t stream) {
    return a.r.mask ? launch_forward<TYPE, G, true, ENT, UNIT>(a, stream)
                    : launch_forward<TYPE, G, false, ENT, UNIT>(a, stream);
}

template <int TYPE, int G>
cudaError_t forward_ent(const OutForward &a, cudaStream_t stream) {
    const bool ent = a.teacher.count == 0;
    if constexpr (TYPE == TN_TYPE_C64) {
        if (a.r.scale == 1.f)
            return ent ? forward_mask<TYPE, G, true, true>(a, stream) : forward_mask<TYPE, G, false, true>(a, stream);
    }
    return ent ? forward_mask<TYPE, G, true, false>(a, stream) : forward_mask<TYPE, G, false, false>(a, stream);
}

}  // namespace

template <int TYPE>
cudaError_t outcomes_forward_of(const OutForward &a, bool warp_rows, cudaStream_t stream) {
    return warp_rows ? forward_ent<TYPE, 32>(a, stream) : forward_ent<TYPE, kOutThreads>(a, stream);
}

}  // namespace tn
