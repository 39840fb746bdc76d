// Scores of outcome distributions, and the loss against a teacher: one pass
// over the rows.  Included by the translation unit of each entry type.
//
// Per row: log Z = ln sum exp(scale z), H = log Z - scale sum p z, log p of
// given entries, and the k largest entries with their indices.  A thread keeps a reference entry z0
// and, with d = scale log2(e) (z - z0),
//     s = sum 2^d,   t = sum 2^d d;
// then log Z = scale z0 + ln s, H = ln s - ln2 t / s and log p = scale (z - z0) -
// ln s.  z0 follows the
// largest entry seen only once that is more than 2^8 above it: any reference
// near the maximum will do, and a rescale on every new maximum would be a
// divergent branch in most steps.
//
// Alternatives cost the pass one maximum per chunk of vectors (a vector is 16
// bytes, a chunk what a warp reads in one step, or less of it for many
// alternatives).  Ordered by (value, lowest index first), the k best entries
// lie in the k best groups of any division into contiguous index ranges
// ordered by (largest entry, lowest range first): k groups that come before a
// group each hold an entry that comes before all of that group's.  So the k
// best chunks are found, and only those are read again.  In segments of a long
// row the maxima form a tree (of 32 chunks, of a segment), and the search goes
// down it.
//
// Rows of up to 4 KiB (where there are many, 16 KiB) are a warp's.  Longer ones
// are one CTA's, or cut into segments of one CTA each where there are few; a
// second, dependent kernel then joins the segments in order and searches for
// the alternatives.  It is a kernel of its own because the search is a few
// thousand instructions that only the first of a row's warps would run: beside
// the streaming loop they cost that loop its registers and its instruction
// cache.
//
// What bounds it.  32-bit entries: memory (2^26 amplitudes 83 us, 6.5 TB/s;
// 2048x50001 f32 67 us, 6.1 TB/s).  16-bit ones: twice the entries a byte, and
// neither memory nor issue slots are full (2048x50001 bf16 42 us, 4.8 TB/s; with
// alternatives 54 and 55 % of them): warps wait for their loads, 44 % of the
// most that an SM holds; without the entropy, for the loss, 39 us.
// Alternatives: their maxima, and the search, which is latency, about ten
// dependent steps (the same with one alternative 55 us, with 20 67; 1x32768 with
// 5 8.8 us, without 4.4).  Short rows: what a row costs besides its entries
// (20000 rows of 64 amplitudes 10 us, with 4 alternatives 15.6).
#pragma once

#include "outcomes.cuh"

namespace tn {

namespace {

constexpr int kU = 4;               // vectors of a thread's step
constexpr float kLag = 8.f;         // of the reference, in powers of two
constexpr float kFar = 4.253529586511730e37f;   // 2^125
constexpr float kTiny = 7.888609052210118e-31f; // 2^-100

// ---- running sums -----------------------------------------------------------

// The same for a weight below 2^-100 z.
__device__ __noinline__ float wide_distance(float v, float z, float c2) {
    return v == 0.f ? -__builtin_huge_valf()
                    : c2 * (lg2(__fdiv_rn(v * 0x1p100f, z * 0x1p-100f)) - 200.f);
}

// Distance of order value v from reference z in powers of two (amplitudes:
// of the weights' quotient, so that the reference itself is at 0 exactly; z is
// the larger there, and the logarithm of a quotient near 1 may be above 0.  A
// quotient below fp32's range counts where the scale is small).
template <int TYPE>
__device__ __forceinline__ float distance(float v, float z, float c2) {
    if constexpr (Entry<TYPE>::kReal) return (v - z) * c2;
    const float q = __fdiv_rn(v, z);
    if (q < 0x1p-100f && c2 < 1.f) return wide_distance(v, z, c2);
    return min_nan(c2 * lg2(q), 0.f);
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
// value) would overflow there, those below half of `floor` would not be told
// from absent ones, and the rounding of a ref beyond 2^31 (2^7 and more: masks
// written as -1e10) would itself be too large an exponent: ref = -inf then
// sends every vector through far(), which works with differences of logits.
// Different logits that far out differ by 2^7 powers of two at least, so the
// sums of smaller ones are dropped on the way back.  (A rounding of up to 80
// leaves room for sums; far() costs, 2048x50001 bf16 with one half filled 71
// against 46 us, and -1e9 stays out of it up to scale 4.)
//
// Amplitudes: the quotient w / z0 as q = w (1 / z0) with one Newton correction
// q + (w - q z0) / z0 (Markstein 1990), which makes z0 / z0 exactly 1.  z0 is
// at least 2^-100, for a finite reciprocal and a correction that is not lost.
// Where all weights are smaller and the scale is above 2, powers of quotients by
// that could vanish: inv = infinity then sends every vector through far(), which
// divides.  z0 moves where a weight's power is 2^8 above its own, at a quotient
// of 2^(8 / scale) (256 at most).  From scale 2^12 on, where the logarithm's error
// (2^-22) counts, far() takes all and moves at each larger weight.  Up to scale 1/4,
// where a weight far below another counts beside it, z0 is 1 at most, so that no
// quotient is below its weight, and powers (2^32 at most) need no nearer one.
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
    // Whether a logit, of the rounded product r, can be the reference of the
    // straight way.  False for NaN and infinities.
    static __device__ __forceinline__ bool near(float lm, float r, float c2, float floor) {
        return fabsf(r) <= kFar && lm >= 0.5f * floor && fabsf(fmaf(lm, c2, -r)) <= 80.f;
    }
    // The reference for a largest weight.
    static __device__ __forceinline__ float first(float lm, float c2) {
        if (!UNIT && c2 <= 0.25f && lm > 1.f) return 1.f;
        return lm < kTiny ? kTiny : lm;
    }
    // Whether a row's largest weight is one for far().
    static __device__ __forceinline__ bool divided(float lm, float c2) {
        return c2 > 2.f && (lm < kTiny || c2 >= 4096.f);
    }
    // Add a vector: v its order values, for real logits not below `floor`, lm
    // their largest before that.  False if it is one for far().
    __device__ __forceinline__ bool add(const float (&v)[E], float lm, const OutRows &a) {
        const float c2 = a.c2;
        if constexpr (En::kReal) {
            if (!(fmaf(lm, c2, -ref) <= kLag)) {
                if (lm == absent<TYPE>()) return true;
                const float r = lm * c2;
                if (!near(lm, r, c2, a.floor) || (ref == -__builtin_huge_valf() && s.x != 0.f && !(lm > z0)))
                    return false;
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
            if (UNIT ? !(lm * inv <= 256.f) : !(lm * inv < a.lag)) {
                if (lm == 0.f) return true;
                if (!UNIT && divided(lm, c2) && inv == __builtin_huge_valf()) return false;
                const float z = first(lm, c2);
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
    __device__ __forceinline__ bool add_step(const uint4 (&raw)[kU], const OutRows &a) {
        const float c2 = a.c2;
        static_assert(!ENT, "the entropy's sum needs a near reference");
        constexpr float kBig = 0x1p100f;
        constexpr float kInf = __builtin_huge_valf();
        if (En::kReal ? ref == -kInf : inv == kInf) {
            if (s.x != 0.f || s.y != 0.f) return false;   // (far out, or divided)
            float lm = vector_max<TYPE>(raw[0]);
#pragma unroll
            for (int u = 1; u < kU; ++u) lm = max_nan(lm, vector_max<TYPE>(raw[u]));
            if (lm == absent<TYPE>()) return true;
            if constexpr (En::kReal) {
                const float r = lm * c2;
                if (!near(lm, r, c2, a.floor)) return false;
                ref = r;
                z0 = lm;
            } else {
                if (!(lm < kInf) || (!UNIT && divided(lm, c2))) return false;
                z0 = first(lm, c2);
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
    // the same for logits far out and weights to be divided: v as they are
    __device__ __forceinline__ void far(const float (&v)[E], float lm, float c2) {
        if (!(lm <= z0)) {
            move_by(z0 == absent<TYPE>() ? 0.f : distance<TYPE>(z0, lm, c2));
            z0 = lm;
        }
        ref = -__builtin_huge_valf();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = distance<TYPE>(v[i], z0, c2);
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
        if (En::kReal && ref != -__builtin_huge_valf()) {
            const float left = fmaf(z0, c2, -ref), one = ex2(left);
            if (a.s == one && (!ENT || a.t == one * left)) {   // of one entry: exactly 1 and 0
                a.s = 1.f;
                a.t = 0.f;
            } else {
                a.move_by(-left);
            }
        }
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

// Positions of the keys before a cut, of n <= PER G keys in shared memory, in
// ascending order.  Every thread keeps PER consecutive keys in registers; a
// histogram of 256 bins over the range in question finds the bin with the k-th
// key, which is the cut unless too many keys share it: then it is the next
// range (a factor of 256 smaller each time; one or two are the rule).
template <int PER, int G>
__device__ __noinline__ Cut cut_keys(Group<G> g, const uint32_t *keys, int n, int k, int most, uint32_t *out,
                                     uint32_t *bins) {
    uint32_t key[PER];
    const int i0 = g.t * PER;
    uint32_t mx = 0, nz = 0, mn = 0xffffffffu;     // mn: smallest but 0, less 1
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = i0 + i < n ? keys[i0 + i] : 0u;
        mx = max(mx, key[i]);
        mn = min(mn, key[i] - 1);
        nz += key[i] != 0;
    }
    mx = g.max(mx);
    uint32_t lo = ~g.max(~mn) + 1, hi = mx, above = 0;
    nz = g.sum(nz);
    Cut c = {1u, 0xffffffffu, nz};
    while (nz > (uint32_t)k) {
        const int shift = max(0, 24 - __clz((hi - lo) | 1));
        for (int i = g.t; i < 256; i += G) bins[i] = 0;
        g.sync();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] >= lo && key[i] <= hi) atomicAdd(bins + ((key[i] - lo) >> shift), 1u);
        g.sync();
        // every warp on its own: lane l has the bins 255 - 8 l .. 248 - 8 l
        const uint4 b0 = reinterpret_cast<const uint4 *>(bins)[63 - 2 * g.lane];
        const uint4 b1 = reinterpret_cast<const uint4 *>(bins)[62 - 2 * g.lane];
        const uint32_t bin[8] = {b0.w, b0.z, b0.y, b0.x, b1.w, b1.z, b1.y, b1.x};
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += bin[i];
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (g.lane >= o) upto += x;
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, above + upto >= (uint32_t)k)) - 1;
        uint32_t before = above + upto - mine, at = 0;
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (at == (uint32_t)i && before + bin[i] < (uint32_t)k) {
                before += bin[i];
                ++at;
            }
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) in = at == (uint32_t)i ? bin[i] : in;
        at += 8 * g.lane;
        before = __shfl_sync(0xffffffffu, before, src);
        in = __shfl_sync(0xffffffffu, in, src);
        at = 255 - __shfl_sync(0xffffffffu, at, src);
        c.thr = lo + (at << shift);
        if (before + in <= (uint32_t)most) {
            c.count = before + in;
            break;
        }
        if (shift == 0) {
            c.ties = k - before;
            c.count = k;
            break;
        }
        g.sync();      // (all have read the bins)
        above = before;
        lo = c.thr;
        hi = lo + min(hi - lo, (1u << shift) - 1);
    }
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        gt += key[i] > c.thr;
        eq += key[i] == c.thr;
    }
    uint32_t pg = gt, pe = eq;
    g.scan2(pg, pe);
    uint32_t at = pg + min(pe, c.ties);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (key[i] > c.thr || (key[i] == c.thr && pe++ < c.ties)) out[at++] = i0 + i;
    g.sync();
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

// ---- the end of a row -------------------------------------------------------

// What a row's sums say: the reference's logit z0, ls = ln s (-inf: an empty
// row) and H; NaN where an entry was NaN or +inf.
struct Norm {
    float z0, ls, entropy;
    __device__ __forceinline__ float logz(const OutRows &r) const {
        return __fadd_rn(__fmul_rn(r.scale, z0), ls);
    }
};

template <int TYPE>
__device__ __forceinline__ Norm normaliser(const Sums<TYPE> &a) {
    constexpr float kInf = __builtin_huge_valf();
    Norm n;
    n.z0 = Entry<TYPE>::kReal ? a.z0 : logf(a.z0);
    if (a.s == 0.f) {
        n.ls = -kInf;
        n.entropy = 0.f;
    } else if (a.s < kInf) {
        n.ls = logf(a.s);
        n.entropy = n.ls - kLn2 * (a.t / a.s);
    } else {
        n.ls = n.entropy = __int_as_float(0x7fffffff);
    }
    return n;
}

// From the reference, not from log Z, whose rounding is ln V's size and more where
// scale z is large (64 at 1e9: a row of nothing but a mask's fill).
template <int TYPE>
__device__ __forceinline__ float log_prob(const OutRows &r, float v, const Norm &n) {
    // not fused: a row's only entry has log p = 0 exactly
    return __fadd_rn(__fmul_rn(r.scale, (Entry<TYPE>::kReal ? v : logf(v)) - n.z0), -n.ls);
}

// The loss of a row by one warp.
template <int TYPE>
__device__ __forceinline__ float teacher_loss(int count, const OutRows &r, const Teacher &te, const Norm &norm) {
    constexpr float kInf = __builtin_huge_valf();
    float loss = 0.f, bad = 0.f;
#pragma unroll 1
    for (int j = threadIdx.x % 32; j < count; j += 32) {
        if (te.id[j] == -2) bad = __int_as_float(0x7fffffff);
        if (te.id[j] >= 0 && te.q[j] != 0.f) {
            const float v = te.value[j];
            const float lp = v == absent<TYPE>() ? -kInf : log_prob<TYPE>(r, v, norm);
            loss += te.q[j] * (te.logq[j] - lp);
        }
    }
    if (norm.ls == -kInf) loss = 0.f;
    loss += bad;
#pragma unroll
    for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    return loss;
}

template <int TYPE, bool ENT, int G>
__device__ __forceinline__ void finish_row(Group<G> &g, const OutForward &a, const Row<TYPE> &r,
                                           Teacher &te, int64_t row, const Norm &norm) {
    constexpr float kInf = __builtin_huge_valf();
    if (g.t == 0) a.logz[row] = norm.logz(a.r);
    if constexpr (ENT) {
        if (g.t == 0) a.entropy[row] = norm.entropy;
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
                lp = v == absent<TYPE>() ? -kInf : log_prob<TYPE>(a.r, v, norm);
            }
            a.logp[row * a.n_given + j] = lp;
        }
    } else {
        if (g.warp == 0) {
            te.normalise(a.teacher);
            const float loss = teacher_loss<TYPE>(a.teacher.count, a.r, te, norm);
            if (g.t == 0) a.loss[row] = loss;
        }
    }
}

// Shared memory of a group (all offsets multiples of 16 bytes).
struct Scratch {
    uint32_t *keys;       // maxima (key_words)
    uint64_t *cand;       // candidates (cand_len)
    uint64_t *best;       // the k best, in order
    uint32_t *pos, *pos2; // chunks: out_most(k) each, of a tree out_room(k)
    uint32_t *n;          // counters
    uint32_t *lists;      // of a tree: segments and groups of chunks
    __device__ __forceinline__ Scratch(unsigned char *base, const OutForward &a) {
        const int kk = (a.n_top + 3) / 4 * 4, pp = ((a.tree ? out_room(a.n_top) : out_most(a.n_top)) + 3) / 4 * 4;
        keys = reinterpret_cast<uint32_t *>(base);
        cand = reinterpret_cast<uint64_t *>(keys + a.key_words);
        best = cand + a.cand_len;
        pos = reinterpret_cast<uint32_t *>(best + kk);
        pos2 = pos + pp;
        n = pos2 + pp;
        lists = n + 4;
    }
    // First k (up to `most`) of keys[0 .. nk) into pos; returns their number,
    // `least` a lower bound of the k best entries.
    template <int G>
    __device__ __forceinline__ int cut(Group<G> &g, int nk, int k, int most, uint32_t &least) const {
        uint32_t *bins = reinterpret_cast<uint32_t *>(cand);
        if (G > 32 && nk <= 256) {      // few enough for one warp, without barriers
            if (g.t < 32) {
                const Cut c = cut_keys<8>(Group<32>(nullptr), keys, nk, k, most, pos, bins);
                if (g.t == 0) {
                    n[1] = c.count;
                    n[2] = c.thr;
                }
            }
            g.sync();
            least = n[2];
            return (int)n[1];
        }
        const Cut c = cut_keys<G == 32 ? kOutWarpVecs / 32 : kOutTree / G>(g, keys, nk, k, most, pos, bins);
        least = c.thr;
        return (int)c.count;
    }
    __device__ __forceinline__ void offer(uint32_t key, uint32_t index, int len) const {
        const uint32_t at = atomicAdd(n, 1u);
        if (at < (uint32_t)len) cand[at] = candidate(key, index);
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

// largest order value of vector j
template <int TYPE>
__device__ __forceinline__ float row_vector_max(const Row<TYPE> &r, int64_t j) {
    const auto x = row_vector<TYPE>(r, j);
    float lm = absent<TYPE>();
#pragma unroll
    for (int e = 0; e < Entry<TYPE>::E; ++e) lm = fmaxf(lm, x.v[e]);
    return lm;
}

// The k best entries of a row into sm.best, from the nc chunks of 2^log
// vectors in sm.pos (ascending; `least` a lower bound of the k best), as
// candidates whose index is ((place in sm.pos << log) + vector) E + entry.
// Returns their number, or -1: too many entries at the bound.
template <int TYPE, bool MASK, int G>
__device__ __forceinline__ int best_of_chunks(Group<G> &g, const Scratch &sm, const Row<TYPE> &r, int nc,
                                              uint32_t least, int k, int log, int cand_len) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr int kAgain = G == 32 ? 2 : 8;     // vectors in flight per thread
    const int low = (1 << log) - 1, work = nc << log;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    // vectors with an entry of at least `bar` (the lowest present value at the
    // lowest), then those entries
    const float bar = fmaxf(key_value(least), En::kReal ? -3.402823466e38f : 1.401298464e-45f);
    uint32_t *list = reinterpret_cast<uint32_t *>(sm.cand + cand_len / 2);   // cand_len places
    const bool words = !MASK || r.mask_words();
    if (g.t == 0) sm.n[0] = sm.n[3] = 0;
    g.sync();
    const auto keep_vector = [&](int i) {
        const uint32_t at = atomicAdd(sm.n + 3, 1u);
        if (at < (uint32_t)cand_len) list[at] = i;
    };
#pragma unroll 1
    for (int b = g.t; b - g.t < work; b += kAgain * G) {
        uint4 q[kAgain];
        uint32_t odd = 0;       // vectors to be read entry by entry
#pragma unroll
        for (int u = 0; u < kAgain; ++u) {
            const int i = b + u * G;
            q[u] = En::absent_vector();
            if (i >= work) continue;
            const int64_t j = ((int64_t)sm.pos[i >> log] << log) + (i & low);
            if (j >= all) continue;
            const int64_t e0 = j * E - r.head;
            if (words && r.inside(e0)) {
                q[u] = r.raw(e0);
                if (MASK) En::blank(q[u], r.keep_word(e0));
            } else {
                odd |= 1u << u;
            }
        }
#pragma unroll
        for (int u = 0; u < kAgain; ++u) {
            if (b - g.t + u * G >= work) break;
            if (vector_max<TYPE>(q[u]) >= bar) keep_vector(b + u * G);
        }
#pragma unroll 1
        for (; odd; odd &= odd - 1) {
            const int i = b + (__ffs(odd) - 1) * G;
            if (row_vector_max<TYPE>(r, ((int64_t)sm.pos[i >> log] << log) + (i & low)) >= bar) keep_vector(i);
        }
    }
    g.sync();
    const int nl = (int)sm.n[3];
    if (nl > cand_len) return -1;
#pragma unroll 1
    for (int i = g.t; i < nl * E; i += G) {
        const int x = (int)list[i / E], e = i % E;
        const int64_t at = (((int64_t)sm.pos[x >> log] << log) + (x & low)) * E - r.head + e;
        const float v = at >= 0 && at < r.cols ? row_value<TYPE>(r, at) : absent<TYPE>();
        if (v >= bar) sm.offer(order_key<TYPE>(v), x * E + e, cand_len / 2);
    }
    g.sync();
    const int n = (int)sm.n[0];
    if (n > cand_len / 2) return -1;
    return rank_candidates(g, sm, n, k);
}

// The same from exactly the k best chunks, whatever lies at the bound (long
// runs of equal or of sorted entries): the k best of their vectors, then of
// those vectors' entries.
template <int TYPE, int G>
__device__ __noinline__ int best_of_exact_chunks(Group<G> g, const Scratch sm, const Row<TYPE> r, int nc, int k,
                                                 int log) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    const int low = (1 << log) - 1;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    uint32_t *sub = reinterpret_cast<uint32_t *>(sm.cand);
    g.sync();
#pragma unroll 1
    for (int i = g.t; i < nc << log; i += G) {
        const int64_t j = ((int64_t)sm.pos[i >> log] << log) + (i & low);
        sub[i] = j < all ? order_key<TYPE>(row_vector_max<TYPE>(r, j)) : 0u;
    }
    g.sync();
    const int nv = select(g, [=](int i) { return sub[i]; }, nc << log, k, sm.pos2);
#pragma unroll 1
    for (int i = g.t; i < nv * E; i += G) {
        const int x = (int)sm.pos2[i / E], e = i % E;
        const int64_t at = (((int64_t)sm.pos[x >> log] << log) + (x & low)) * E - r.head + e;
        const float v = at >= 0 && at < r.cols ? row_value<TYPE>(r, at) : absent<TYPE>();
        const uint32_t key = order_key<TYPE>(v);
        sm.cand[i] = key ? candidate(key, x * E + e) : 0;
    }
    g.sync();
    return rank_candidates(g, sm, nv * E, k);
}

// The k best entries of a row whose nk chunk maxima are in sm.keys.
template <int TYPE, bool MASK, int G>
__device__ __forceinline__ int best_entries(Group<G> &g, const Scratch &sm, const Row<TYPE> &r, int nk, int k,
                                            int log, int cand_len) {
    uint32_t least;
    const int nc = sm.cut(g, nk, k, log ? out_most(k) : k, least);
    int found = best_of_chunks<TYPE, MASK>(g, sm, r, nc, least, k, log, cand_len);
    if (found < 0) {
        g.sync();
        const int exact = sm.cut(g, nk, k, k, least);
        found = best_of_exact_chunks<TYPE>(g, sm, r, exact, k, log);
    }
    return found;
}

// Alternative i of the row, from sm.best.
template <int TYPE>
__device__ __forceinline__ void put_alternative(const OutForward &a, const Row<TYPE> &r, const Scratch &sm, int i,
                                                int log, const Norm &norm, int64_t *ids, float *lps) {
    constexpr int E = Entry<TYPE>::E;
    const uint64_t c = sm.best[i];
    const uint32_t x = 0xffffffffu - (uint32_t)c, j = x / E;
    ids[i] = (((int64_t)sm.pos[j >> log] << log) + (j & ((1 << log) - 1))) * E + x % E - r.head;
    lps[i] = log_prob<TYPE>(a.r, key_value((uint32_t)(c >> 32)), norm);
}

// ---- the kernels ------------------------------------------------------------

// SHORT: rows of one vector a lane, whose alternatives need no search.
template <int TYPE, int G, bool SHORT, bool MASK, bool ENT, bool UNIT>
__global__ void __launch_bounds__(kOutThreads, G == 32 && !SHORT ? 6 : kOutCtas)
outcomes_forward(const __grid_constant__ OutForward a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr int kGroups = kOutThreads / G;
    constexpr float kInf = __builtin_huge_valf();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t red[4 * kOutThreads / 32];
    constexpr int kTeacher = ENT ? 16 : TN_OUTCOMES_MAX_IDS * 20 + 16;
    __shared__ __align__(16) unsigned char teachers[kGroups * kTeacher];
    Teacher te(teachers + threadIdx.x / G * kTeacher, ENT ? 0 : a.teacher.count);
    pdl_trigger();
    Group<G> g(red);
    const uint32_t item = blockIdx.x * kGroups + threadIdx.x / G, segs = (uint32_t)a.r.segs;
    const int64_t row = G == 32 ? item : item / segs;
    const int64_t seg = G == 32 ? 0 : item % segs;
    const Scratch sm(smem + (G == 32 ? (size_t)(threadIdx.x / G) * a.group_bytes : 0), a);
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;

    const Row<TYPE> r(a.r, row);
    const int64_t v0 = seg * a.r.seg_vecs;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    const int64_t v1 = min(all, v0 + a.r.seg_vecs);
    const int nv = static_cast<int>(max((int64_t)0, v1 - v0));   // may be 0 in a row's last segment
    const int k = ENT ? a.n_top : 0;
    const int log = a.chunk_log;                // one maximum per 2^log vectors
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

    // The largest entries of the step's chunks, as they are; keys are made of
    // them once the row is read (a warp's rows: at once).
    const auto put_maxima = [&](int b, float (&lm)[kU]) {
        float *maxima = reinterpret_cast<float *>(sm.keys);
        if (G > 32 && log == kOutChunkLog) {
            const float x = warp_max(fmaxf(fmaxf(lm[0], lm[1]), fmaxf(lm[2], lm[3])));
            if (g.lane == 0) maxima[b >> kOutChunkLog] = x;
        } else if (G > 32 && log >= 5) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (log == 6 && (u & 1) == 0) continue;
                const float x = warp_max(log == 6 ? fmaxf(lm[u], lm[u - (u & 1)]) : lm[u]);
                const int at = (b + u * 32) >> log;
                if (g.lane == 0 && at << log < nv) maxima[at] = x;
            }
        } else {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = b + u * 32 + g.lane;
                float x = lm[u];
#pragma unroll 1
                for (int o = 1; o < 1 << log; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                if ((g.lane & ((1 << log) - 1)) == 0 && j < nv) {
                    if (G == 32) sm.keys[j >> log] = order_key<TYPE>(x);
                    else maxima[j >> log] = x;
                }
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
                    raw[u] = __ldcg(vecs + b + u * 32 + g.lane);
                    En::blank(raw[u], keep[u]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    raw[u] = __ldcg(vecs + b + u * 32 + g.lane);
            }
        } else {
            // the row's first or last vectors, or a strided row
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = b + u * 32 + g.lane;
                raw[u] = En::absent_vector();
                if (j >= lo && j < hi && (!MASK || words)) {
                    raw[u] = __ldcg(vecs + j);
                    if (MASK) En::blank(raw[u], r.keep_word((v0 + j) * E - r.head));
                } else if (j < nv) {
                    later |= 1u << u;
                }
            }
        }
        if constexpr (!ENT) {
            if (!st.add_step(raw, a.r)) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (b + u * 32 + g.lane < nv) later |= 1u << u;
            }
        } else {
#pragma unroll
            for (int u = 0; u < (SHORT ? 1 : kU); ++u) {
                float v[E];
                lm[u] = decode<TYPE>(raw[u], v, a.r.floor);
                if (!st.add(v, lm[u], a.r)) later |= 1u << u;
            }
        }
        if (__any_sync(0xffffffffu, later)) {
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
                if (!st.add(v, m, a.r)) st.far(x.v, m, a.r.c2);
                if constexpr (ENT) {
#pragma unroll
                    for (int i = 0; i < kU; ++i) lm[i] = i == u ? fmaxf(lm[i], m) : lm[i];
                }
            }
            __syncwarp();
        }
        if (ENT && !SHORT && k > 0) put_maxima(b, lm);
    }
    Sums<TYPE> sum = st.done(a.r.c2);
    combine(g, sum, a.r.c2);     // its barriers also publish the maxima
    g.sync();
    if (G > 32 && a.finish) {
        // leave the segment's part for the second kernel
        if (g.t == 0) {
            OutPartial p;
            p.z0 = sum.z0;
            p.s = sum.s;
            p.t = sum.t;
            p.pad = 0;
            a.partials[row * segs + seg] = p;
        }
        if (ENT && k > 0) {
            const int nc = (nv + (1 << log) - 1) >> log;
            uint32_t *to = a.maxima + (row * segs + seg) * a.seg_chunks;
            for (int i = g.t; i < a.seg_chunks; i += G) {
                const uint32_t x = i < nc ? order_key<TYPE>(__uint_as_float(sm.keys[i])) : 0u;
                to[i] = x;
                sm.keys[i] = x;
            }
            if (a.tree) {
                g.sync();
                // the maxima of 32 chunks, and of the segment
                uint32_t *up = a.supers + (row * segs + seg) * 33;
                uint32_t top = 0;
                for (int i = g.warp; i < 32; i += Group<G>::kWarps) {
                    const int at = i * 32 + g.lane;
                    const uint32_t x = __reduce_max_sync(0xffffffffu, at < nc ? sm.keys[at] : 0u);
                    if (g.lane == 0) up[1 + i] = x;
                    top = max(top, x);
                }
                top = g.max(top);
                if (g.t == 0) up[0] = top;
            }
        }
        return;
    }
    const Norm norm = normaliser<TYPE>(sum);
    finish_row<TYPE, ENT>(g, a, r, te, row, norm);
    if constexpr (ENT && G == 32) {
        if (k == 0) return;
        const bool valid = sum.s < kInf;
        int64_t *ids = a.top_ids + row * k;
        float *lps = a.top_logp + row * k;
        int found = 0;
        if constexpr (SHORT) {
            // one vector a lane: take the largest k times; lane i has the key of
            // alternative i until their log p are due, 32 at once
            uint32_t mine = 0;
            const auto put_log_probs = [&](int first, int end) {
                if (first + g.lane < end) lps[first + g.lane] = log_prob<TYPE>(a.r, key_value(mine), norm);
            };
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
                }
                if ((found & 31) == g.lane) mine = mx;
                if ((found & 31) == 31) put_log_probs(found - 31, found + 1);
            }
            put_log_probs(found & ~31, found);
        } else if (valid) {
            g.sync();
            found = best_entries<TYPE, MASK>(g, sm, r, (nv + (1 << log) - 1) >> log, k, log, a.cand_len);
            for (int i = g.t; i < found; i += G) put_alternative<TYPE>(a, r, sm, i, log, norm, ids, lps);
        }
        for (int i = found + g.t; i < k; i += G) {
            ids[i] = -1;
            lps[i] = valid ? -kInf : norm.ls;
        }
    }
}

// The maxima of a row with a tree: of segment i, of group i % 32 of 32 chunks
// of the segment list[i / 32], or of chunk i % 32 of the group list[i / 32]
// (as segment 32 + group), 0 for none.
struct Tree {
    const uint32_t *supers, *maxima;
    int chunks;             // of a segment
    const uint32_t *list;
    __device__ __forceinline__ int chunk(int i) const {
        const uint32_t x = list[i >> 5], c = (x & 31) * 32 + (i & 31);
        return c < (uint32_t)chunks ? (int)((x >> 5) * chunks + c) : -1;
    }
    __device__ __forceinline__ uint32_t at(int level, int i) const {
        if (level == 0) return __ldcg(supers + (int64_t)i * 33);
        if (level == 1) return __ldcg(supers + (int64_t)list[i >> 5] * 33 + 1 + (i & 31));
        const int c = chunk(i);
        return c < 0 ? 0u : __ldcg(maxima + c);
    }
};

// A lower bound of the k best entries from n maxima of a level, taken together
// as many in a row as leaves kOutTree of them; 1 if they are not enough.
template <int G>
__device__ __noinline__ uint32_t tree_bound(Group<G> g, const Scratch sm, const Tree tree, int level, int n, int k) {
    const int per = (n + kOutTree - 1) / kOutTree, nk = (n + per - 1) / per;
#pragma unroll 1
    for (int i = g.t; i < nk; i += G) {
        uint32_t x = 0;
#pragma unroll 4
        for (int j = i * per; j < min(n, (i + 1) * per); ++j) x = max(x, tree.at(level, j));
        sm.keys[i] = x;
    }
    g.sync();
    uint32_t least;
    sm.cut(g, nk, k, out_most(k), least);
    g.sync();
    return least;
}

// The chunks to read again of a row with a tree of maxima, into sm.pos in
// ascending order: the segments with a maximum of at least a bound, their
// groups of 32 chunks, those groups' chunks.  The bound is a cut of the first
// level that has four times as many maxima as there are alternatives (about
// 1.15 k chunks lie above it then, unless entries are equal or sorted).  Returns
// their number, or -1: more than there is room for.
template <int G>
__device__ __noinline__ int chunks_of_tree(Group<G> g, const Scratch sm, const OutForward &a, int64_t row,
                                           uint32_t &least) {
    const int k = a.n_top, segs = (int)a.r.segs, room = out_room(k);
    uint32_t *groups = sm.lists + kOutList;
    Tree tree = {a.supers + row * segs * 33, a.maxima + row * segs * a.seg_chunks, a.seg_chunks, sm.lists};
    // the n maxima of a level that reach the bound
    const auto gather = [&](int level, int n, uint32_t *out, int len) {
        if (g.t == 0) sm.n[0] = 0;
        g.sync();
#pragma unroll 4
        for (int i = g.t; i < n; i += G)
            if (tree.at(level, i) >= least) {
                const uint32_t at = atomicAdd(sm.n, 1u);
                if (at < (uint32_t)len)
                    out[at] = level == 0 ? i : level == 1 ? tree.list[i >> 5] * 32 + (i & 31) : tree.chunk(i);
            }
        g.sync();
        const int found = (int)min(sm.n[0], 0x7fffffffu);
        g.sync();      // (all have read it: the next level starts by clearing it)
        return found;
    };
    least = 1;
    if (segs >= 4 * k) least = tree_bound(g, sm, tree, 0, segs, k);
    const int ns = gather(0, segs, sm.lists, kOutList);
    if (ns > kOutList) return -1;
    if (least == 1 && ns * ((a.seg_chunks + 31) / 32) >= 4 * k) least = tree_bound(g, sm, tree, 1, ns * 32, k);
    const int ng = gather(1, ns * 32, groups, kOutList);
    if (ng > kOutList) return -1;
    tree.list = groups;
    if (least == 1) least = tree_bound(g, sm, tree, 2, ng * 32, k);
    const int n = gather(2, ng * 32, sm.pos2, room);
    if (n > room) return -1;
#pragma unroll 1
    for (int i = g.t; i < n; i += G) {
        const uint32_t x = sm.pos2[i];
        int at = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) at += sm.pos2[j] < x;
        sm.pos[at] = x;
    }
    g.sync();
    return n;
}

// Exactly the k best chunks of such a row.
template <int G>
__device__ __noinline__ int exact_chunks_of_tree(Group<G> g, const Scratch sm, const OutForward &a, int64_t row) {
    const int k = a.n_top, segs = (int)a.r.segs, chunks = a.seg_chunks;
    const uint32_t *supers = a.supers + row * segs * 33;
    const uint32_t *maxima = a.maxima + row * segs * chunks;
    const uint32_t *pos = sm.pos;
    g.sync();
    const int ns = select(g, [=](int i) { return __ldcg(supers + (int64_t)i * 33); }, segs, k, sm.pos);
    const int nc = select(g, [=](int i) { return __ldcg(maxima + (int64_t)pos[i / chunks] * chunks + i % chunks); },
                          ns * chunks, k, sm.pos2);
#pragma unroll 1
    for (int i = g.t; i < nc; i += G) {
        const int x = (int)sm.pos2[i];
        sm.pos2[i] = pos[x / chunks] * chunks + x % chunks;
    }
    g.sync();
#pragma unroll 1
    for (int i = g.t; i < nc; i += G) sm.pos[i] = sm.pos2[i];
    g.sync();
    return nc;
}

// What follows the streaming kernel for rows in segments or with
// alternatives: a group a row joins the segments' sums in order and searches.
// It waits for memory and for itself most of the time (about ten dependent
// steps), so many rows are better served by a warp each, all at once, than by
// a CTA each in turn.
template <int G>
constexpr int finish_threads() { return G == 32 ? 128 : G; }
template <int TYPE, int G, int CTAS, bool MASK, bool ENT>
__global__ void __launch_bounds__(finish_threads<G>(), CTAS) outcomes_finish(const __grid_constant__ OutForward a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr float kInf = __builtin_huge_valf();
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kGroups = finish_threads<G>() / G;
    __shared__ uint32_t red[4 * G / 32];
    constexpr int kTeacher = ENT ? 16 : TN_OUTCOMES_MAX_IDS * 20 + 16;
    __shared__ __align__(16) unsigned char teacher[kGroups * kTeacher];
    Teacher te(teacher + threadIdx.x / G * kTeacher, ENT ? 0 : a.teacher.count);
    pdl_trigger();
    Group<G> g(red);
    const int64_t row = blockIdx.x * kGroups + threadIdx.x / G;
    const int segs = (int)a.r.segs, k = ENT ? a.n_top : 0, log = a.chunk_log;
    const Scratch sm(smem + threadIdx.x / G * a.group_bytes, a);
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;
    const Row<TYPE> r(a.r, row);
    // (the workspace is read past the L1 cache: this grid may have started while
    // the previous call's was still filling it)
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g.t < segs) f = __ldcg(reinterpret_cast<const float4 *>(a.partials + row * segs + g.t));
    const int nk = segs * a.seg_chunks;
    if (ENT && k > 0 && !a.tree) {
#pragma unroll 4
        for (int i = g.t; i < nk; i += G) sm.keys[i] = __ldcg(a.maxima + row * nk + i);
    }
    if (!ENT) te.read(g, a.teacher, a.r, r, row, true);
    Sums<TYPE> sum;
#pragma unroll 1
    for (int i = g.t; i < segs; i += G) {
        Sums<TYPE> o;
        o.z0 = f.x;
        o.s = f.y;
        o.t = f.z;
        const float z = max_nan(sum.z0, o.z0);
        if (sum.z0 != z) sum.move_to(z, a.r.c2);
        if (o.z0 != z) o.move_to(z, a.r.c2);
        sum.s += o.s;
        sum.t += o.t;
        if (i + G < segs) f = __ldcg(reinterpret_cast<const float4 *>(a.partials + row * segs + i + G));
    }
    combine(g, sum, a.r.c2);
    g.sync();
    const bool valid = sum.s < kInf;
    const Norm norm = normaliser<TYPE>(sum);
    finish_row<TYPE, ENT>(g, a, r, te, row, norm);
    if constexpr (ENT) {
        if (k == 0) return;
        int64_t *ids = a.top_ids + row * k;
        float *lps = a.top_logp + row * k;
        int found = 0;
        if (valid && !a.tree) {
            found = best_entries<TYPE, MASK>(g, sm, r, nk, k, log, a.cand_len);
        } else if (valid) {
            uint32_t least;
            const int nc = chunks_of_tree(g, sm, a, row, least);
            found = nc < 0 ? -1 : best_of_chunks<TYPE, MASK>(g, sm, r, nc, least, k, log, a.cand_len);
            if (found < 0) {
                const int exact = exact_chunks_of_tree(g, sm, a, row);
                found = best_of_exact_chunks<TYPE>(g, sm, r, exact, k, log);
            }
        }
        for (int i = g.t; i < found; i += G) put_alternative<TYPE>(a, r, sm, i, log, norm, ids, lps);
        for (int i = found + g.t; i < k; i += G) {
            ids[i] = -1;
            lps[i] = valid ? -kInf : norm.ls;
        }
    }
}

template <class Kernel>
cudaError_t launch_rows(Kernel *kernel, int64_t ctas, int threads, size_t smem, const OutForward &a,
                        cudaStream_t stream) {
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3((unsigned)ctas), dim3(threads), smem, stream, a);
}

template <int TYPE, bool MASK, bool ENT, bool UNIT>
cudaError_t launch_forward(const OutForward &a, bool warp_rows, cudaStream_t stream) {
    if (warp_rows) {
        const int groups = kOutThreads / 32;
        const int64_t ctas = (a.r.rows + groups - 1) / groups;
        if (ENT && a.r.seg_vecs <= 32)
            return launch_rows(outcomes_forward<TYPE, 32, ENT, MASK, ENT, UNIT>, ctas, kOutThreads, 0, a, stream);
        return launch_rows(outcomes_forward<TYPE, 32, false, MASK, ENT, UNIT>, ctas, kOutThreads,
                           (size_t)groups * a.group_bytes, a, stream);
    }
    const size_t keys = ENT && a.n_top > 0 ? (size_t)(a.seg_chunks + 3) / 4 * 16 : 0;
    cudaError_t e = launch_rows(outcomes_forward<TYPE, kOutThreads, false, MASK, ENT, UNIT>, a.r.rows * a.r.segs, kOutThreads,
                                keys, a, stream);
    if (e != cudaSuccess || !a.finish) return e;
    // Many rows: a warp each, if their maxima fit its registers; few: as many
    // threads as help one, with all their registers where a row has an SM, or two
    // such CTAs an SM where the search is long.  A warp, 128 threads, 512: 2048x50001
    // bf16 with one alternative 54, 60, 118 us; 1000x50001 with 20 47, 43, 71;
    // 64x131072 with 20 38, 17.7, 13.3.  128, twice 512, 512 threads: 300x65536 f32
    // with 64 alternatives 29.1, 24.2, 28.3 (masked 39.4, 31.2, 37.4), with 20 22.7,
    // 20.4, with 5 18.6, 19.5; 64x131072 bf16 with 20 17.7, 14.6, 13.3.
    if constexpr (ENT) {
        if (a.r.rows >= kOutTarget && a.r.segs * a.seg_chunks <= kOutWarpVecs)
            return launch_rows(outcomes_finish<TYPE, 32, 6, MASK, ENT>, (a.r.rows + 3) / 4, 128, (size_t)4 * a.group_bytes,
                               a, stream);
        if (a.r.rows > kOutSms && a.r.rows <= 2 * kOutSms && a.n_top >= 16)
            return launch_rows(outcomes_finish<TYPE, 512, 2, MASK, ENT>, a.r.rows, 512, a.group_bytes, a, stream);
    }
    if (a.r.rows > kOutSms)
        return launch_rows(outcomes_finish<TYPE, 128, 6, MASK, ENT>, a.r.rows, 128, a.group_bytes, a, stream);
    return launch_rows(outcomes_finish<TYPE, 512, 1, MASK, ENT>, a.r.rows, 512, a.group_bytes, a, stream);
}

template <int TYPE, bool ENT, bool UNIT>
cudaError_t forward_mask(const OutForward &a, bool warp_rows, cudaStream_t stream) {
    return a.r.mask ? launch_forward<TYPE, true, ENT, UNIT>(a, warp_rows, stream)
                    : launch_forward<TYPE, false, ENT, UNIT>(a, warp_rows, stream);
}

}  // namespace

template <int TYPE>
cudaError_t outcomes_forward_of(const OutForward &a, bool warp_rows, cudaStream_t stream) {
    const bool ent = a.teacher.count == 0;
    if constexpr (TYPE == TN_TYPE_C64) {
        if (a.r.scale == 1.f)
            return ent ? forward_mask<TYPE, true, true>(a, warp_rows, stream)
                       : forward_mask<TYPE, false, true>(a, warp_rows, stream);
    }
    return ent ? forward_mask<TYPE, true, false>(a, warp_rows, stream)
               : forward_mask<TYPE, false, false>(a, warp_rows, stream);
}

}  // namespace tn
