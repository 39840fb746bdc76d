// Scores of outcome distributions, and the loss against a teacher: one pass
// over the rows.
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
#include "outcomes.cuh"

namespace tn {

namespace {

constexpr int kU = 4;               // vectors in flight per thread
constexpr float kLag = 8.f;         // of the reference, in powers of two

// ---- running sums -----------------------------------------------------------

// Distance of order value v from reference z in powers of two.  Amplitudes
// divide (correctly rounded) rather than subtract logarithms: the reference
// itself is at distance 0 exactly, and weights near it lose nothing.
template <int TYPE>
__device__ __forceinline__ float distance(float v, float z, float c2) {
    if constexpr (Entry<TYPE>::kReal) return (v - z) * c2;
    else return c2 * lg2(__fdiv_rn(v, z));
}

// z0: reference, an order value that was seen (absent until then).
template <int TYPE>
struct Sums {
    float z0 = absent<TYPE>(), s = 0.f, t = 0.f;

    __device__ __forceinline__ void move_to(float z, float c2) {
        const float d = distance<TYPE>(z0, z, c2);
        const float f = ex2(d);
        t = s == 0.f ? 0.f : f * (t + s * d);
        s = s == 0.f ? 0.f : f * s;
        z0 = z;
    }
};

template <int TYPE, bool UNIT>
__device__ __forceinline__ void add_vector(Sums<TYPE> &a, const float (&v)[Entry<TYPE>::E], float lm,
                                           float c2) {
    constexpr int E = Entry<TYPE>::E;
    if (lm == absent<TYPE>()) return;
    if (distance<TYPE>(lm, a.z0, c2) > kLag) a.move_to(lm, c2);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        // max: an absent entry adds 0 to t, not 0 times -inf
        float d, e;
        if constexpr (Entry<TYPE>::kReal) {
            d = max_nan(distance<TYPE>(v[i], a.z0, c2), -1e30f);
            e = ex2(d);
        } else {
            const float w = __fdiv_rn(v[i], a.z0);
            d = max_nan(c2 * lg2(w), -1e30f);
            e = UNIT ? w : ex2(d);     // |a|^2 itself at scale 1
        }
        a.s += e;
        a.t = fmaf(e, d, a.t);
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

// Positions of the first k of n keys in the order (key descending, position
// ascending), keys of 0 left out; written to out in ascending position order.
// Returns their number.  A bisection finds a threshold: at most 32 steps,
// usually about twelve, because any threshold with k keys above it will do.
template <int G, class KeyAt>
__device__ int select(Group<G> &g, KeyAt key, int n, int k, uint32_t *out) {
    uint32_t mx = 0, nz = 0;
    for (int i = g.t; i < n; i += G) {
        const uint32_t x = key(i);
        mx = max(mx, x);
        nz += x != 0;
    }
    mx = g.max(mx);
    nz = g.sum(nz);
    uint32_t thr = 1, ties = 0xffffffffu;     // take keys > thr and `ties` keys == thr
    if (nz > static_cast<uint32_t>(k)) {
        uint32_t lo = 1, hi = mx + 1, above = 0;   // count(>= lo) > k, above = count(>= hi) < k
        while (true) {
            if (hi - lo <= 1) {
                thr = lo;
                ties = k - above;
                break;
            }
            const uint32_t mid = lo + (hi - lo) / 2;
            uint32_t c = 0;
            for (int i = g.t; i < n; i += G) c += key(i) >= mid;
            c = g.sum(c);
            if (c == static_cast<uint32_t>(k)) {
                thr = mid;
                break;
            }
            if (c > static_cast<uint32_t>(k)) lo = mid;
            else {
                hi = mid;
                above = c;
            }
        }
    }
    const int per = (n + G - 1) / G;
    const int i0 = min(n, g.t * per), i1 = min(n, i0 + per);
    uint32_t gt = 0, eq = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = key(i);
        gt += x > thr;
        eq += x == thr;
    }
    uint32_t pg = gt, pe = eq;
    g.scan2(pg, pe);
    uint32_t at = pg + min(pe, ties);
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = key(i);
        if (x > thr) out[at++] = i;
        else if (x == thr) {
            if (pe < ties) out[at++] = i;
            ++pe;
        }
    }
    g.sync();
    return static_cast<int>(min(nz, static_cast<uint32_t>(k)));
}

// Rank of candidate i among n candidates in the same order.
__device__ __forceinline__ int rank_of(const uint32_t *keys, int n, int i) {
    const uint32_t x = keys[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += keys[j] > x || (keys[j] == x && j < i);
    return r;
}

// Shared memory of a group, in words.
struct Scratch {
    uint32_t *keys, *sub, *pos, *pos2, *pos3, *wkey;
    __device__ __forceinline__ Scratch(uint32_t *base, const OutForward &a)
        : keys(base), sub(keys + a.key_words), pos(sub + a.sub_words), pos2(pos + a.n_top),
          pos3(pos2 + a.n_top), wkey(pos3 + a.n_top) {}
};

// ---- the end of a row -------------------------------------------------------

template <int TYPE>
__device__ __forceinline__ float log_prob(const OutRows &r, float v, float logz) {
    if constexpr (Entry<TYPE>::kReal) return fmaf(v, r.scale, -logz);
    else return fmaf(r.scale, logf(v), -logz);
}

template <int TYPE, int G>
__device__ __forceinline__ void finish_row(Group<G> &g, const OutForward &a, const Row<TYPE> &r,
                                           int64_t row, float logz, float entropy) {
    constexpr float kInf = __builtin_huge_valf();
    if (g.t == 0) a.logz[row] = logz;
    if (a.teacher.count == 0) {
        if (g.t == 0) a.entropy[row] = entropy;
        for (int j = g.t; j < a.n_given; j += G) {
            const int64_t id = a.given[row * a.n_given + j];
            float lp;
            if (id == -1) {
                lp = 0.f;
            } else if (id < 0 || id >= r.cols) {
                lp = __int_as_float(0x7fffffff);
                flag_bad_id(a.r, row);
            } else {
                const float v = r.value(id);
                lp = v == absent<TYPE>() ? -kInf : log_prob<TYPE>(a.r, v, logz);
            }
            a.logp[row * a.n_given + j] = lp;
        }
    } else {
        Teacher<G> te;
        te.load(g, a.teacher, a.r, r, row);
        float loss = 0.f;
#pragma unroll
        for (int i = 0; i < Teacher<G>::kPer; ++i)
            if (te.id[i] >= 0 && te.q[i] != 0.f) {
                const float v = r.value(te.id[i]);
                const float lp = v == absent<TYPE>() ? -kInf : log_prob<TYPE>(a.r, v, logz);
                loss += te.q[i] * (te.logq[i] - lp);
            }
        if (logz == -kInf) loss = 0.f;
        if (te.bad) loss = __int_as_float(0x7fffffff);
        loss = g.sum(loss);
        if (g.t == 0) a.loss[row] = loss;
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
        logz = fmaf(r.scale, Entry<TYPE>::kReal ? a.z0 : logf(a.z0), ls);
        entropy = ls - kLn2 * (a.t / a.s);
    } else {
        logz = entropy = __int_as_float(0x7fffffff);
    }
}

// ---- the kernel -------------------------------------------------------------

template <int TYPE, int G, bool MASK, bool UNIT>
__global__ void __launch_bounds__(kOutThreads)
outcomes_forward(const __grid_constant__ OutForward a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr int kGroups = kOutThreads / G;
    extern __shared__ uint32_t smem[];
    __shared__ uint32_t red[4 * kOutThreads / 32];
    __shared__ bool last;
    pdl_trigger();
    Group<G> g(red);
    const int64_t item = (int64_t)blockIdx.x * kGroups + threadIdx.x / G;
    const int64_t row = G == 32 ? item : item / a.r.segs;
    const int64_t seg = G == 32 ? 0 : item - row * a.r.segs;
    Scratch sm(smem + (size_t)(threadIdx.x / G) * (a.key_words + a.sub_words + 4 * a.n_top), a);
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;

    const Row<TYPE> r(a.r, row);
    const int64_t v0 = seg * a.r.seg_vecs;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    const int64_t v1 = min(all, v0 + a.r.seg_vecs);
    const int nv = static_cast<int>(max((int64_t)0, v1 - v0));   // may be 0 in a row's last segment
    const int k = a.n_top;
    const bool chunks = nv > kOutKeys;      // one maximum per 32 vectors

    Sums<TYPE> sum;
    for (int b = 0; b < nv; b += kU * G) {
        uint4 raw[kU];
        uint32_t bits[kU];
        bool in[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + g.t;
            const int64_t e0 = (v0 + j) * E - r.head;
            in[u] = j < nv && r.inside(e0);
            if (in[u]) raw[u] = r.raw(e0);
        }
        if constexpr (MASK) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (in[u]) bits[u] = r.keep_bits((v0 + b + u * G + g.t) * E - r.head);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + g.t;
            float v[E];
            if (in[u]) {
                En::values(raw[u], v);
                if constexpr (MASK) {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (!(bits[u] >> i & 1)) v[i] = absent<TYPE>();
                }
            } else if (j < nv) {
                r.vector(v0 + j, v);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = absent<TYPE>();
            }
            float lm = v[0];
#pragma unroll
            for (int i = 1; i < E; ++i) lm = max_nan(lm, v[i]);
            add_vector<TYPE, UNIT>(sum, v, lm, a.r.c2);
            if (k > 0) {
                uint32_t key = order_key<TYPE>(lm);
                if (chunks) {
                    key = __reduce_max_sync(0xffffffffu, key);
                    if (g.lane == 0 && j < nv) sm.keys[j >> 5] = key;
                } else if (j < nv) {
                    sm.keys[j] = key;
                }
            }
        }
    }
    combine(g, sum, a.r.c2);     // its barriers also publish the maxima
    g.sync();

    // the segment's alternatives: wkey / pos3 hold their keys and their entry
    // index within the segment, best first at their rank
    int found = 0;
    const bool valid = sum.s < __builtin_huge_valf();
    if (k > 0 && valid) {
        const uint32_t *keys = sm.keys;
        int nsel;
        if (chunks) {
            const int nc = select(g, [=](int i) { return keys[i]; }, (nv + 31) >> 5, k, sm.pos);
            for (int c = g.warp; c < nc; c += Group<G>::kWarps) {
                const int j = (int)sm.pos[c] * 32 + g.lane;
                uint32_t key = 0;
                if (j < nv) {
                    float v[E];
                    r.vector(v0 + j, v);
                    float lm = v[0];
#pragma unroll
                    for (int i = 1; i < E; ++i) lm = max_nan(lm, v[i]);
                    key = order_key<TYPE>(lm);
                }
                sm.sub[c * 32 + g.lane] = key;
            }
            g.sync();
            const uint32_t *sub = sm.sub;
            nsel = select(g, [=](int i) { return sub[i]; }, nc * 32, k, sm.pos2);
            for (int i = g.t; i < nsel; i += G) {
                const uint32_t x = sm.pos2[i];
                sm.pos2[i] = sm.pos[x >> 5] * 32 + (x & 31);
            }
        } else {
            nsel = select(g, [=](int i) { return keys[i]; }, nv, k, sm.pos2);
        }
        g.sync();
        for (int i = g.t; i < nsel; i += G) {
            float v[E];
            r.vector(v0 + sm.pos2[i], v);
#pragma unroll
            for (int e = 0; e < E; ++e) sm.keys[i * E + e] = order_key<TYPE>(v[e]);
        }
        g.sync();
        found = select(g, [=](int i) { return keys[i]; }, nsel * E, k, sm.pos);
        for (int i = g.t; i < found; i += G) sm.wkey[i] = sm.keys[sm.pos[i]];
        g.sync();
        for (int i = g.t; i < found; i += G) {
            const uint32_t x = sm.pos[i];
            const int rank = rank_of(sm.wkey, found, i);
            sm.pos3[rank] = sm.pos2[x / E] * E + x % E;
            sm.keys[rank] = sm.wkey[i];
        }
        g.sync();
    }

    float logz, entropy;
    if (G == 32 || a.r.segs == 1) {
        normaliser<TYPE>(a.r, sum, logz, entropy);
        finish_row<TYPE>(g, a, r, row, logz, entropy);
        for (int i = g.t; i < k; i += G) {
            const bool have = i < found;
            a.top_ids[row * k + i] = have ? (int64_t)sm.pos3[i] - r.head : -1;
            a.top_logp[row * k + i] = have ? log_prob<TYPE>(a.r, key_value(sm.keys[i]), logz)
                                      : valid ? -__builtin_huge_valf() : logz;
        }
        return;
    }

    if constexpr (G > 32) {
        // leave the segment's part in the workspace; the last one joins
        const int64_t slot = row * a.r.segs + seg;
        if (g.t == 0) {
            OutPartial p;
            p.z0 = sum.z0;
            p.s = sum.s;
            p.t = sum.t;
            p.pad = 0;
            a.partials[slot] = p;
        }
        for (int i = g.t; i < k; i += G)
            a.lists[slot * k + i] = i < found ? make_uint2(sm.keys[i], sm.pos3[i]) : make_uint2(0, 0);
        __threadfence();
        __syncthreads();
        if (g.t == 0) last = atomicAdd(a.tickets + row, 1u) == (uint32_t)a.r.segs - 1;
        __syncthreads();
        if (!last) return;
        __threadfence();
        if (g.t == 0) a.tickets[row] = 0;    // ready for the next call

        const int segs = static_cast<int>(a.r.segs);
        const int64_t slot0 = row * a.r.segs;
        sum = Sums<TYPE>();
        for (int i = g.t; i < segs; i += G) {
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
        normaliser<TYPE>(a.r, sum, logz, entropy);
        finish_row<TYPE>(g, a, r, row, logz, entropy);
        if (k == 0) return;
        found = 0;
        const bool valid_row = sum.s < __builtin_huge_valf();
        if (valid_row) {
            // lists are sorted: a segment's first key is its largest, and the
            // first key of eight consecutive ones theirs
            const uint2 *lists = a.lists + slot0 * k;
            const int ns = select(g, [=](int i) { return __ldcg(lists + (int64_t)i * k).x; }, segs, k,
                                  sm.pos);
            const int oct = (k + 7) / 8;
            for (int i = g.t; i < ns * oct; i += G)
                sm.sub[i] = __ldcg(lists + (int64_t)sm.pos[i / oct] * k + i % oct * 8).x;
            g.sync();
            const uint32_t *sub = sm.sub;
            const int no = select(g, [=](int i) { return sub[i]; }, ns * oct, k, sm.pos2);
            for (int i = g.t; i < no * 8; i += G) {
                const uint32_t x = sm.pos2[i / 8];
                const int at = (int)x % oct * 8 + i % 8;
                sm.keys[i] = at < k ? __ldcg(lists + (int64_t)sm.pos[x / oct] * k + at).x : 0u;
            }
            g.sync();
            const uint32_t *keys = sm.keys;
            found = select(g, [=](int i) { return keys[i]; }, no * 8, k, sm.pos3);
            for (int i = g.t; i < found; i += G) sm.wkey[i] = sm.keys[sm.pos3[i]];
            g.sync();
            for (int i = g.t; i < found; i += G) {
                const int rank = rank_of(sm.wkey, found, i);
                const uint32_t x = sm.pos2[sm.pos3[i] / 8];
                const uint32_t sg = sm.pos[x / oct];
                const int64_t local =
                    __ldcg(lists + (int64_t)sg * k + x % oct * 8 + sm.pos3[i] % 8).y;
                a.top_ids[row * k + rank] = (int64_t)sg * a.r.seg_vecs * E + local - r.head;
                a.top_logp[row * k + rank] = log_prob<TYPE>(a.r, key_value(sm.wkey[i]), logz);
            }
        }
        for (int i = found + g.t; i < k; i += G) {
            a.top_ids[row * k + i] = -1;
            a.top_logp[row * k + i] = valid_row ? -__builtin_huge_valf() : logz;
        }
    }
}

template <int TYPE, int G, bool MASK, bool UNIT>
cudaError_t launch(const OutForward &a, cudaStream_t stream) {
    const int64_t items = a.r.rows * a.r.segs;
    const int groups = kOutThreads / G;
    const size_t smem = sizeof(uint32_t) * groups * ((size_t)a.key_words + a.sub_words + 4 * a.n_top);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(outcomes_forward<TYPE, G, MASK, UNIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(outcomes_forward<TYPE, G, MASK, UNIT>, dim3((unsigned)((items + groups - 1) / groups)),
                      dim3(kOutThreads), smem, stream, a);
}

template <int TYPE, int G>
cudaError_t launch_mask(const OutForward &a, cudaStream_t stream) {
    if constexpr (TYPE == TN_TYPE_C64) {
        if (a.r.scale == 1.f)
            return a.r.mask ? launch<TYPE, G, true, true>(a, stream) : launch<TYPE, G, false, true>(a, stream);
    }
    return a.r.mask ? launch<TYPE, G, true, false>(a, stream) : launch<TYPE, G, false, false>(a, stream);
}

}  // namespace

OutSplit out_split(int32_t type, int64_t cols, int64_t rows) {
    const int64_t E = kOutVecBytes / out_entry_bytes(type);
    OutSplit s;
    s.vecs = (cols + E - 1 + E - 1) / E;   // the first vector may hold one entry only
    s.warp_rows = s.vecs <= kOutWarpVecs;
    s.segs = 1;
    s.seg_vecs = s.vecs;
    if (s.warp_rows) return s;
    // four CTAs fit on an SM; a CTA of less than two vectors a thread gains
    // nothing
    const int64_t target = 4 * 152;
    int64_t want = rows >= target ? 1 : (target + rows - 1) / rows;
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

cudaError_t launch_outcomes_forward(int32_t type, const OutForward &a, bool warp_rows,
                                    cudaStream_t stream) {
    switch (type) {
        case TN_TYPE_C64:
            return warp_rows ? launch_mask<TN_TYPE_C64, 32>(a, stream)
                             : launch_mask<TN_TYPE_C64, kOutThreads>(a, stream);
        case TN_TYPE_F32:
            return warp_rows ? launch_mask<TN_TYPE_F32, 32>(a, stream)
                             : launch_mask<TN_TYPE_F32, kOutThreads>(a, stream);
        case TN_TYPE_BF16:
            return warp_rows ? launch_mask<TN_TYPE_BF16, 32>(a, stream)
                             : launch_mask<TN_TYPE_BF16, kOutThreads>(a, stream);
        default:
            return warp_rows ? launch_mask<TN_TYPE_F16, 32>(a, stream)
                             : launch_mask<TN_TYPE_F16, kOutThreads>(a, stream);
    }
}

}  // namespace tn
