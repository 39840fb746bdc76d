// Drawing outcomes from rows: weights, filters and draws.
//
// An outcome is a whole number, and near a border between two outcomes any
// rounding decides it: a sum of 10^5 weights in fp32 is wrong by some 2^-22, and one
// draw in ten of a broad row lies that near to a border.  So weights are computed as
// pairs of fp32 numbers (43 bits) and summed as 64-bit integers, in
// units of 2^-shift of the largest, the shift chosen by an estimate of the row's
// sum so that it uses 61 bits.  Integer sums need no order: histograms by
// shared-memory atomics, partial sums of CTAs and of warps are all exact.
#pragma once

#include "outcomes.cuh"
#include "sampling.h"

namespace tn {

// 2^(i/32) and 2^(j/1024), each as the sum of two fp32 numbers
static __device__ const float2 kCoarse[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9e0p+0f, -0x1.5c0424p-25f}, {0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.6247ecp+0f, -0x1.f8b550p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246eb0p-26f},
};
static __device__ const float2 kFine[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.002c60p+0f, 0x1.78ba34p-26f}, {0x1.0058c8p+0f, 0x1.b68702p-26f},
    {0x1.008538p+0f, 0x1.7d77c2p-27f}, {0x1.00b1b0p+0f, -0x1.6950d0p-26f}, {0x1.00de2ep+0f, 0x1.a1dc1ep-25f},
    {0x1.010ab6p+0f, -0x1.34d0bcp-26f}, {0x1.013744p+0f, 0x1.326d6ep-26f}, {0x1.0163dap+0f, 0x1.3f6666p-25f},
    {0x1.019078p+0f, 0x1.5ad434p-25f}, {0x1.01bd1ep+0f, 0x1.dc5c2ep-26f}, {0x1.01e9ccp+0f, -0x1.eec114p-32f},
    {0x1.021682p+0f, -0x1.789fb0p-25f}, {0x1.02433ep+0f, 0x1.252dd6p-26f}, {0x1.027004p+0f, -0x1.df89dep-25f},
    {0x1.029cd0p+0f, -0x1.98a37ep-26f}, {0x1.02c9a4p+0f, -0x1.887fa0p-28f}, {0x1.02f680p+0f, -0x1.626868p-30f},
    {0x1.032364p+0f, -0x1.5ea7ecp-27f}, {0x1.035050p+0f, -0x1.1421f2p-25f}, {0x1.037d42p+0f, 0x1.c2377ap-25f},
    {0x1.03aa3ep+0f, 0x1.70aafep-28f}, {0x1.03d742p+0f, -0x1.cdd4aep-25f}, {0x1.04044cp+0f, -0x1.76954ap-28f},
    {0x1.04315ep+0f, 0x1.0dcff0p-25f}, {0x1.045e78p+0f, 0x1.eac818p-25f}, {0x1.048b9cp+0f, -0x1.9534c4p-25f},
    {0x1.04b8c6p+0f, -0x1.6f70bcp-25f}, {0x1.04e5f8p+0f, -0x1.a1356ap-25f}, {0x1.051330p+0f, 0x1.d83408p-25f},
    {0x1.054072p+0f, 0x1.ff05d8p-26f}, {0x1.056dbcp+0f, -0x1.448794p-28f},
};

// 2^(k/1024), k = 0 .. 1023, in shared memory: the products of the two.
constexpr int kRoots = 1024;
template <int NT>
__device__ __forceinline__ void make_roots(float2 *roots) {
    for (int k = threadIdx.x; k < kRoots; k += NT) {
        const float2 c = kCoarse[k >> 5], f = kFine[k & 31];
        const float h = c.x * f.x, l = fmaf(c.x, f.x, -h) + fmaf(c.x, f.y, c.y * f.x), x = h + l;
        roots[k] = make_float2(x, (h - x) + l);
    }
}

// What a row's weights are computed from.
struct RowPlan {
    float m;            // largest order value
    float ch, cl;       // beta log2(e) as a pair
    float down;         // amplitudes at beta = 1: 2^-x with weights up to 2^x
    int shift;          // a weight of 1 is 2^shift
    int down_log;       // x
    double beta;
    int state;          // kDraw, or how the row ends
    bool greedy;
    uint64_t bound;     // entries of at least this rank are left
};
enum { kDraw = 0, kEmpty = 1, kUndefined = 2 };

// Rank of an entry: by order value, then by index (lowest first); absent ones have
// none.  Any present entry's is at least kPresent.
constexpr uint64_t kPresent = 1ull << 32;
template <int TYPE>
__device__ __forceinline__ uint64_t rank_of(float v, int64_t e) {
    const uint32_t k = order_key<TYPE>(v);
    return k ? static_cast<uint64_t>(k) << 32 | (0xffffffffu - static_cast<uint32_t>(e)) : 0;
}

// beta log2(e) (v - m) as a pair of fp32 numbers.
__device__ __forceinline__ float2 exponent(const RowPlan &p, float v) {
    const float d = v - p.m, b = d - v;                     // d + e is the exact difference
    const float e = (v - (d - b)) + (-p.m - b);
    const float h = d * p.ch;
    return make_float2(h, fmaf(d, p.cl, fmaf(e, p.ch, fmaf(d, p.ch, -h))));
}

// The weight of a present entry, 1 at least (so that a draw of u = 0 finds the
// first entry left).  2^t of a pair t: 2^(k/1024) from a table, the rest (at most
// 2^-11) by the exponential series, whose first term is kept as a pair.
__device__ __forceinline__ uint64_t weight_real(const RowPlan &p, const float2 *roots, float v) {
    constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f, kMagic = 12582912.f;
    const float2 t = exponent(p, v);
    if (!(t.x > -64.f)) return 1;
    const float km = fmaf(t.x, 1024.f, kMagic), kf = __fadd_rn(km, -kMagic);
    const int k = static_cast<int>(__float_as_uint(km) - __float_as_uint(kMagic));
    const float r = fmaf(kf, -0x1p-10f, t.x);               // exact
    const float g = r * kLn2Hi;
    const float gl = fmaf(r, kLn2Hi, -g) + fmaf(r, kLn2Lo, t.y * kLn2Hi);
    const float lo = fmaf(g * g, fmaf(g, 1.f / 6, 0.5f), gl);   // 2^r - 1 = g + lo
    const float2 root = roots[k & (kRoots - 1)];
    const float a = root.x * g, al = fmaf(root.x, g, -a);
    const float w0 = root.x + a;
    const float wm = ((root.x - w0) + a) + (al + fmaf(root.x, lo, fmaf(root.y, g, root.y)));
    const float w = w0 + wm, wl = (w0 - w) + wm;            // (t's low part makes wm up to 2^-19)
    // w + wl in units of 2^-44 (conversions of fp32 to 64-bit integers would run on the fp64 pipe):
    // w, below 2, to 2^-22 from the mantissa of w + 2, what is left of it with wl from
    // that of a sum with kMagic (it is less than 2^-22)
    const float up = __fadd_rn(w, 2.f), rest = (w - __fadd_rn(up, -2.f)) + wl;
    const int low = static_cast<int>(__float_as_uint(fmaf(rest, 0x1p44f, kMagic)) - __float_as_uint(kMagic));
    const int64_t n = static_cast<int64_t>(static_cast<int>(__float_as_uint(up) - 0x40000000u)) * (1 << 22) + low;
    const int x = (k >> 10) + p.shift - 44;
    const uint64_t whole = x >= 0 ? static_cast<uint64_t>(n) << x : x > -64 ? static_cast<uint64_t>(n) >> -x : 0;
    return whole > 0 ? whole : 1;
}

// A number of 0 <= v < 4 in units of 2^-shift, the same way.
__device__ __forceinline__ uint64_t in_units(float v, int shift) {
    const uint32_t b = __float_as_uint(v);
    const uint64_t n = (b & 0x7fffffu) | 0x800000u;
    const int x = static_cast<int>(b >> 23) - 150 + shift;
    return x >= 0 ? n << x : x > -64 ? n >> -x : 0;
}

template <int TYPE>
__device__ __forceinline__ uint64_t weight(const RowPlan &p, const float2 *roots, float v) {
    if constexpr (Entry<TYPE>::kReal) {
        return weight_real(p, roots, v);
    } else {
        uint64_t n;
        if (p.beta == 1.0) {
            n = in_units(v * p.down, p.shift);
        } else {
            const double x = p.beta * log(static_cast<double>(v) / p.m);
            n = x < -60.0 ? 1 : static_cast<uint64_t>(__double2ll_rn(ldexp(exp(x), p.shift)));
        }
        return n > 0 ? n : 1;
    }
}
// The same in fp32, relative to the largest: for an estimate of the sum.
template <int TYPE>
__device__ __forceinline__ float rough_weight(const RowPlan &p, float v) {
    if constexpr (Entry<TYPE>::kReal) return ex2((v - p.m) * p.ch);
    else if (p.beta == 1.0) return v * p.down;
    else return ex2(static_cast<float>(p.beta) * lg2(v / p.m));
}

template <int TYPE>
__device__ __forceinline__ void vector_values(const Row<TYPE> &r, int64_t j, float (&v)[Entry<TYPE>::E]) {
    using En = Entry<TYPE>;
    const int64_t e0 = j * En::E - r.head;
    if (r.inside(e0)) {
        uint4 q = r.raw(e0);
        if (r.m) En::blank(q, row_keep<TYPE>(r, e0));
        En::values(q, v);
    } else {
        const Values<En::E> o = row_vector<TYPE>(r, j);
#pragma unroll
        for (int i = 0; i < En::E; ++i) v[i] = o.v[i];
    }
}

// f(order values, vector) of vectors first, first + stride, .. below hi, N at a time with
// their loads in flight together; `edge` is the first vector behind those that the
// caller's threads read at a time (N stride further than the first of them), so that
// they all take the same way.
template <int TYPE, int N, class F>
__device__ __forceinline__ void vectors_at(const Row<TYPE> &r, int64_t in_lo, int64_t in_hi, int64_t from, int64_t edge,
                                           int64_t first, int stride, int64_t hi, F f) {
    using En = Entry<TYPE>;
    if (from >= in_lo && edge <= in_hi && edge <= hi) {
        uint4 q[N];
        const uint4 *p = r.vectors() + first;
#pragma unroll
        for (int n = 0; n < N; ++n) q[n] = __ldcg(p + n * stride);
        if (r.m) {
            typename Row<TYPE>::Keep keep[N];
#pragma unroll
            for (int n = 0; n < N; ++n) keep[n] = r.keep((first + n * stride) * En::E - r.head);
#pragma unroll
            for (int n = 0; n < N; ++n) En::blank(q[n], keep[n]);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float v[En::E];
            En::values(q[n], v);
            f(v, first + n * stride);
        }
    } else {
#pragma unroll 1
        for (int n = 0; n < N; ++n) {
            const int64_t j = first + n * stride;
            if (j >= hi) break;
            float v[En::E];
            vector_values<TYPE>(r, j, v);
            f(v, j);
        }
    }
}
// The same of all vectors lo .. hi - 1, by NT threads.
template <int TYPE, int NT, int N, class F>
__device__ __forceinline__ void each_vector(const Row<TYPE> &r, int64_t lo, int64_t hi, F f) {
    int64_t in_lo, in_hi;
    r.inside_range(in_lo, in_hi);
    for (int64_t from = lo; from < hi; from += N * NT)
        vectors_at<TYPE, N>(r, in_lo, in_hi, from, from + N * NT, from + threadIdx.x, NT, hi, f);
}

__device__ __forceinline__ uint64_t shfl_up(uint64_t x, int o) {
    return __shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(x), o);
}
__device__ __forceinline__ uint64_t shfl_from(uint64_t x, int lane) {
    return __shfl_sync(0xffffffffu, static_cast<unsigned long long>(x), lane);
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(x), o);
    return x;
}
// inclusive
__device__ __forceinline__ uint64_t warp_scan(uint64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = shfl_up(x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// floor(u z) and ceil(u z) of a number 0 <= u <= 1, exact.
__device__ __forceinline__ uint64_t share(double u, uint64_t z, bool up) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(u));
    const int e = static_cast<int>(b >> 52 & 0x7ff);
    const uint64_t m = (b & ((1ull << 52) - 1)) | (e ? 1ull << 52 : 0);
    const int right = 1075 - (e ? e : 1);                   // u = m 2^-right
    const unsigned __int128 p = static_cast<unsigned __int128>(m) * z;
    if (right >= 128) return up && p != 0;
    uint64_t q = static_cast<uint64_t>(p >> right);
    if (up && (p & ((static_cast<unsigned __int128>(1) << right) - 1)) != 0) ++q;
    return q;
}

// Parameters of a row; false if one is invalid.
struct Filters {
    float beta, top_p, min_p;
    int32_t top_k;
    bool greedy;
};
__device__ __forceinline__ bool filters_of(const SampleArgs &a, int64_t row, Filters &f) {
    const float t = a.f.temperatures ? a.f.temperatures[row] : a.f.temperature;
    f.top_p = a.f.top_ps ? a.f.top_ps[row] : a.f.top_p;
    f.min_p = a.f.min_ps ? a.f.min_ps[row] : a.f.min_p;
    f.top_k = a.f.top_ks ? a.f.top_ks[row] : a.f.top_k;
    f.greedy = t == 0.f || f.top_k == 1;
    f.beta = t == 0.f ? 1.f : fminf(__fdiv_rn(a.r.scale, t), 3.402823466e38f);
    return t >= 0.f && t <= 3.402823466e38f && f.top_p == f.top_p && f.min_p <= 1.f;
}

// What follows from a row's largest order value.
template <int TYPE>
__device__ __forceinline__ void plan_row(RowPlan &p, float m, bool valid, const Filters &f) {
    p.m = m;
    p.beta = f.beta;
    const double c = static_cast<double>(f.beta) * 1.4426950408889634;
    p.ch = c < 3.4e38 ? static_cast<float>(c) : 3.402823466e38f;
    p.cl = c < 3.4e38 ? static_cast<float>(c - p.ch) : 0.f;
    p.greedy = f.greedy;
    p.bound = kPresent;
    int x = 0;
    if (!Entry<TYPE>::kReal) frexpf(m, &x);                 // m < 2^x
    x = x < -126 ? -126 : x > 126 ? 126 : x;                // (2^-x is a number; weights may be up to 4)
    p.down_log = x;
    p.down = ldexpf(1.f, -x);
    p.shift = 0;
    p.state = !valid || m != m || m == __builtin_huge_valf() ? kUndefined : m == absent<TYPE>() ? kEmpty : kDraw;
}
// and from an estimate of its weights' sum
__device__ __forceinline__ int shift_of(float sum) {
    int x;
    frexpf(fminf(fmaxf(sum, 0.25f), 0x1p33f) * 1.001f, &x);
    return 61 - x;
}

// Entries of weight >= min_p of the largest: those of order value >= this.
template <int TYPE>
__device__ __forceinline__ float least_value(const RowPlan &p, float min_p) {
    double x;
    if constexpr (Entry<TYPE>::kReal) x = p.m + log(static_cast<double>(min_p)) / p.beta;
    else if (p.beta == 1.0) x = static_cast<double>(p.m) * min_p;
    else x = p.m * exp(log(static_cast<double>(min_p)) / p.beta);
    float v = static_cast<float>(x);
    if (v < x) v = nextafterf(v, __builtin_huge_valf());
    return fminf(v, p.m);
}

// log p of an entry left, from the weights' sum.
template <int TYPE>
__device__ __noinline__ float log_p(const RowPlan &p, float v, uint64_t total) {
    constexpr double kLn2d = 0.693147180559945309;
    double z = log(static_cast<double>(total)) - p.shift * kLn2d, x;
    if constexpr (Entry<TYPE>::kReal) {
        x = p.beta * (static_cast<double>(v) - p.m);
    } else if (p.beta == 1.0) {
        x = log(static_cast<double>(v));
        z += p.down_log * kLn2d;
    } else {
        x = p.beta * log(static_cast<double>(v) / p.m);
    }
    return static_cast<float>(x - z);
}

// ---- a row of one CTA -------------------------------------------------------

struct Select {
    uint32_t lo[256], hi[256], count[256];
    int digit;
    uint32_t in_digit;
    uint64_t above;
    bool whole;
};

template <int TYPE, int NT>
struct RowCta {
    static constexpr int E = Entry<TYPE>::E;
    Row<TYPE> r;
    int64_t vecs;
    const RowPlan *p;
    const float2 *roots;
    Select *sel;
    uint64_t *sums;     // NT / 32

    // f(order value, index) of every entry of the row
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        each_vector<TYPE, NT, 1>(r, 0, vecs, [&](const float (&v)[E], int64_t j) {
#pragma unroll
            for (int i = 0; i < E; ++i) f(v[i], j * E - r.head + i);
        });
    }
    __device__ __forceinline__ uint64_t sum(uint64_t x) const {
        x = warp_sum(x);
        __syncthreads();
        if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = x;
        __syncthreads();
        x = 0;
        for (int w = 0; w < NT / 32; ++w) x += sums[w];
        return x;
    }
    // Weights' sum (or the number) of the entries of at least that rank.
    template <bool MASS>
    __device__ __noinline__ uint64_t total(uint64_t bound) const {
        uint64_t s = 0;
        each([&](float v, int64_t e) {
            if (rank_of<TYPE>(v, e) >= bound) s += MASS ? weight<TYPE>(*p, roots, v) : 1;
        });
        return sum(s);
    }
    // The rank down to which entries, largest first, reach `target` in weight (or
    // number), of those of at least the rank `bound`; `bound` if all do not.  Eight
    // bits of the rank at a time, from the top: sums by digit, then on with the digit in
    // which the target is reached.
    template <bool MASS>
    __device__ __noinline__ uint64_t select(uint64_t target, uint64_t bound) const {
        uint64_t prefix = 0, above = 0;
        for (int shift = 56; shift >= 0; shift -= 8) {
            if (shift == 24 && r.cols <= 1 << 24) {         // the same digit in every index
                prefix |= 0xffull << 24;
                continue;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 256; i += NT) sel->lo[i] = sel->hi[i] = sel->count[i] = 0;
            __syncthreads();
            each([&](float v, int64_t e) {
                const uint64_t k = rank_of<TYPE>(v, e);
                if (k < bound || k == 0 || (shift < 56 && (k ^ prefix) >> (shift + 8))) return;
                const int d = static_cast<int>(k >> shift & 255);
                atomicAdd(&sel->count[d], 1u);
                if constexpr (MASS) {
                    const uint64_t w = weight<TYPE>(*p, roots, v);
                    const uint32_t l = static_cast<uint32_t>(w), old = atomicAdd(&sel->lo[d], l);
                    const uint32_t h = static_cast<uint32_t>(w >> 32) + (old + l < l);
                    if (h) atomicAdd(&sel->hi[d], h);
                }
            });
            __syncthreads();
            if (threadIdx.x < 32) {     // eight digits a lane, from the top
                const int lane = threadIdx.x;
                uint64_t own = 0;
                for (int i = 0; i < 8; ++i) {
                    const int d = 255 - lane * 8 - i;
                    own += MASS ? static_cast<uint64_t>(sel->hi[d]) << 32 | sel->lo[d] : sel->count[d];
                }
                uint64_t upto = above + warp_scan(own, lane);
                const uint32_t reached = __ballot_sync(0xffffffffu, upto >= target);
                if (lane == 0) sel->digit = -1;
                __syncwarp();
                if (reached && lane == __ffs(reached) - 1) {
                    upto -= own;
                    for (int i = 0; i < 8; ++i) {
                        const int d = 255 - lane * 8 - i;
                        const uint64_t x = MASS ? static_cast<uint64_t>(sel->hi[d]) << 32 | sel->lo[d] : sel->count[d];
                        if (upto + x >= target) {
                            sel->digit = d;
                            sel->in_digit = sel->count[d];
                            sel->above = upto;
                            sel->whole = upto + x == target;
                            break;
                        }
                        upto += x;
                    }
                }
            }
            __syncthreads();
            if (sel->digit < 0) return bound;
            above = sel->above;
            prefix |= static_cast<uint64_t>(sel->digit) << shift;
            if (sel->in_digit == 1 || sel->whole) break;    // all of the digit, whatever follows
        }
        return prefix > bound ? prefix : bound;
    }
};

// The first of n sums at which their total exceeds `target`, which becomes what is
// left of it there; one warp.
__device__ __forceinline__ int64_t locate(const uint64_t *sums, int64_t n, uint64_t &target) {
    const int lane = threadIdx.x % 32;
    for (int64_t base = 0; base < n; base += 32) {
        const uint64_t own = base + lane < n ? __ldcg(sums + base + lane) : 0, upto = warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, upto > target);
        if (over) {
            const int l = __ffs(over) - 1;
            target -= shfl_from(upto - own, l);
            return base + l;
        }
        target -= shfl_from(upto, 31);
    }
    return 0;
}

// The same of sums that are added up already: a search by 32.
__device__ __forceinline__ int64_t locate_upto(const ulonglong2 *upto, int64_t n, uint64_t &target) {
    const int lane = threadIdx.x % 32;
    int64_t lo = 0, len = n;
    while (len > 1) {
        const int64_t step = (len + 31) / 32, at = lo + (lane + 1) * step - 1;
        const bool over = lane * step < len && (at >= lo + len - 1 || __ldcg(&upto[at]).x > target);
        const int l = __ffs(__ballot_sync(0xffffffffu, over)) - 1;
        len = len - l * step < step ? len - l * step : step;
        lo += l * step;
    }
    if (lo > 0) target -= __ldcg(&upto[lo - 1]).x;
    return lo;
}

// One warp: a draw of row r.  Where the row has segments, `partials` holds their
// sums up to each (the first of a pair).
template <int TYPE>
__device__ void warp_draw(const SampleArgs &a, const Row<TYPE> &r, int64_t vecs, const RowPlan &p, const float2 *roots,
                          const uint64_t *masses, int64_t pieces, const ulonglong2 *partials, uint64_t total,
                          int64_t at, int64_t row) {
    constexpr int E = Entry<TYPE>::E;
    const int lane = threadIdx.x % 32;
    const double u = a.wide ? static_cast<const double *>(a.u)[at] : static_cast<const float *>(a.u)[at];
    if (!(u >= 0.0 && u < 1.0)) {
        if (lane == 0) {
            a.ids[at] = -1;
            a.logp[at] = __uint_as_float(0x7fc00000u);
            flag_bad_id(a.r, row);
        }
        return;
    }
    uint64_t target = p.greedy ? 0 : share(u, total, false);
    int64_t first = 0;
    if (partials) {
        first = locate_upto(partials, a.segs, target) * a.seg_pieces;
        pieces = pieces - first < a.seg_pieces ? pieces - first : a.seg_pieces;
    }
    const int64_t piece = first + locate(masses + first, pieces, target);
    for (int i = 0; i < kPieceVecs / 32; ++i) {
        const int64_t j = piece * kPieceVecs + i * 32 + lane;
        float v[E];
        uint64_t w[E], own = 0;
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = 0;
        if (j < vecs) {
            vector_values<TYPE>(r, j, v);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const uint64_t rank = rank_of<TYPE>(v[k], j * E - r.head + k);
                if (rank >= p.bound) w[k] = weight<TYPE>(p, roots, v[k]);
                own += w[k];
            }
        }
        const uint64_t upto = warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, upto > target);
        if (!over) {
            target -= shfl_from(upto, 31);
            continue;
        }
        if (lane == __ffs(over) - 1) {
            uint64_t left = target - (upto - own);
            bool found = false;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                if (!found && w[k] > left) {
                    found = true;
                    a.ids[at] = j * E - r.head + k;
                    a.logp[at] = p.greedy ? 0.f : log_p<TYPE>(p, v[k], total);
                }
                left -= w[k];
            }
        }
        return;
    }
}

// Outcomes of a row that has none.
__device__ __forceinline__ void no_draws(const SampleArgs &a, int64_t row, int state) {
    for (int64_t d = threadIdx.x; d < a.draws; d += kDrawThreads) {
        a.ids[row * a.draws + d] = -1;
        a.logp[row * a.draws + d] = state == kEmpty ? -__builtin_huge_valf() : __uint_as_float(0x7fc00000u);
    }
    if (threadIdx.x == 0) a.kept[row] = 0;
}

template <int TYPE, int NT>
__global__ void __launch_bounds__(NT) sample_rows_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ float2 roots[kRoots];
    __shared__ RowPlan plan;
    __shared__ Select sel;
    __shared__ uint64_t sums[NT / 32];
    __shared__ uint32_t red[4 * (NT / 32)];
    pdl_trigger();
    make_roots<kDrawThreads>(roots);
    pdl_wait();
    Group<NT> g(red);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int64_t row = blockIdx.x; row < a.r.rows; row += gridDim.x) {
        RowCta<TYPE, NT> c{Row<TYPE>(a.r, row), 0, &plan, roots, &sel, sums};
        c.vecs = (c.r.head + c.r.cols + E - 1) / E;
        float m = absent<TYPE>();
        c.each([&](float v, int64_t) { m = max_nan(m, v); });
        m = g.max(m);
        Filters f;
        const bool valid = filters_of(a, row, f);
        __syncthreads();
        if (threadIdx.x == 0) {
            plan_row<TYPE>(plan, m, valid, f);
            if (!valid) flag_bad_id(a.r, row);
        }
        __syncthreads();
        if (plan.state != kDraw) {
            no_draws(a, row, plan.state);
            continue;
        }
        if (!plan.greedy) {
            float s = 0.f;
            c.each([&](float v, int64_t) {
                if (v != absent<TYPE>()) s += rough_weight<TYPE>(plan, v);
            });
            s = g.sum(s);
            if (threadIdx.x == 0) plan.shift = shift_of(s);
            __syncthreads();
        }
        uint64_t bound = kPresent;
        if (plan.greedy) {
            bound = c.template select<false>(1, kPresent);
        } else {
            if (f.top_k > 0 && f.top_k < a.r.cols) bound = c.template select<false>(f.top_k, bound);
            if (f.top_p < 1.f) {
                const uint64_t all = c.template total<true>(bound), t = share(fmaxf(f.top_p, 0.f), all, true);
                bound = c.template select<true>(t > 0 ? t : 1, bound);
            }
            if (f.min_p > 0.f) {
                const uint64_t least = static_cast<uint64_t>(order_key<TYPE>(least_value<TYPE>(plan, f.min_p))) << 32;
                if (least > bound) bound = least;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) plan.bound = bound;
        __syncthreads();
        // sums of pieces
        uint64_t *masses = a.masses + row * a.pieces;
        const int64_t pieces = (c.vecs + kPieceVecs - 1) / kPieceVecs;
        uint64_t total = 0, kept = 0;
        for (int64_t q = warp; q < pieces; q += NT / 32) {
            uint64_t own = 0;
            for (int i = 0; i < kPieceVecs / 32; ++i) {
                const int64_t j = q * kPieceVecs + i * 32 + lane;
                if (j >= c.vecs) break;
                float v[E];
                vector_values<TYPE>(c.r, j, v);
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (rank_of<TYPE>(v[k], j * E - c.r.head + k) >= bound) {
                        own += weight<TYPE>(plan, roots, v[k]);
                        ++kept;
                    }
            }
            total += own;
            own = warp_sum(own);
            if (lane == 0) masses[q] = own;
        }
        total = c.sum(total);
        kept = c.sum(kept);
        if (threadIdx.x == 0) a.kept[row] = static_cast<int64_t>(kept);
        __syncthreads();
        for (int64_t d = warp; d < a.draws; d += NT / 32)
            warp_draw<TYPE>(a, c.r, c.vecs, plan, roots, masses, pieces, nullptr, total, row * a.draws + d,
                            row);
        __syncthreads();
    }
}

// ---- rows in segments -------------------------------------------------------
//
// One CTA a segment, a kernel for each pass over the rows; the CTA that finishes a
// row's last segment does what follows for the row:
//   top_kernel      the largest entry and a rough sum of weights; then the row's plan
//   bins_kernel     weights (and numbers) by bins of the order value, where a row has
//                   a top_k or top_p; then the bin in which they cut
//   cut_kernel      that bin's entries into a list; then sorted, the last rank left
//   sums_kernel     sums of the weights left, by pieces and segments; then a few draws
//   draws_kernel    many draws, a warp each
// Passes are bound by memory or, those with weights, by arithmetic (some 60
// operations an entry); launches hide behind each other's ends.

struct RowState {
    RowPlan plan;
    float top_p, min_p;
    int32_t top_k;
    int32_t narrow;         // whether bins are wanted
    float bin_scale;
    int32_t slot_lo, slot_hi;   // slots (see slot_of) of the entries to sort
    uint32_t expected;      // their number
    uint64_t above, all;    // weights (or number, without top_p) before them, of all
    uint64_t total;         // weights left
    uint32_t arrived[4];
    uint32_t listed;
};

struct RowBins {
    unsigned long long mass[kBins];
    uint32_t count[kBins];
};

// Place of an order value on a scale from the largest down, of kBins bins of kBins
// slots: for logits linear, for amplitudes linear between powers of two.  A larger
// value's is never greater (roundings are monotone).
template <int TYPE>
__device__ __forceinline__ int slot_of(const RowPlan &p, float bin_scale, float v) {
    constexpr int kLast = kBins * kBins - 1;
    if constexpr (Entry<TYPE>::kReal) {
        const float t = (p.m - v) * bin_scale;
        return t < static_cast<float>(kLast) ? static_cast<int>(t) : kLast;
    } else {
        const uint32_t d = (__float_as_uint(p.m) - __float_as_uint(v)) >> 7;
        return d < kLast ? static_cast<int>(d) : kLast;
    }
}

template <int TYPE>
struct Segment {
    Row<TYPE> r;
    int64_t row, seg, vecs, lo, hi;     // vectors of the row and of the segment

    __device__ __forceinline__ explicit Segment(const SampleArgs &a)
        : r(a.r, static_cast<int64_t>(blockIdx.x / static_cast<uint32_t>(a.segs))) {
        row = blockIdx.x / static_cast<uint32_t>(a.segs);
        seg = blockIdx.x - row * a.segs;
        vecs = (r.head + r.cols + Entry<TYPE>::E - 1) / Entry<TYPE>::E;
        lo = seg * a.seg_pieces * kPieceVecs;
        hi = lo + a.seg_pieces * kPieceVecs;
        if (hi > vecs) hi = vecs;
    }
};

// Whether this CTA is the last of its row's to come here.  What the others wrote
// before is visible to it.
__device__ __forceinline__ bool last_of_row(const SampleArgs &a, RowState &s, int which) {
    __shared__ bool last;
    if (a.segs == 1) {
        __syncthreads();
        return true;
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomicAdd(&s.arrived[which], 1u) == a.segs - 1;
        if (last) s.arrived[which] = 0;
        __threadfence();
    }
    __syncthreads();
    return last;
}

template <int TYPE>
__global__ void __launch_bounds__(kDrawThreads) top_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ uint32_t red[4 * kDrawWarps];
    pdl_trigger();
    pdl_wait();
    Group<kDrawThreads> g(red);
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    Filters f;
    const bool valid = filters_of(a, c.row, f);
    // the sum relative to the largest entry so far
    const float ch = fminf(f.beta * kLog2E, 3.402823466e38f);
    float m = absent<TYPE>(), s = 0.f;
    each_vector<TYPE, kDrawThreads, 4>(c.r, c.lo, c.hi, [&](const float (&v)[E], int64_t) {
        float top = v[0];
#pragma unroll
        for (int i = 1; i < E; ++i) top = max_nan(top, v[i]);
        if (!(top <= m)) {
            if constexpr (Entry<TYPE>::kReal) s *= ex2((m - top) * ch);
            else if (f.beta != 1.f) s *= m > 0.f ? ex2(f.beta * (lg2(m) - lg2(top))) : 0.f;
            m = max_nan(m, top);
        }
        if constexpr (Entry<TYPE>::kReal) {
            if (top != absent<TYPE>()) {
#pragma unroll
                for (int i = 0; i < E; ++i) s += ex2((v[i] - m) * ch);
            }
        } else if (f.beta == 1.f) {
#pragma unroll
            for (int i = 0; i < E; ++i) s += v[i];
        } else if (m > 0.f) {
            const float l = lg2(m);
#pragma unroll
            for (int i = 0; i < E; ++i) s += v[i] > 0.f ? ex2(f.beta * (lg2(v[i]) - l)) : 0.f;
        }
    });
    // threads', then segments'
    const auto moved = [&](float from, float to) {
        if (from == absent<TYPE>()) return 0.f;
        if constexpr (Entry<TYPE>::kReal) return ex2((from - to) * ch);
        else return f.beta == 1.f ? 1.f : ex2(f.beta * (lg2(from) - lg2(to)));
    };
    const float own = m;
    m = g.max(m);
    s = g.sum(own == absent<TYPE>() ? 0.f : s * moved(own, m));
    if (a.segs > 1) {
        ulonglong2 *parts = a.partials + c.row * a.segs;
        if (threadIdx.x == 0)
            __stcg(&parts[c.seg], make_ulonglong2(__float_as_uint(m), __float_as_uint(s)));
        if (!last_of_row(a, st, 0)) return;
        m = absent<TYPE>();
        for (int64_t i = threadIdx.x; i < a.segs; i += kDrawThreads)
            m = max_nan(m, __uint_as_float(static_cast<uint32_t>(__ldcg(&parts[i]).x)));
        m = g.max(m);
        s = 0.f;
        for (int64_t i = threadIdx.x; i < a.segs; i += kDrawThreads) {
            const ulonglong2 p = __ldcg(&parts[i]);
            s += __uint_as_float(static_cast<uint32_t>(p.y)) * moved(__uint_as_float(static_cast<uint32_t>(p.x)), m);
        }
        s = g.sum(s);
    }
    __shared__ int state;
    if (threadIdx.x == 0) {
        RowPlan p;
        plan_row<TYPE>(p, m, valid, f);
        if (!valid) flag_bad_id(a.r, c.row);
        state = p.state;
        st.narrow = 0;
        st.listed = 0;
        if (p.state == kDraw) {
            if (!Entry<TYPE>::kReal && f.beta == 1.f) s *= p.down;
            p.shift = p.greedy ? 0 : shift_of(s);
            if (p.greedy) {
                p.bound = static_cast<uint64_t>(order_key<TYPE>(m)) << 32;
            } else {
                if (f.min_p > 0.f) p.bound = static_cast<uint64_t>(order_key<TYPE>(least_value<TYPE>(p, f.min_p))) << 32;
                st.narrow = (f.top_k > 0 && f.top_k < a.r.cols) || f.top_p < 1.f;
            }
        }
        st.plan = p;
        st.top_p = fmaxf(f.top_p, 0.f);
        st.top_k = f.top_k;
        // 32 bins a power of two in weight; for top_k, whose place has nothing to do with weights, 128
        // a unit of the logits at most
        const float scale = 32.f * p.ch;
        st.bin_scale = kBins * fminf(scale, f.top_k > 0 ? 128.f : 0x1p80f);
    }
    __syncthreads();
    if (state != kDraw) no_draws(a, c.row, state);
}

__device__ __forceinline__ void add_mass(uint32_t *lo, uint32_t *hi, uint64_t w) {
    const uint32_t l = static_cast<uint32_t>(w), old = atomicAdd(lo, l);
    const uint32_t h = static_cast<uint32_t>(w >> 32) + (old + l < l);
    if (h) atomicAdd(hi, h);
}

// exclusive prefix sums over the CTA's threads; `sums` has kDrawWarps + 1 places, the
// last for the total
__device__ __forceinline__ uint64_t cta_scan(uint64_t x, uint64_t *sums) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint64_t upto = warp_scan(x, lane);
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    uint64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kDrawWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    if (threadIdx.x == 0) sums[kDrawWarps] = total;
    __syncthreads();
    return before + upto - x;
}

// FINE: the bins are the slots of the bin in which the first pass ended, where it
// has more entries than are sorted.
template <int TYPE, bool FINE>
__global__ void __launch_bounds__(kDrawThreads) bins_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E, kOwn = kBins / kDrawThreads;
    __shared__ uint32_t lo[kBins], hi[kBins], count[kBins];
    __shared__ float2 roots[kRoots];
    __shared__ uint64_t sums[kDrawWarps + 1], nums[kDrawWarps + 1];
    pdl_trigger();
    make_roots<kDrawThreads>(roots);
    for (int i = threadIdx.x; i < kBins; i += kDrawThreads) lo[i] = hi[i] = count[i] = 0;
    pdl_wait();
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    if (!st.narrow || (FINE && (st.expected <= kSorted || st.slot_hi - st.slot_lo != kBins - 1))) return;
    const RowPlan p = st.plan;
    const float bin_scale = st.bin_scale;
    const bool by_mass = st.top_p < 1.f;
    const int64_t k = st.top_k > 0 && st.top_k < a.r.cols ? st.top_k : 0;
    const int first = FINE ? st.slot_lo : 0;
    const uint64_t above0 = FINE ? st.above : 0;
    __syncthreads();
    each_vector<TYPE, kDrawThreads, 2>(c.r, c.lo, c.hi, [&](const float (&v)[E], int64_t) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (v[i] == absent<TYPE>()) continue;
            int b = slot_of<TYPE>(p, bin_scale, v[i]) - first;
            if (!FINE) b /= kBins;
            if (FINE && (b < 0 || b >= kBins)) continue;
            atomicAdd(&count[b], 1u);
            if (by_mass) add_mass(&lo[b], &hi[b], weight<TYPE>(p, roots, v[i]));
        }
    });
    __syncthreads();
    RowBins *all = a.segs > 1 ? a.bins + c.row : nullptr;
    if (all) {
        for (int i = threadIdx.x; i < kBins; i += kDrawThreads)
            if (count[i]) {
                atomicAdd(&all->count[i], count[i]);
                if (by_mass) atomicAdd(&all->mass[i], static_cast<unsigned long long>(hi[i]) << 32 | lo[i]);
            }
        if (!last_of_row(a, st, 1)) return;
    }
    uint64_t mass[kOwn], own_mass = 0, own_count = 0;
    uint32_t num[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int b = threadIdx.x * kOwn + i;
        num[i] = all ? __ldcg(&all->count[b]) : count[b];
        mass[i] = all ? __ldcg(&all->mass[b]) : static_cast<uint64_t>(hi[b]) << 32 | lo[b];
        if (all) {      // left clear
            all->count[b] = 0;
            all->mass[b] = 0;
        }
        own_mass += mass[i];
        own_count += num[i];
    }
    uint64_t before_mass = cta_scan(own_mass, sums), before_count = cta_scan(own_count, nums);
    const uint64_t total = sums[kDrawWarps], entries = nums[kDrawWarps];
    const bool cut_k = FINE ? k > 0 : k > 0 && static_cast<uint64_t>(k) < entries;
    if (!cut_k && !by_mass) {       // fewer entries than top_k
        if (threadIdx.x == 0) st.narrow = 0;
        return;
    }
    uint64_t target = cut_k ? k : share(st.top_p, FINE ? st.all : total, true);
    if (target == 0) target = 1;
    uint64_t before = above0 + (cut_k ? before_count : before_mass), through = before_count;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const uint64_t x = cut_k ? num[i] : mass[i];
        through += num[i];
        if (before < target && before + x >= target) {      // one thread, one bin
            const int b = threadIdx.x * kOwn + i;
            // with both filters the second needs all that the first leaves
            const bool both = cut_k && by_mass;
            st.slot_lo = both ? 0 : FINE ? first + b : b * kBins;
            st.slot_hi = FINE ? first + b : b * kBins + kBins - 1;
            st.expected = static_cast<uint32_t>(both ? through : num[i]);
            st.above = both ? 0 : before;
            st.all = FINE ? st.all : total;
            if (!cut_k) st.top_k = 0;
        }
        before += x;
    }
}

// Ranks in descending order; n a power of two.
__device__ __forceinline__ void sort_ranks(uint64_t *x, int n) {
    for (int size = 2; size <= n; size *= 2)
        for (int step = size / 2; step; step /= 2) {
            __syncthreads();
            for (int t = threadIdx.x; t < n / 2; t += kDrawThreads) {
                const int i = 2 * t - (t & (step - 1)), j = i + step;
                const uint64_t y = x[i], z = x[j];
                if ((y < z) == ((i & size) == 0)) {
                    x[i] = z;
                    x[j] = y;
                }
            }
        }
    __syncthreads();
}

template <int TYPE>
__global__ void __launch_bounds__(kDrawThreads) cut_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ uint64_t list[kSorted];
    __shared__ float2 roots[kRoots];
    __shared__ Select sel;
    __shared__ uint64_t sums[kDrawWarps + 1];
    __shared__ RowPlan plan;
    __shared__ uint32_t listed;
    pdl_trigger();
    make_roots<kDrawThreads>(roots);
    pdl_wait();
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    if (!st.narrow) return;
    const bool by_mass = st.top_p < 1.f, sorted = st.expected <= kSorted;
    if (threadIdx.x == 0) {
        plan = st.plan;
        listed = 0;
    }
    __syncthreads();
    uint64_t *to = a.segs > 1 ? a.lists + c.row * kSorted : list;
    uint32_t *counter = a.segs > 1 ? &st.listed : &listed;
    if (sorted) {
        const float bin_scale = st.bin_scale;
        const int lo = st.slot_lo, hi = st.slot_hi;
        const RowPlan own = plan;       // (not read again behind every atomic)
        each_vector<TYPE, kDrawThreads, 4>(c.r, c.lo, c.hi, [&](const float (&v)[E], int64_t j) {
            uint32_t in = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int s = slot_of<TYPE>(own, bin_scale, v[i]);
                if (v[i] != absent<TYPE>() && s >= lo && s <= hi) in |= 1u << i;
            }
            if (!in) return;
            uint32_t at = atomicAdd(counter, static_cast<uint32_t>(__popc(in)));
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (in >> i & 1) {
                    if (at < kSorted) to[at] = rank_of<TYPE>(v[i], j * E - c.r.head + i);
                    ++at;
                }
        });
    }
    if (!last_of_row(a, st, 2)) return;
    uint64_t bound = kPresent;
    if (sorted) {
        const uint32_t found = a.segs > 1 ? __ldcg(&st.listed) : listed;
        const int n = static_cast<int>(found < kSorted ? found : kSorted);
        int room = 2;
        while (room < n) room *= 2;
        for (int i = threadIdx.x; i < room; i += kDrawThreads)
            list[i] = i >= n ? 0 : a.segs > 1 ? __ldcg(&to[i]) : list[i];
        sort_ranks(list, room);
        int64_t left = n;
        if (st.top_k > 0) {
            left = st.top_k - static_cast<int64_t>(by_mass ? 0 : st.above);
            if (left > n) left = n;
            bound = list[left > 0 ? left - 1 : 0];
        }
        if (by_mass) {
            // of consecutive ranks, a thread each
            const int per = static_cast<int>((left + kDrawThreads - 1) / kDrawThreads);
            const int lo = threadIdx.x * per < left ? threadIdx.x * per : static_cast<int>(left);
            const int hi = lo + per < left ? lo + per : static_cast<int>(left);
            uint64_t own = 0;
            for (int i = lo; i < hi; ++i)
                own += weight<TYPE>(plan, roots, key_value(static_cast<uint32_t>(list[i] >> 32)));
            uint64_t upto = st.above + cta_scan(own, sums);
            uint64_t target = share(st.top_p, st.top_k > 0 ? sums[kDrawWarps] : st.all, true);
            if (target == 0) target = 1;
            __shared__ uint64_t cut;
            if (threadIdx.x == 0) cut = left > 0 ? list[left - 1] : kPresent;
            __syncthreads();
            for (int i = lo; i < hi; ++i) {
                const uint64_t w = weight<TYPE>(plan, roots, key_value(static_cast<uint32_t>(list[i] >> 32)));
                if (upto < target && upto + w >= target) cut = list[i];
                upto += w;
            }
            __syncthreads();
            bound = cut;
        }
    } else {
        // more equal (or nearly equal) entries than are sorted: digit by digit
        RowCta<TYPE, kDrawThreads> cta{c.r, c.vecs, &plan, roots, &sel, sums};
        if (st.top_k > 0) bound = cta.template select<false>(st.top_k, bound);
        if (by_mass) {
            const uint64_t all = cta.template total<true>(bound), t = share(st.top_p, all, true);
            bound = cta.template select<true>(t > 0 ? t : 1, bound);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        st.listed = 0;
        if (bound > plan.bound) st.plan.bound = bound;
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kDrawThreads) sums_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ float2 roots[kRoots];
    __shared__ uint64_t sums[kDrawWarps + 1], nums[kDrawWarps + 1];
    pdl_trigger();
    make_roots<kDrawThreads>(roots);
    pdl_wait();
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    const RowPlan p = st.plan;
    if (p.state != kDraw) return;
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t *masses = a.masses + c.row * a.pieces;
    uint64_t total = 0, kept = 0;
    uint32_t number = 0;
    const uint32_t bound_key = static_cast<uint32_t>(p.bound >> 32), bound_index = 0xffffffffu - static_cast<uint32_t>(p.bound);
    int64_t in_lo, in_hi;
    c.r.inside_range(in_lo, in_hi);
    for (int64_t q = c.lo / kPieceVecs + warp; q * kPieceVecs < c.hi; q += kDrawWarps) {
        uint64_t own = 0;
        vectors_at<TYPE, kPieceVecs / 32>(
            c.r, in_lo, in_hi, q * kPieceVecs, (q + 1) * kPieceVecs, q * kPieceVecs + lane, 32, c.hi,
            [&](const float (&v)[E], int64_t j) {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const uint32_t key = order_key<TYPE>(v[k]);
                    if (key > bound_key ||
                        (key == bound_key && static_cast<uint32_t>(j * E - c.r.head + k) <= bound_index)) {
                        own += weight<TYPE>(p, roots, v[k]);
                        ++number;
                    }
                }
            });
        total += own;
        own = warp_sum(own);
        if (lane == 0) __stcg(&masses[q], own);
    }
    kept = number;
    cta_scan(total, sums);
    cta_scan(kept, nums);
    total = sums[kDrawWarps];
    kept = nums[kDrawWarps];
    const ulonglong2 *parts = nullptr;
    if (a.segs > 1) {
        ulonglong2 *mine = a.partials + c.row * a.segs;
        if (threadIdx.x == 0) __stcg(&mine[c.seg], make_ulonglong2(total, kept));
        if (!last_of_row(a, st, 3)) return;
        parts = mine;
        // sums up to each segment, of consecutive ones by a thread each
        const int per = static_cast<int>((a.segs + kDrawThreads - 1) / kDrawThreads), s0 = threadIdx.x * per;
        total = kept = 0;
        for (int i = s0; i < s0 + per && i < a.segs; ++i) {
            const ulonglong2 x = __ldcg(&mine[i]);
            total += x.x;
            kept += x.y;
        }
        cta_scan(kept, nums);
        uint64_t upto = cta_scan(total, sums);
        for (int i = s0; i < s0 + per && i < a.segs; ++i) {
            const ulonglong2 x = __ldcg(&mine[i]);
            upto += x.x;
            __stcg(&mine[i], make_ulonglong2(upto, x.y));
        }
        __syncthreads();
        total = sums[kDrawWarps];
        kept = nums[kDrawWarps];
    } else {
        __syncthreads();        // the pieces' sums
    }
    if (threadIdx.x == 0) {
        a.kept[c.row] = p.greedy ? 1 : static_cast<int64_t>(kept);
        st.total = total;
    }
    if (a.draws > kFewDraws) return;
    const int64_t pieces = (c.vecs + kPieceVecs - 1) / kPieceVecs;
    for (int64_t d = warp; d < a.draws; d += kDrawWarps)
        warp_draw<TYPE>(a, c.r, c.vecs, p, roots, masses, pieces, parts, total, c.row * a.draws + d, c.row);
}

template <int TYPE>
__global__ void __launch_bounds__(kDrawThreads) draws_kernel(const __grid_constant__ SampleArgs a) {
    __shared__ float2 roots[kRoots];
    pdl_trigger();
    make_roots<kDrawThreads>(roots);
    pdl_wait();
    __syncthreads();
    const int64_t ctas = (a.draws + kDrawWarps - 1) / kDrawWarps;
    const int64_t row = blockIdx.x / ctas, d = (blockIdx.x - row * ctas) * kDrawWarps + threadIdx.x / 32;
    const RowState &st = a.state[row];
    const RowPlan p = st.plan;
    if (p.state != kDraw || d >= a.draws) return;
    const Row<TYPE> r(a.r, row);
    const int64_t vecs = (r.head + r.cols + Entry<TYPE>::E - 1) / Entry<TYPE>::E;
    warp_draw<TYPE>(a, r, vecs, p, roots, a.masses + row * a.pieces, (vecs + kPieceVecs - 1) / kPieceVecs,
                    a.segs > 1 ? a.partials + row * a.segs : nullptr, st.total, row * a.draws + d, row);
}

template <int TYPE>
cudaError_t sample_of(const SampleArgs &a, cudaStream_t stream) {
    const dim3 block(kDrawThreads);
    if (!a.state) {
        const int64_t ctas = a.r.rows < kDrawTarget ? a.r.rows : kDrawTarget;
        return launch_pdl(sample_rows_kernel<TYPE, kDrawThreads>, dim3(static_cast<unsigned>(ctas)), block, 0, stream, a);
    }
    const dim3 grid(static_cast<unsigned>(a.r.rows * a.segs));
    cudaError_t e = launch_pdl(top_kernel<TYPE>, grid, block, 0, stream, a);
    if (e == cudaSuccess && a.filtered) {
        e = launch_pdl(bins_kernel<TYPE, false>, grid, block, 0, stream, a);
        if (e == cudaSuccess && a.r.cols >= kLongRow)
            e = launch_pdl(bins_kernel<TYPE, true>, grid, block, 0, stream, a);
        if (e == cudaSuccess) e = launch_pdl(cut_kernel<TYPE>, grid, block, 0, stream, a);
    }
    if (e == cudaSuccess) e = launch_pdl(sums_kernel<TYPE>, grid, block, 0, stream, a);
    if (e == cudaSuccess && a.draws > kFewDraws) {
        const int64_t ctas = a.r.rows * ((a.draws + kDrawWarps - 1) / kDrawWarps);
        e = launch_pdl(draws_kernel<TYPE>, dim3(static_cast<unsigned>(ctas)), block, 0, stream, a);
    }
    return e;
}

}  // namespace tn
