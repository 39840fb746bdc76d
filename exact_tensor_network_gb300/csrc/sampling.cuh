// Drawing outcomes from rows: weights, filters and draws.
//
// An outcome is a whole number, and near a border between two outcomes any
// rounding decides it: a sum of 10^5 weights in fp32 is wrong by some 2^-22, and one
// draw in ten of a broad row lies that near to a border.  So weights are computed as
// pairs of fp32 numbers (44 bits and more) and summed as 64-bit integers, in
// units of 2^-shift of the largest, the shift chosen by an estimate of the row's
// sum so that it uses 61 bits.  Integer sums need no order: histograms by
// shared-memory atomics, partial sums of CTAs and of warps are all exact.
#pragma once

#include "outcomes.cuh"
#include "sampling.h"

namespace tn {

// 2^(j/64) as the sum of two fp32 numbers
static __device__ const float2 kRoots[64] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.02c9a4p+0f, -0x1.887fa0p-28f},
    {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.087452p+0f, -0x1.e2990ep-26f},
    {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.1429aap+0f, 0x1.d525bcp-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1a35bep+0f, 0x1.6df96ep-25f},
    {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f},
    {0x1.29e9e0p+0f, -0x1.5c0424p-25f}, {0x1.2d285ap+0f, 0x1.b900c2p-26f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f}, {0x1.33c08cp+0f, -0x1.b37d20p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f},
    {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.4160a2p+0f, 0x1.f72e2ap-28f},
    {0x1.44e086p+0f, 0x1.8624b4p-30f}, {0x1.486a2cp+0f, -0x1.47d866p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f},
    {0x1.5342b6p+0f, -0x1.2c5610p-25f}, {0x1.56f474p+0f, -0x1.295b04p-25f},
    {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f},
    {0x1.6247ecp+0f, -0x1.f8b550p-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.6dfb24p+0f, -0x1.cd72e8p-27f},
    {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.7e2f34p+0f, -0x1.261634p-25f},
    {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.868d9ap+0f, -0x1.2edb44p-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f},
    {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a0c668p+0f, -0x1.2886a6p-26f},
    {0x1.a5503cp+0f, -0x1.b83b54p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f},
    {0x1.b7f770p+0f, -0x1.a09438p-25f}, {0x1.bcc1eap+0f, -0x1.f687c6p-25f},
    {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.d072d4p+0f, 0x1.40f130p-25f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.da9e60p+0f, 0x1.ed9942p-27f},
    {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f},
    {0x1.f50766p+0f, -0x1.246eb0p-26f}, {0x1.fa7c18p+0f, 0x1.9e90d8p-28f},
};

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
// first entry left).  2^t of a pair t: 2^(k/64) from a table, the rest (at most
// 2^-7) by the exponential series, whose first two terms are kept as pairs.
__device__ __forceinline__ uint64_t weight_real(const RowPlan &p, const float2 *roots, float v) {
    constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f, kMagic = 12582912.f;
    const float2 t = exponent(p, v);
    if (!(t.x > -64.f)) return 1;
    const float kf = __fadd_rn(fmaf(t.x, 64.f, kMagic), -kMagic);
    const float r = fmaf(kf, -0x1p-6f, t.x);                // exact
    const float g = r * kLn2Hi;
    const float gl = fmaf(r, kLn2Hi, -g) + fmaf(r, kLn2Lo, t.y * kLn2Hi);
    const float s = g * g, sl = fmaf(g, g, -s), half = 0.5f * s;
    const float tail = g * s * fmaf(g, 1.f / 24, 1.f / 6);
    const float q = g + half;                               // 2^r - 1 = q + ql
    const float ql = ((g - q) + half) + fmaf(g, gl, 0.5f * sl) + (gl + tail);
    const int k = static_cast<int>(kf);
    const float2 root = roots[k & 63];
    const float a = root.x * q, al = fmaf(root.x, q, -a);
    const float w = root.x + a;
    const float wl = ((root.x - w) + a) + (al + root.y + fmaf(root.x, ql, root.y * q));
    const int x = (k >> 6) + p.shift;
    if (x < -1) return 1;
    const float unit = __uint_as_float(static_cast<uint32_t>(x + 127) << 23);
    const long long n = __float2ll_rn(w * unit) + __float2ll_rn(wl * unit);
    return n > 0 ? static_cast<uint64_t>(n) : 1;
}

template <int TYPE>
__device__ __forceinline__ uint64_t weight(const RowPlan &p, const float2 *roots, float v) {
    if constexpr (Entry<TYPE>::kReal) {
        return weight_real(p, roots, v);
    } else {
        long long n;
        if (p.beta == 1.0) {
            n = __float2ll_rn(v * p.down * __uint_as_float(static_cast<uint32_t>(p.shift + 127) << 23));
        } else {
            const double x = p.beta * log(static_cast<double>(v) / p.m);
            n = x < -60.0 ? 1 : __double2ll_rn(ldexp(exp(x), p.shift));
        }
        return n > 0 ? static_cast<uint64_t>(n) : 1;
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
    frexpf(sum * 1.001f, &x);
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
        for (int64_t j = threadIdx.x; j < vecs; j += NT) {
            float v[E];
            vector_values<TYPE>(r, j, v);
#pragma unroll
            for (int i = 0; i < E; ++i) f(v[i], j * E - r.head + i);
        }
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

// One warp: a draw of row r from its pieces' sums.
template <int TYPE>
__device__ void warp_draw(const SampleArgs &a, const Row<TYPE> &r, int64_t vecs, const RowPlan &p, const float2 *roots,
                          const uint64_t *masses, int64_t pieces, uint64_t total, int64_t at, int64_t row) {
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
    uint64_t target = share(u, total, false);
    int64_t piece = 0;
    for (int64_t base = 0; base < pieces; base += 32) {
        const uint64_t own = base + lane < pieces ? masses[base + lane] : 0, upto = warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, upto > target);
        if (over) {
            const int l = __ffs(over) - 1;
            target -= shfl_from(upto - own, l);
            piece = base + l;
            break;
        }
        target -= shfl_from(upto, 31);
    }
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

template <int TYPE, int NT>
__global__ void __launch_bounds__(NT) sample_rows_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ float2 roots[64];
    __shared__ RowPlan plan;
    __shared__ Select sel;
    __shared__ uint64_t sums[NT / 32];
    __shared__ uint32_t red[4 * (NT / 32)];
    pdl_trigger();
    if (threadIdx.x < 64) roots[threadIdx.x] = kRoots[threadIdx.x];
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
            for (int64_t d = threadIdx.x; d < a.draws; d += NT) {
                a.ids[row * a.draws + d] = -1;
                a.logp[row * a.draws + d] = plan.state == kEmpty ? -__builtin_huge_valf() : __uint_as_float(0x7fc00000u);
            }
            if (threadIdx.x == 0) a.kept[row] = 0;
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
            warp_draw<TYPE>(a, c.r, c.vecs, plan, roots, masses, pieces, total, row * a.draws + d, row);
        __syncthreads();
    }
}

template <int TYPE>
cudaError_t sample_of(const SampleArgs &a, cudaStream_t stream) {
    const int64_t ctas = a.r.rows < 8 * kOutSms ? a.r.rows : 8 * kOutSms;
    return launch_pdl(sample_rows_kernel<TYPE, kRowThreads>, dim3(static_cast<unsigned>(ctas)), dim3(kRowThreads), 0,
                      stream, a);
}

}  // namespace tn
