// Device helpers of the operators on outcome distributions: reading rows
// (types, strides, masks), groups of threads that share a row, teachers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "outcomes.h"

namespace tn {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Results below 2^-126 are flushed to 0: next to sums that hold a term of
// about 1 they are nothing, and keeping them costs three more instructions.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 bytes from global to shared memory, asynchronously
__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return reinterpret_cast<float2 &>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return reinterpret_cast<float2 &>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return reinterpret_cast<float2 &>(d);
}
// larger of two, NaN if either is (a row with a NaN has no distribution: it
// must not be lost in a maximum)
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// largest of a warp's
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// NaN if one is
__device__ __forceinline__ float warp_max_nan(float x) {
    float y;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// ---- entries ----------------------------------------------------------------
//
// An entry is worked on as its order value v, by which alternatives are
// ranked: the logit itself, or w = re^2 + im^2 of an amplitude with every
// operation rounded (no fused multiply-add, so that equal amplitudes tie in
// any other implementation of the definition too).  kAbsent marks an absent
// entry.

// Mask bytes: 0x80 in every nonzero byte; those bits spread over the bytes
// that a selector names; one of two by such a mask.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t x) {
    return (((x & 0x7f7f7f7fu) + 0x7f7f7f7fu) | x) & 0x80808080u;
}
__device__ __forceinline__ uint32_t spread(uint32_t k, uint32_t selector) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(d) : "r"(k), "r"(selector));
    return d;
}
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t mask, uint32_t b) {
    return (a & mask) | (b & ~mask);
}
__device__ __forceinline__ void blank16(uint4 &r, uint64_t keep, uint32_t absent) {
    const uint32_t a = nonzero_bytes(static_cast<uint32_t>(keep));
    const uint32_t b = nonzero_bytes(static_cast<uint32_t>(keep >> 32));
    r.x = pick(r.x, spread(a, 0x9988), absent);
    r.y = pick(r.y, spread(a, 0xbbaa), absent);
    r.z = pick(r.z, spread(b, 0x9988), absent);
    r.w = pick(r.w, spread(b, 0xbbaa), absent);
}

// absent_vector: 16 bytes of absent entries; blank: make the entries absent
// whose mask byte is 0.
template <int TYPE>
struct Entry;

template <>
struct Entry<TN_TYPE_F32> {
    using T = float;
    static constexpr int E = 4;
    static constexpr bool kReal = true;
    static __device__ __forceinline__ float value(T x) { return x; }
    static __device__ __forceinline__ void values(const uint4 &r, float (&v)[E]) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 absent_vector() {
        return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
    }
    static __device__ __forceinline__ void blank(uint4 &r, uint32_t keep) {
        const uint32_t k = nonzero_bytes(keep);
        r.x = pick(r.x, spread(k, 0x8888), 0xff800000u);
        r.y = pick(r.y, spread(k, 0x9999), 0xff800000u);
        r.z = pick(r.z, spread(k, 0xaaaa), 0xff800000u);
        r.w = pick(r.w, spread(k, 0xbbbb), 0xff800000u);
    }
};

template <>
struct Entry<TN_TYPE_BF16> {
    using T = __nv_bfloat16;
    static constexpr int E = 8;
    static constexpr bool kReal = true;
    static __device__ __forceinline__ float value(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ void values(const uint4 &r, float (&v)[E]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 absent_vector() {
        return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    }
    static __device__ __forceinline__ void blank(uint4 &r, uint64_t keep) { blank16(r, keep, 0xff80ff80u); }
};

template <>
struct Entry<TN_TYPE_F16> {
    using T = __half;
    static constexpr int E = 8;
    static constexpr bool kReal = true;
    static __device__ __forceinline__ float value(T x) { return __half2float(x); }
    static __device__ __forceinline__ void values(const uint4 &r, float (&v)[E]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 absent_vector() {
        return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
    }
    static __device__ __forceinline__ void blank(uint4 &r, uint64_t keep) { blank16(r, keep, 0xfc00fc00u); }
};

template <>
struct Entry<TN_TYPE_C64> {
    using T = float2;
    static constexpr int E = 2;
    static constexpr bool kReal = false;
    static __device__ __forceinline__ float value(T a) {
        return __fadd_rn(__fmul_rn(a.x, a.x), __fmul_rn(a.y, a.y));
    }
    static __device__ __forceinline__ void values(const uint4 &r, float (&v)[E]) {
        v[0] = value(make_float2(__uint_as_float(r.x), __uint_as_float(r.y)));
        v[1] = value(make_float2(__uint_as_float(r.z), __uint_as_float(r.w)));
    }
    static __device__ __forceinline__ uint4 absent_vector() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void blank(uint4 &r, uint32_t keep) {
        if (!(keep & 0xff)) r.x = r.y = 0;
        if (!(keep & 0xff00)) r.z = r.w = 0;
    }
};

template <int TYPE>
__device__ __forceinline__ constexpr float absent() {
    return Entry<TYPE>::kReal ? -__builtin_huge_valf() : 0.f;
}

// Order value as an unsigned integer of the same order (-0 and +0 equal); 0
// for absent entries.
template <int TYPE>
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return v == absent<TYPE>() ? 0u : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// ---- one row ----------------------------------------------------------------
//
// Vectors are 16-byte pieces of the row that start at 16-byte boundaries:
// vector j holds entries j E - head .. j E - head + E - 1, of which those in
// [0, cols) exist.  Only vectors that lie inside the row are read as such;
// the others (and every vector of a strided row, where head is 0) entry by
// entry.
//
// Vectors and masks are read past the L1 cache, which they would only pass
// through: a grid starts before the one that writes its rows has ended, so it
// may not take them for constant (1 to 3 % on 16-bit rows, whose search reads
// some vectors twice).

template <int TYPE>
struct Row {
    using En = Entry<TYPE>;
    const typename En::T *p;
    const uint8_t *m;
    int64_t cols, cs, mcs;
    int head;

    __device__ __forceinline__ Row(const OutRows &a, int64_t row)
        : p(reinterpret_cast<const typename En::T *>(a.data) + row * a.row_stride),
          m(a.mask ? a.mask + row * a.mask_row_stride : nullptr),
          cols(a.cols), cs(a.col_stride), mcs(a.mask_col_stride), head(0) {
        if (cs == 1)
            head = static_cast<int>((reinterpret_cast<uintptr_t>(p) % kOutVecBytes) / sizeof(typename En::T));
    }
    __device__ __forceinline__ bool inside(int64_t e0) const {
        return cs == 1 && e0 >= 0 && e0 + En::E <= cols;
    }
    __device__ __forceinline__ uint4 raw(int64_t e0) const {
        return __ldcg(reinterpret_cast<const uint4 *>(p + e0));
    }
    __device__ __forceinline__ bool kept(int64_t e) const { return !m || m[e * mcs] != 0; }
    __device__ __forceinline__ float value(int64_t e) const {
        return kept(e) ? En::value(p[e * cs]) : absent<TYPE>();
    }
    // The mask bytes of the vector at e0, which lies inside the row, entry i in
    // byte i.  They lie at any offset from the data's vectors: one aligned
    // word, or two and a shift where both are inside the mask's row.
    using Keep = typename std::conditional<En::E == 8, uint64_t, uint32_t>::type;
    // whether every vector's mask bytes are one aligned word
    __device__ __forceinline__ bool mask_words() const {
        return mcs == 1 && (reinterpret_cast<uintptr_t>(m) - head) % En::E == 0;
    }
    __device__ __forceinline__ Keep keep_word(int64_t e0) const {
        if constexpr (En::E == 2) return __ldcg(reinterpret_cast<const uint16_t *>(m + e0));
        else return __ldcg(reinterpret_cast<const Keep *>(m + e0));
    }
    __device__ __forceinline__ Keep keep(int64_t e0) const {
        constexpr int E = En::E;
        if constexpr (E >= 4) {
            if (mcs == 1) {
                const uint8_t *q = m + e0;
                const int off = static_cast<int>(reinterpret_cast<uintptr_t>(q) % E);
                const uint8_t *b = q - off;
                if (off == 0) return __ldcg(reinterpret_cast<const Keep *>(b));
                if (b >= m && b + 2 * E <= m + cols) {
                    const Keep lo = __ldcg(reinterpret_cast<const Keep *>(b));
                    const Keep hi = __ldcg(reinterpret_cast<const Keep *>(b) + 1);
                    return (lo >> (8 * off)) | (hi << (8 * (E - off)));
                }
            }
        }
        Keep w = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) w |= static_cast<Keep>(m[(e0 + i) * mcs]) << (8 * i);
        return w;
    }
    // vectors [lo, hi) lie inside the row
    __device__ __forceinline__ void inside_range(int64_t &lo, int64_t &hi) const {
        lo = cs == 1 ? (head + En::E - 1) / En::E : 0;
        hi = cs == 1 ? (head + cols) / En::E : 0;
    }
    __device__ __forceinline__ const uint4 *vectors() const {
        return reinterpret_cast<const uint4 *>(p - head);
    }
};

// Out of line, for what is not in a kernel's steady loop (inlined, these
// would be most of its code, and that code's instruction-cache misses most of
// a short row's time).
template <int E>
struct Values {
    float v[E];
};

template <int TYPE>
__device__ __noinline__ typename Row<TYPE>::Keep row_keep(const Row<TYPE> r, int64_t e0) {
    return r.keep(e0);
}

// order value of entry e
template <int TYPE>
__device__ __noinline__ float row_value(const Row<TYPE> r, int64_t e) {
    return r.value(e);
}

// order values of vector j, absent outside the row
template <int TYPE>
__device__ __noinline__ Values<Entry<TYPE>::E> row_vector(const Row<TYPE> r, int64_t j) {
    using En = Entry<TYPE>;
    Values<En::E> o;
    const int64_t e0 = j * En::E - r.head;
    if (r.inside(e0)) {
        uint4 q = r.raw(e0);
        if (r.m) En::blank(q, row_keep<TYPE>(r, e0));
        En::values(q, o.v);
    } else {
#pragma unroll
        for (int i = 0; i < En::E; ++i) {
            const int64_t e = e0 + i;
            o.v[i] = absent<TYPE>();
            if (e >= 0 && e < r.cols) o.v[i] = r.value(e);
        }
    }
    return o;
}

// ---- groups -----------------------------------------------------------------
//
// G threads that share a row: a warp or the whole CTA.  Sums and scans of a
// CTA go through `red`, two halves used in turn so that each needs one barrier.

template <int G>
struct Group {
    static constexpr int kWarps = G / 32;
    int t, lane, warp;   // thread in the group, lane, warp in the group
    uint32_t *red;       // 2 * 2 * kWarps words (unused by a warp)
    int half;

    __device__ __forceinline__ explicit Group(uint32_t *r)
        : t(threadIdx.x % G), lane(threadIdx.x % 32), warp(threadIdx.x % G / 32), red(r), half(0) {}
    __device__ __forceinline__ void sync() const {
        if constexpr (G == 32) __syncwarp();
        else __syncthreads();
    }
    __device__ __forceinline__ uint32_t *slot() {
        half ^= 1;
        return red + half * 2 * kWarps;
    }
    __device__ __forceinline__ uint32_t sum(uint32_t x) {
        x = __reduce_add_sync(0xffffffffu, x);
        if constexpr (G > 32) {
            uint32_t *s = slot();
            if (lane == 0) s[warp] = x;
            __syncthreads();
            x = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x += s[w];
        }
        return x;
    }
    __device__ __forceinline__ uint32_t max(uint32_t x) {
        x = __reduce_max_sync(0xffffffffu, x);
        if constexpr (G > 32) {
            uint32_t *s = slot();
            if (lane == 0) s[warp] = x;
            __syncthreads();
            x = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x = ::max(x, s[w]);
        }
        return x;
    }
    // NaN if any is
    __device__ __forceinline__ float max(float x) {
#pragma unroll
        for (int o = 16; o; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
        if constexpr (G > 32) {
            uint32_t *s = slot();
            if (lane == 0) s[warp] = __float_as_uint(x);
            __syncthreads();
            x = __uint_as_float(s[0]);
#pragma unroll
            for (int w = 1; w < kWarps; ++w) x = max_nan(x, __uint_as_float(s[w]));
        }
        return x;
    }
    // two sums, added in a fixed order
    __device__ __forceinline__ void sum2(float &x, float &y) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, o);
            y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        if constexpr (G > 32) {
            uint32_t *s = slot();
            if (lane == 0) {
                s[2 * warp] = __float_as_uint(x);
                s[2 * warp + 1] = __float_as_uint(y);
            }
            __syncthreads();
            x = y = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                x += __uint_as_float(s[2 * w]);
                y += __uint_as_float(s[2 * w + 1]);
            }
        }
    }
    __device__ __forceinline__ float sum(float x) {
        float y = 0.f;
        sum2(x, y);
        return x;
    }
    // exclusive prefix sums of two counters over the group's threads
    __device__ __forceinline__ void scan2(uint32_t &x, uint32_t &y) {
        const uint32_t x0 = x, y0 = y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += a;
                y += b;
            }
        }
        if constexpr (G > 32) {
            uint32_t *s = slot();
            if (lane == 31) {
                s[2 * warp] = x;
                s[2 * warp + 1] = y;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (w < warp) {
                    x += s[2 * w];
                    y += s[2 * w + 1];
                }
        }
        x -= x0;
        y -= y0;
    }
};

// ---- ids and teachers -------------------------------------------------------

__device__ __forceinline__ void flag_bad_id(const OutRows &a, int64_t row) {
    if (atomicCAS(&a.status->code, ERR_NONE, ERR_DESC) == ERR_NONE)
        a.status->where = static_cast<int32_t>(row);
}

// A row's teacher in shared memory: ids (-1 where left out), probabilities,
// their logarithms and, where the loss is wanted, the row's order values
// there, in teacher_bytes(count) at `base`.  The group reads it (its loads in
// flight together) with read(); after a barrier one warp normalises it.
struct Teacher {
    int64_t *id;
    float *q, *logq, *value;
    float *used;   // 1 if anything is left, else 0

    __device__ __forceinline__ Teacher(void *base, int count)
        : id(static_cast<int64_t *>(base)), q(reinterpret_cast<float *>(id + count)), logq(q + count),
          value(logq + count), used(value + count) {}

    // one of the row's outcomes, between its loads and its place: item() loads
    // it, look() what the row holds there, settle() waits for that
    template <int TYPE>
    struct Item {
        int64_t x;
        float l;
        typename Entry<TYPE>::T v;
        uint8_t keep;
    };
    template <int TYPE>
    static __device__ __forceinline__ Item<TYPE> item(const OutTeacher &a, int64_t row, int j) {
        const int64_t at = row * a.count + j;
        Item<TYPE> t;
        t.x = a.ids[at];
        if (a.type == TN_TYPE_F32) t.l = static_cast<const float *>(a.logits)[at];
        else if (a.type == TN_TYPE_BF16) t.l = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[at]);
        else t.l = __half2float(static_cast<const __half *>(a.logits)[at]);
        return t;
    }
    template <int TYPE>
    static __device__ __forceinline__ void look(Item<TYPE> &t, const Row<TYPE> &r, bool values) {
        const bool in = t.x >= 0 && t.x < r.cols;
        t.v = typename Entry<TYPE>::T();
        if (in && values) t.v = r.p[t.x * r.cs];
        t.keep = 1;
        if (in && r.m) t.keep = r.m[t.x * r.mcs];
    }
    template <int TYPE>
    __device__ __forceinline__ void settle(int j, const Item<TYPE> &t, const OutRows &rows, const Row<TYPE> &r,
                                           int64_t row) const {
        const bool in = t.x >= 0 && t.x < r.cols, wrong = !in && t.x != -1;
        const bool used_ = in && t.keep && t.l != -__builtin_huge_valf();
        if (wrong) flag_bad_id(rows, row);
        id[j] = used_ ? t.x : wrong ? -2 : -1;       // -2: an id out of range
        logq[j] = used_ ? t.l : -__builtin_huge_valf();   // (not scaled yet)
        value[j] = Entry<TYPE>::value(t.v);
    }
    template <int TYPE, int G>
    __device__ __forceinline__ void read(const Group<G> &g, const OutTeacher &a, const OutRows &rows,
                                         const Row<TYPE> &r, int64_t row, bool values) {
        constexpr int kPer = G < TN_OUTCOMES_MAX_IDS ? TN_OUTCOMES_MAX_IDS / G : 1;
#pragma unroll (kPer < 4 ? kPer : 4)
        for (int i = 0; i < kPer; ++i) {
            const int j = g.t + i * G;
            if (j >= a.count) break;
            Item<TYPE> t = item<TYPE>(a, row, j);
            look<TYPE>(t, r, values);
            settle<TYPE>(j, t, rows, r, row);
        }
    }
    // One warp.  Differences are scaled, which cannot overflow to where all
    // outcomes are left out (or none is finite).
    __device__ __forceinline__ void normalise(const OutTeacher &a) const {
        const int count = a.count;
        const int lane = threadIdx.x % 32;
        float top = -__builtin_huge_valf(), total = 0.f;
#pragma unroll 1
        for (int j = lane; j < count; j += 32) top = max_nan(top, logq[j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
        for (int j = lane; j < count; j += 32) {
            const float l = (logq[j] - top) * a.scale, e = id[j] >= 0 ? expf(l) : 0.f;
            logq[j] = l;
            q[j] = e;
            total += e;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const float logt = logf(total);
#pragma unroll 1
        for (int j = lane; j < count; j += 32) {
            logq[j] -= logt;
            q[j] = id[j] >= 0 ? q[j] / total : 0.f;
        }
        if (lane == 0) *used = top == -__builtin_huge_valf() ? 0.f : 1.f;
        __syncwarp();
    }
};

}  // namespace tn
