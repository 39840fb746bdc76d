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
#pragma once

#include "outcomes.cuh"

namespace tn {

namespace {

constexpr int kGradU = 4;           // vectors in flight per thread

struct RowGrad {
    float mult, alpha, beta, logz, entropy;
    float inv_z;      // amplitudes at scale 1: p = w inv_z (0: not used)
    float scale;
};

// What multiplies the entry (an amplitude) or is the gradient itself (a real
// logit).  v: order value of a present entry.
template <int TYPE>
__device__ __forceinline__ float entry_grad(const RowGrad &c, float v, float add) {
    if constexpr (Entry<TYPE>::kReal) {
        const float lp = __fadd_rn(__fmul_rn(v, c.scale), -c.logz);
        const float p = ex2(lp * kLog2E);
        return c.mult * fmaf(p, fmaf(c.beta, lp + c.entropy, c.alpha), add);
    } else {
        // 2 / w dL/dz, with p / w taken together
        float lp = 0.f, pw = c.inv_z;
        if (c.beta != 0.f || c.inv_z == 0.f) {
            lp = __fadd_rn(__fmul_rn(c.scale, logf(v)), -c.logz);
            if (c.inv_z == 0.f) pw = ex2(lp * kLog2E) / v;
        }
        const float dense = pw * fmaf(c.beta, lp + c.entropy, c.alpha);
        return 2.f * c.mult * (add == 0.f ? dense : dense + add / v);
    }
}

template <int TYPE>
__device__ __forceinline__ typename Entry<TYPE>::T to_entry(float g, typename Entry<TYPE>::T x) {
    if constexpr (TYPE == TN_TYPE_F32) return g;
    else if constexpr (TYPE == TN_TYPE_BF16) return __float2bfloat16_rn(g);
    else if constexpr (TYPE == TN_TYPE_F16) return __float2half_rn(g);
    else return make_float2(g * x.x, g * x.y);
}

// g[i] of the vector's entries as 16 bytes of the rows' type
template <int TYPE>
__device__ __forceinline__ uint4 pack(const float (&g)[Entry<TYPE>::E], const uint4 &raw) {
    uint4 o;
    if constexpr (TYPE == TN_TYPE_F32) {
        o = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                       __float_as_uint(g[3]));
    } else if constexpr (TYPE == TN_TYPE_C64) {
        o = make_uint4(__float_as_uint(g[0] * __uint_as_float(raw.x)),
                       __float_as_uint(g[0] * __uint_as_float(raw.y)),
                       __float_as_uint(g[1] * __uint_as_float(raw.z)),
                       __float_as_uint(g[1] * __uint_as_float(raw.w)));
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

template <int TYPE, int G, bool MASK>
__global__ void __launch_bounds__(kOutThreads) outcomes_grad(const __grid_constant__ OutGrad a) {
    using En = Entry<TYPE>;
    using T = typename En::T;
    constexpr int E = En::E;
    constexpr int kGroups = kOutThreads / G;
    constexpr float kInf = __builtin_huge_valf();
    extern __shared__ int64_t lists[];
    __shared__ uint32_t red[4 * kOutThreads / 32];
    pdl_trigger();
    Group<G> g(red);
    const int64_t item = (int64_t)blockIdx.x * kGroups + threadIdx.x / G;
    const int64_t row = G == 32 ? item : item / a.r.segs;
    const int64_t seg = G == 32 ? 0 : item - row * a.r.segs;
    const int n = a.teacher.count ? a.teacher.count : a.n_given;
    int64_t *ids = lists + (size_t)(threadIdx.x / G) * n;
    float *adds = reinterpret_cast<float *>(lists + (size_t)kGroups * n) + (size_t)(threadIdx.x / G) * n;
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;

    const Row<TYPE> r(a.r, row);
    const int64_t v0 = seg * a.r.seg_vecs;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    const int64_t v1 = min(all, v0 + a.r.seg_vecs);
    const int nv = static_cast<int>(max((int64_t)0, v1 - v0));

    RowGrad c;
    c.scale = a.r.scale;
    c.logz = a.logz[row];
    c.beta = 0.f;
    c.entropy = 0.f;
    if (a.teacher.count) {
        Teacher<G> te;
        te.load(g, a.teacher, a.r, r, row);
#pragma unroll
        for (int i = 0; i < Teacher<G>::kPer; ++i) {
            const int j = g.t + i * G;
            if (j < n) {
                ids[j] = te.id[i];
                adds[j] = -te.q[i];
            }
        }
        c.alpha = te.used;
        c.mult = a.g_loss[row] * a.r.scale;
    } else {
        float total = 0.f;
        for (int j = g.t; j < n; j += G) {
            int64_t id = a.given[row * n + j];
            if (id < -1 || id >= r.cols) {
                flag_bad_id(a.r, row);
                id = -1;
            }
            if (id >= 0 && r.value(id) == absent<TYPE>()) id = -1;
            const float x = id >= 0 ? a.g_logp[row * n + j] : 0.f;
            ids[j] = id;
            adds[j] = x;
            total += x;
        }
        c.alpha = -g.sum(total);
        if (a.g_entropy) {
            c.beta = -a.g_entropy[row];
            c.entropy = a.entropy[row];
        }
        c.mult = a.r.scale;
    }
    c.inv_z = !En::kReal && a.r.scale == 1.f && c.logz > -80.f && c.logz < 80.f ? expf(-c.logz) : 0.f;

    T *out = reinterpret_cast<T *>(a.grad) + row * a.grad_row_stride;
    const int64_t os = a.grad_col_stride;
    // vectors of the gradient are aligned where the row's are, or never
    const bool wide = os == 1 && r.cs == 1 &&
                      (reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(r.p)) % kOutVecBytes == 0;

    for (int b = 0; b < nv; b += kGradU * G) {
        uint4 raw[kGradU];
        bool in[kGradU];
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
            const int j = b + u * G + g.t;
            const int64_t e0 = (v0 + j) * E - r.head;
            in[u] = wide && j < nv && r.inside(e0);
            if (in[u]) raw[u] = r.raw(e0);
        }
        if constexpr (MASK) {
#pragma unroll
            for (int u = 0; u < kGradU; ++u)
                if (in[u]) En::blank(raw[u], r.keep((v0 + b + u * G + g.t) * E - r.head));
        }
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
            const int j = b + u * G + g.t;
            const int64_t e0 = (v0 + j) * E - r.head;
            if (in[u]) {
                float v[E];
                En::values(raw[u], v);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float x = entry_grad<TYPE>(c, v[i], 0.f);
                    v[i] = v[i] == absent<TYPE>() ? 0.f : x;
                }
                *reinterpret_cast<uint4 *>(out + e0) = pack<TYPE>(v, raw[u]);
            } else if (j < nv) {
#pragma unroll 1
                for (int i = 0; i < E; ++i) {
                    const int64_t e = e0 + i;
                    if (e < 0 || e >= r.cols) continue;
                    const float v = r.value(e);
                    T o = to_entry<TYPE>(0.f, T());
                    if (v != absent<TYPE>()) o = to_entry<TYPE>(entry_grad<TYPE>(c, v, 0.f), r.p[e * r.cs]);
                    out[e * os] = o;
                }
            }
        }
    }
    if (n == 0) return;
    g.sync();
    const int64_t e_lo = v0 * E - r.head, e_hi = v1 * E - r.head;
    for (int j = g.t; j < n; j += G) {
        const int64_t id = ids[j];
        if (id < 0 || id < e_lo || id >= e_hi) continue;
        float add = 0.f;
        bool first = true;
        for (int i = 0; i < n; ++i)
            if (ids[i] == id) {
                first = first && i >= j;
                add += adds[i];
            }
        if (!first) continue;
        const float v = r.value(id);
        if (v != absent<TYPE>())
            out[id * os] = to_entry<TYPE>(entry_grad<TYPE>(c, v, add), r.p[id * r.cs]);
    }
}

template <int TYPE, int G, bool MASK>
cudaError_t launch_grad(const OutGrad &a, cudaStream_t stream) {
    const int64_t items = a.r.rows * a.r.segs;
    const int groups = kOutThreads / G;
    const int n = a.teacher.count ? a.teacher.count : a.n_given;
    const size_t smem = (size_t)groups * n * (sizeof(int64_t) + sizeof(float));
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
