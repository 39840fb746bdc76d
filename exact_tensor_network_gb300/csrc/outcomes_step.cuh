// Loss and gradient of a row in one pass over memory: the row waits in shared
// memory between the sums and the gradient, so that it is read once and its
// gradient written once.  Included by the translation unit of each entry type.
//
// A cluster of up to eight CTAs holds a row (kStepSlice bytes a CTA, so that
// three CTAs are on an SM and one's loads run beside another's stores; more
// for longer rows, more CTAs for few rows).  Every thread copies its own
// vectors to shared memory ahead of the sums (cp.async, no barrier), the CTAs
// exchange their sums through distributed shared memory, and every thread
// reads its own vectors back for the gradient.  Rows of one warp are held by
// one warp each.
#pragma once

#include "outcomes_forward.cuh"
#include "outcomes_grad.cuh"

namespace tn {

namespace {

constexpr int kStepAhead = 4;      // steps of kU vectors in flight per thread

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 cluster_load(const float4 *p, int rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), far;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(far)
                 : "memory");
    return v;
}

// The dense part of a vector where the row's sums are at hand.
template <int TYPE>
struct Dense {
    float2 z0, c2, ls, ma;
    __device__ __forceinline__ Dense(const RowGrad &c, float z, float s, float c2_)
        : z0(make_float2(-z, -z)), c2(make_float2(c2_, c2_)) {
        const float l = -log2f(s), m = c.mult * c.alpha;
        ls = make_float2(l, l);
        ma = make_float2(m, m);
    }
    __device__ __forceinline__ uint4 grad(const RowGrad &c, const uint4 &raw) const {
        if constexpr (Entry<TYPE>::kReal) {
            constexpr int E = Entry<TYPE>::E;
            float v[E];
            Entry<TYPE>::values(raw, v);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 d = fma2(add2(make_float2(v[i], v[i + 1]), z0), c2, ls);
                const float2 o = mul2(make_float2(ex2(d.x), ex2(d.y)), ma);
                v[i] = o.x;
                v[i + 1] = o.y;
            }
            return pack<TYPE>(v, raw);
        } else {
            return dense_grad<TYPE, false>(c, raw);
        }
    }
};

template <int TYPE, int G, bool MASK, bool UNIT>
__global__ void __launch_bounds__(G == 32 ? kOutThreads : G, G == 32 ? 6 : 3)
outcomes_step(const __grid_constant__ OutStep a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr int kGroups = G == 32 ? kOutThreads / 32 : 1;
    constexpr float kInf = __builtin_huge_valf();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t red[4 * G / 32];
    __shared__ float4 part;
    __shared__ Teacher teachers[kGroups];
    pdl_trigger();
    Group<G> g(red);
    const int group = threadIdx.x / G;
    const uint32_t item = blockIdx.x * kGroups + group, ranks = G == 32 ? 1 : (uint32_t)a.r.segs;
    const int64_t row = G == 32 ? item : item / ranks;
    const int rank = G == 32 ? 0 : item % ranks;
    const int n = a.teacher.count;
    Teacher &te = teachers[group];
    uint4 *hold = reinterpret_cast<uint4 *>(smem) + group * a.r.seg_vecs + g.t;
    pdl_wait();
    if (G == 32 && row >= a.r.rows) return;

    const Row<TYPE> r(a.r, row);
    const int64_t v0 = rank * a.r.seg_vecs;
    const int64_t all = (r.head + r.cols + E - 1) / E;
    const int64_t v1 = min(all, v0 + a.r.seg_vecs);
    const int nv = static_cast<int>(max((int64_t)0, v1 - v0));
    const bool words = !MASK || r.mask_words();
    int64_t in0, in1;
    r.inside_range(in0, in1);
    // vectors [lo, hi) go through shared memory; the row's first and last
    // (all of a strided row's, or of one whose mask bytes are not words) do not
    const int lo = (int)max((int64_t)0, min((int64_t)nv, in0 - v0));
    const int hi = words ? max(lo, (int)max((int64_t)0, min((int64_t)nv, in1 - v0))) : lo;
    const uint4 *vecs = r.vectors() + v0 + g.t;
    const int64_t first = v0 * E - r.head;

    const auto whole = [&](int b) { return b >= lo && b + kU * G <= hi; };
    const auto copy_step = [&](int b) {
        if (whole(b)) {
#pragma unroll
            for (int u = 0; u < kU; ++u) copy16(hold + b + u * G, vecs + b + u * G);
        } else if (b < nv) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = b + u * G + g.t;
                if (j >= lo && j < hi) copy16(hold + b + u * G, vecs + b + u * G);
            }
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStepAhead; ++i) copy_step(i * kU * G);
    typename Row<TYPE>::Keep next_keep[kU];
    const auto load_keep = [&](int b) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + g.t;
            if (j >= lo && j < hi) next_keep[u] = r.keep_word(first + (int64_t)j * E);
        }
    };
    if (MASK) load_keep(0);

    te.read(g, a.teacher, a.r, r, row, rank == 0);

    Stream<TYPE, false, UNIT> st;
#pragma unroll 1
    for (int b = 0; b < nv; b += kU * G) {
        uint32_t later = 0;
        typename Row<TYPE>::Keep keep[kU];
        if (MASK) {
#pragma unroll
            for (int u = 0; u < kU; ++u) keep[u] = next_keep[u];
            load_keep(b + kU * G);
        }
        copy_wait<kStepAhead - 1>();
        const bool full = whole(b);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + g.t;
            const bool in = full || (j >= lo && j < hi);
            uint4 raw = En::absent_vector();
            if (in) {
                raw = hold[b + u * G];
                if (MASK) {
                    En::blank(raw, keep[u]);
                    hold[b + u * G] = raw;
                }
            } else if (j < nv) {
                later |= 1u << u;
            }
            float v[E];
            const float lm = decode<TYPE>(raw, v, a.r.floor);
            if (!st.add(v, lm, a.r.c2)) later |= 1u << u;
        }
#pragma unroll 1
        for (; later; later &= later - 1) {
            const auto x = row_vector<TYPE>(r, v0 + b + (__ffs(later) - 1) * G + g.t);
            float v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = x.v[i];
            const float m = largest<TYPE>(v, a.r.floor);
            if (!st.add(v, m, a.r.c2)) st.far(x.v, m, a.r.c2);
        }
        copy_step(b + kStepAhead * kU * G);
    }
    Sums<TYPE> sum = st.done(a.r.c2);
    combine(g, sum, a.r.c2);
    if (G == 32) g.sync();
    if (G > 32 && ranks > 1) {
        if (g.t == 0) part = make_float4(sum.z0, sum.s, 0.f, 0.f);
        cluster_arrive();
        if (g.warp == 0) te.normalise(n);
        cluster_wait();
        // the cluster's sums, one a lane
        sum = Sums<TYPE>();
        if (g.lane < (int)ranks) {
            const float4 f = cluster_load(&part, g.lane);
            sum.z0 = f.x;
            sum.s = f.y;
        }
        float m = sum.z0;
#pragma unroll
        for (int o = 4; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (sum.z0 != m) sum.move_to(m, a.r.c2);
#pragma unroll
        for (int o = 4; o; o >>= 1) sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
        sum.z0 = __shfl_sync(0xffffffffu, m, 0);      // lanes from 8 on saw nothing
        sum.s = __shfl_sync(0xffffffffu, sum.s, 0);
        cluster_arrive();      // (waited for at the end: the others may still read)
    } else if (g.warp == 0) {
        te.normalise(n);
    }
    g.sync();
    float logz, entropy;
    normaliser<TYPE>(a.r, sum, logz, entropy);

    RowGrad c;
    c.scale = a.r.scale;
    c.logz = logz;
    c.beta = c.entropy = 0.f;
    c.alpha = te.used;
    c.mult = a.g_loss[row] * a.r.scale;
    finish_row_grad<TYPE>(c);
    const Out<TYPE> out(a.grad, a.grad_row_stride, a.grad_col_stride, r, row);
    // p = 2^(c2 (z - z0) - log2 s): 1 exactly for a row's only entry
    Dense<TYPE> dense(c, sum.z0, sum.s, a.r.c2);
#pragma unroll 1
    for (int b = 0; b < nv; b += kU * G) {
        if (c.plain && out.wide && whole(b)) {
            uint4 *to = reinterpret_cast<uint4 *>(out.p + first) + b + g.t;
#pragma unroll
            for (int u = 0; u < kU; ++u) to[u * G] = dense.grad(c, hold[b + u * G]);
            continue;
        }
        uint32_t odd = 0;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + g.t;
            if (c.plain && j >= lo && j < hi) out.put(first + (int64_t)j * E, dense.grad(c, hold[b + u * G]));
            else if (j < nv) odd |= 1u << u;
        }
#pragma unroll 1
        for (; odd; odd &= odd - 1) grad_vector<TYPE>(r, c, out, v0 + b + (__ffs(odd) - 1) * G + g.t);
    }
    g.sync();
    const typename En::T *held = reinterpret_cast<const typename En::T *>(hold - g.t);
    grad_ids<TYPE>(g, r, c, out, te.id, te.q, -1.f, n, first, v1 * E - r.head, held, first + (int64_t)lo * E,
                   first + (int64_t)hi * E);
    if (rank == 0 && g.warp == 0) {
        const float loss = teacher_loss<TYPE>(n, a.r, te, logz);
        if (g.t == 0) {
            a.loss[row] = loss;
            a.logz[row] = logz;
        }
    }
    if (G > 32 && ranks > 1) cluster_wait();
}

template <int TYPE, int G, bool MASK, bool UNIT>
cudaError_t launch_step(const OutStep &a, cudaStream_t stream) {
    auto *kernel = outcomes_step<TYPE, G, MASK, UNIT>;
    const int threads = G == 32 ? kOutThreads : G, groups = threads / G;
    const size_t smem = (size_t)groups * a.r.seg_vecs * kOutVecBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.r.rows * a.r.segs + groups - 1) / groups));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.r.segs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.r.segs > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int TYPE, int G>
cudaError_t step_mask(const OutStep &a, cudaStream_t stream) {
    if constexpr (TYPE == TN_TYPE_C64) {
        if (a.r.scale == 1.f)
            return a.r.mask ? launch_step<TYPE, G, true, true>(a, stream) : launch_step<TYPE, G, false, true>(a, stream);
    }
    return a.r.mask ? launch_step<TYPE, G, true, false>(a, stream) : launch_step<TYPE, G, false, false>(a, stream);
}

}  // namespace

template <int TYPE>
cudaError_t outcomes_step_of(const OutStep &a, bool warp_rows, cudaStream_t stream) {
    return warp_rows ? step_mask<TYPE, 32>(a, stream) : step_mask<TYPE, kStepThreads>(a, stream);
}

}  // namespace tn
