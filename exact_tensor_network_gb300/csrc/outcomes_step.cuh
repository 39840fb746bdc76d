// Loss and gradient of a row in one pass over memory: the row waits in shared
// memory between the sums and the gradient, so that it is read once and its
// gradient written once.  Included by the translation unit of each entry type.
//
// A cluster of up to eight CTAs holds a row and goes from row to row.  Every
// thread copies its own vectors to shared memory (cp.async, no barrier for the
// data), sums them, and after the CTAs have exchanged their sums through
// distributed shared memory reads them back for the gradient; once it has used
// its vectors it copies the next row's in their place.  So the loads of the
// next row run beside the stores of this one, and three CTAs an SM cover each
// other's barriers (four with smaller slices: 1024x131072 bf16 143 against 114
// us).  Short rows are held by one warp each.
//
// What bounds it.  A row passes through a chain (its loads, sums, the cluster's
// barrier, the join, the gradient) of some 5 us, which the CTAs of an SM run
// side by side, and every warp pays some 800 instructions a row besides its
// vectors: 1024x131072 bf16 104 to 109 us (5.0 TB/s read and written, memory and
// issue slots at 65 and 62 %), 1000x50000 f32 91 to 97 us (4.2 TB/s), 8192x16384
// bf16 101 us (5.3 TB/s), 2000x16384 amplitudes 121 us (4.3 TB/s); 10000x8000 bf16
// by warps 75 us (4.2 TB/s).  500x32003 f32 (37 us, 3.5 TB/s) takes three rounds of
// 220 clusters for 2.3 rounds' rows.
#pragma once

#include "outcomes_forward.cuh"
#include "outcomes_grad.cuh"

namespace tn {

namespace {

// At most n of this thread's last copy groups still in flight.
__device__ __forceinline__ void copy_wait_all_but(int n) {
    switch (n) {
        case 0: copy_wait<0>(); break;
        case 1: copy_wait<1>(); break;
        case 2: copy_wait<2>(); break;
        case 3: copy_wait<3>(); break;
        case 4: copy_wait<4>(); break;
        case 5: copy_wait<5>(); break;
        case 6: copy_wait<6>(); break;
        default: copy_wait<7>(); break;
    }
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// v to where p is in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ void cluster_store(const float2 *p, int rank, float2 v) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), far;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(far), "f"(v.x), "f"(v.y) : "memory");
}

// The dense part of a vector where the row's sums are at hand.  bf16 reaches
// below the least p that ex2 gives (see dense_grad): it gets 2^64 p, and the
// factor 2^-64.  That rounds the exponent to 2^-19, 2^-11 of a bf16's step; the
// square that dense_grad takes cost the kernel of 256 threads, which has no
// register to spare, 17 % (1024x131072 132 against 115 us).
template <int TYPE>
struct Dense {
    float2 z0, c2, ls, ma;
    __device__ __forceinline__ Dense(const RowGrad &c, float z, float s, float c2_)
        : z0(make_float2(-z, -z)), c2(make_float2(c2_, c2_)) {
        float l = -kLog2E * logf(s), m = c.mult * c.alpha;     // (as log Z has it)
        if constexpr (TYPE == TN_TYPE_BF16) {
            l += 64.f;
            m *= 0x1p-64f;
        }
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
            return pack<TYPE>(v);
        } else {
            return dense_grad<TYPE, false>(c, raw);
        }
    }
};

// A CTA's part of a row.  Vectors [lo, hi) of its nv go through shared memory;
// the row's first and last (all of a strided row's, or of one whose mask bytes
// are not words) do not.
template <int TYPE, bool MASK, int G>
struct Slice {
    Row<TYPE> r;
    int nv, lo, hi, steps;
    int64_t v0, first;       // first vector, first entry
    const uint4 *vecs;

    __device__ __forceinline__ Slice(const OutRows &a, int64_t row, int rank) : r(a, row) {
        constexpr int E = Entry<TYPE>::E;
        // (a row that fits a cluster has fewer than 2^31 entries)
        const int slice = (int)a.seg_vecs, at = rank * slice, end = r.head + (int)r.cols;
        v0 = at;
        first = (int64_t)at * E - r.head;
        nv = max(0, min((end + E - 1) / E - at, slice));
        lo = r.cs == 1 && rank == 0 && r.head > 0 ? min(1, nv) : 0;
        hi = r.cs == 1 && (!MASK || r.mask_words()) ? max(lo, min(nv, end / E - at)) : lo;
        steps = (nv + kU * G - 1) / (kU * G);
        vecs = r.vectors() + v0;
    }
    __device__ __forceinline__ bool whole(int b, int n) const { return b >= lo && b + n <= hi; }
};

// One step (kU vectors a thread, from vector b on) of a row into hold.
template <int TYPE, bool MASK, int G>
__device__ __forceinline__ void copy_step(const Slice<TYPE, MASK, G> &s, uint4 *hold, int b, int t) {
    if (s.whole(b, kU * G)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) copy16(hold + b + u * G + t, s.vecs + b + u * G + t);
    } else if (b < s.nv) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + t;
            if (j >= s.lo && j < s.hi) copy16(hold + j, s.vecs + j);
        }
    }
    copy_commit();
}

// The sums of a slice, whose copies are the last groups (one a step).
template <int TYPE, int G, bool MASK, bool UNIT>
__device__ __forceinline__ Sums<TYPE> sum_slice(const Slice<TYPE, MASK, G> &s, uint4 *hold, int t,
                                                const OutRows &a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    typename Row<TYPE>::Keep next_keep[kU];
    const auto load_keep = [&](int b) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = b + u * G + t;
            if (j >= s.lo && j < s.hi) next_keep[u] = s.r.keep_word(s.first + (int64_t)j * E);
        }
    };
    if (MASK) load_keep(0);
    Stream<TYPE, false, UNIT> st;
#pragma unroll 1
    for (int i = 0; i < s.steps; ++i) {
        const int b = i * kU * G;
        uint32_t later = 0;
        typename Row<TYPE>::Keep keep[kU];
        if (MASK) {
#pragma unroll
            for (int u = 0; u < kU; ++u) keep[u] = next_keep[u];
            load_keep(b + kU * G);
        }
        copy_wait_all_but(s.steps - 1 - i);
        uint4 raw[kU];
        if (s.whole(b, kU * G)) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                raw[u] = hold[b + u * G + t];
                if (MASK) {
                    En::blank(raw[u], keep[u]);
                    hold[b + u * G + t] = raw[u];
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = b + u * G + t;
                raw[u] = En::absent_vector();
                if (j >= s.lo && j < s.hi) {
                    raw[u] = hold[j];
                    if (MASK) {
                        En::blank(raw[u], keep[u]);
                        hold[j] = raw[u];
                    }
                } else if (j < s.nv) {
                    later |= 1u << u;
                }
            }
        }
        if (!st.add_step(raw, a)) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (b + u * G + t < s.nv) later |= 1u << u;
        }
#pragma unroll 1
        for (; later; later &= later - 1) {
            const auto x = row_vector<TYPE>(s.r, s.v0 + b + (__ffs(later) - 1) * G + t);
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = x.v[e];
            const float m = largest<TYPE>(v, a.floor);
            if (!st.add(v, m, a)) st.far(x.v, m, a.c2);
        }
    }
    return st.done(a.c2);
}

// The dense gradient of one step of a slice.
template <int TYPE, int G, bool MASK>
__device__ __forceinline__ void grad_step(const Slice<TYPE, MASK, G> &s, const uint4 *hold, int b, int t,
                                          const RowGrad &c, const Dense<TYPE> &dense, const Out<TYPE> &out) {
    constexpr int E = Entry<TYPE>::E;
    if (c.plain && out.wide && s.whole(b, kU * G)) {
        uint4 *to = reinterpret_cast<uint4 *>(out.p + s.first) + b + t;
#pragma unroll
        for (int u = 0; u < kU; ++u) to[u * G] = dense.grad(c, hold[b + u * G + t]);
        return;
    }
    uint32_t odd = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int j = b + u * G + t;
        if (c.plain && j >= s.lo && j < s.hi) out.put(s.first + (int64_t)j * E, dense.grad(c, hold[j]));
        else if (j < s.nv) odd |= 1u << u;
    }
#pragma unroll 1
    for (; odd; odd &= odd - 1) grad_vector<TYPE>(s.r, c, out, s.v0 + b + (__ffs(odd) - 1) * G + t);
}

// Relative to the reference, as Dense is: log Z may have lost ln s (a row that
// one large value fills).
template <int TYPE>
__device__ __forceinline__ RowGrad step_grad(const OutStep &a, float g_loss, const Norm &norm, float used) {
    RowGrad c;
    c.scale = a.r.scale;
    c.logz = norm.ls;
    c.beta = c.entropy = 0.f;
    c.alpha = used;
    c.mult = g_loss * a.r.scale;
    finish_row_grad<TYPE>(c, norm.z0, norm.logz(a.r));
    return c;
}

// Rows of one warp.
template <int TYPE, bool MASK, bool UNIT>
__global__ void __launch_bounds__(kOutThreads, 6) outcomes_step_warps(const __grid_constant__ OutStep a) {
    using En = Entry<TYPE>;
    constexpr int E = En::E;
    constexpr int kGroups = kOutThreads / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_trigger();
    Group<32> g(nullptr);
    const int group = threadIdx.x / 32;
    const int64_t row = (int64_t)blockIdx.x * kGroups + group;
    const int n = a.teacher.count;
    uint4 *hold = reinterpret_cast<uint4 *>(smem) + group * a.r.seg_vecs;
    unsigned char *lists = smem + kGroups * a.r.seg_vecs * kOutVecBytes +
                           group * (teacher_bytes(n) + repeat_bytes(n) + repeat_sums(n));
    Teacher te(lists, n);
    pdl_wait();
    if (row >= a.r.rows) return;
    const Slice<TYPE, MASK, 32> s(a.r, row, 0);
#pragma unroll 1
    for (int i = 0; i < s.steps; ++i) copy_step<TYPE, MASK, 32>(s, hold, i * kU * 32, g.t);
    te.read(g, a.teacher, a.r, s.r, row, true);
    Sums<TYPE> sum = sum_slice<TYPE, 32, MASK, UNIT>(s, hold, g.t, a.r);
    combine(g, sum, a.r.c2);
    g.sync();
    te.normalise(a.teacher);
    const Norm norm = normaliser<TYPE>(sum);
    const RowGrad c = step_grad<TYPE>(a, a.g_loss[row], norm, *te.used);
    const Dense<TYPE> dense(c, sum.z0, sum.s, a.r.c2);
    const Out<TYPE> out(a.grad, a.grad_row_stride, a.grad_col_stride, s.r, row);
#pragma unroll 1
    for (int i = 0; i < s.steps; ++i) grad_step<TYPE, 32, MASK>(s, hold, i * kU * 32, g.t, c, dense, out);
    g.sync();
    grad_ids<TYPE>(g, s.r, c, out, te.id, te.q, -1.f, n, s.first, s.first + (int64_t)s.nv * E,
                   lists + teacher_bytes(n), reinterpret_cast<const typename En::T *>(hold), s.first + (int64_t)s.lo * E,
                   s.first + (int64_t)s.hi * E);
    const float loss = teacher_loss<TYPE>(n, a.r, te, norm);
    if (g.t == 0) {
        a.loss[row] = loss;
        a.logz[row] = norm.logz(a.r);
    }
}

// Longer rows: the a.r.segs CTAs of a cluster a row.  Two barriers a row:
// the cluster's, at which every warp's sums have reached every CTA, and one
// between reading the entries at the teacher's outcomes and the copies that
// take their place.  What follows from a row but has no hurry (the entries at
// the teacher's outcomes, which others' dense stores must precede) waits for
// the next row's barrier; the next row's teacher is fetched one row ahead.
// G threads, one for each of the teacher's outcomes at least.
template <int TYPE, int G, bool MASK, bool UNIT>
__global__ void __launch_bounds__(G, 3) outcomes_step(const __grid_constant__ OutStep a) {
    using En = Entry<TYPE>;
    using T = typename En::T;
    constexpr int E = En::E, kWarps = G / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 part[2][kWarps * kStepCluster];
    pdl_trigger();
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    const uint32_t ranks = (uint32_t)a.r.segs, clusters = gridDim.x / ranks;
    const int rank = blockIdx.x % ranks, n = a.teacher.count;
    int64_t row = blockIdx.x / ranks;
    uint4 *hold = reinterpret_cast<uint4 *>(smem);
    unsigned char *te_base = smem + a.r.seg_vecs * kOutVecBytes;
    const auto repeats = [&](int i) {     // of the even and of the odd rows
        unsigned char *p = te_base + 2 * teacher_bytes(n);
        return Repeats(p + 2 * repeat_marks(n), p + i * repeat_marks(n), n);
    };
    const auto copy_row = [&](const Slice<TYPE, MASK, G> &x) {
#pragma unroll 1
        for (int i = 0; i < x.steps; ++i) copy_step<TYPE, MASK, G>(x, hold, i * kU * G, t);
    };
    // the cluster's CTAs have all started before any writes to another's memory
    if (ranks > 1) cluster_arrive();
    pdl_wait();

    Slice<TYPE, MASK, G> s(a.r, row, rank);
    copy_row(s);
    {
        Teacher te(te_base, n);
        if (t < n) {
            Teacher::Item<TYPE> it = Teacher::item<TYPE>(a.teacher, row, t);
            Teacher::look<TYPE>(it, s.r, rank == 0);
            te.settle<TYPE>(t, it, a.r, s.r, row);
            if (te.id[t] >= 0) repeats(0).put(t, te.id[t]);
        }
        __syncthreads();
        if (t < n && te.id[t] >= 0) repeats(0).look(te.id, t, te.id[t]);
        if (warp == kWarps - 2) te.normalise(a.teacher);
    }
    if (ranks > 1) cluster_wait();
    int turn = 0;
    T fix = T();                 // the entry of this thread's outcome in the
    T *fix_at = nullptr;         // last row, if it is this CTA's
#pragma unroll 1
    while (true) {
        const int64_t next_row = row + clusters;
        const bool more = next_row < a.r.rows;
        const Slice<TYPE, MASK, G> next(a.r, more ? next_row : row, rank);
        Teacher::Item<TYPE> it;
        if (more && t < n) it = Teacher::item<TYPE>(a.teacher, next_row, t);
        const float g_loss = a.g_loss[row];

        Sums<TYPE> sum = sum_slice<TYPE, G, MASK, UNIT>(s, hold, t, a.r);
        float m = warp_max_nan(sum.z0);
        if (sum.z0 != m) sum.move_to(m, a.r.c2);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
        if (more && t < n) Teacher::look<TYPE>(it, next.r, rank == 0);
        // part alternates: a slot is written again only after the barrier
        // that follows its reading
        float2 *mine = part[turn] + rank * kWarps + warp;
        if (ranks == 1) {
            if (lane == 0) *mine = make_float2(sum.z0, sum.s);
            __syncthreads();
        } else {
            if (lane < (int)ranks) cluster_store(mine, lane, make_float2(sum.z0, sum.s));
            cluster_arrive();
            cluster_wait();
        }
        if (fix_at) *fix_at = fix;
        fix_at = nullptr;
        const int np = (int)ranks * kWarps;
        sum = Sums<TYPE>();
#pragma unroll 1
        for (int i = lane; i < np; i += 32) {
            const float2 f = part[turn][i];
            Sums<TYPE> o;
            o.z0 = f.x;
            o.s = f.y;
            m = max_nan(sum.z0, o.z0);
            if (sum.z0 != m) sum.move_to(m, a.r.c2);
            if (o.z0 != m) o.move_to(m, a.r.c2);
            sum.s += o.s;
        }
        m = warp_max_nan(sum.z0);
        if (sum.z0 != m) sum.move_to(m, a.r.c2);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
        const Norm norm = normaliser<TYPE>(sum);

        Teacher te(te_base + turn * teacher_bytes(n), n);
        const RowGrad c = step_grad<TYPE>(a, g_loss, norm, *te.used);
        const Dense<TYPE> dense(c, sum.z0, sum.s, a.r.c2);
        const Out<TYPE> out(a.grad, a.grad_row_stride, a.grad_col_stride, s.r, row);
        const int64_t id = t < n ? te.id[t] : -1;
        const bool here = id >= 0 && id >= s.first && id < s.first + (int64_t)s.nv * E;
        T x = T();
        float v = absent<TYPE>();
        if (here) {
            const int j = (int)((id - s.first) / E);
            if (j >= s.lo && j < s.hi) {
                x = reinterpret_cast<const T *>(hold)[id - s.first];
                v = En::value(x);
            } else {
                x = s.r.p[id * s.r.cs];
                v = row_value<TYPE>(s.r, id);
            }
        }
        const Teacher then(te_base + (turn ^ 1) * teacher_bytes(n), n);
        const bool given = more && t < n && it.x >= 0;
        if (more && t < n) then.settle<TYPE>(t, it, a.r, next.r, next_row);
        if (given) repeats(turn ^ 1).put(t, it.x);
        __syncthreads();
        if (given) repeats(turn ^ 1).look(then.id, t, it.x);
#pragma unroll 1
        for (int i = 0; i < s.steps; ++i) {
            grad_step<TYPE, G, MASK>(s, hold, i * kU * G, t, c, dense, out);
        }
        if (more) copy_row(next);
        if (warp * 32 < n) {       // (a warp's votes: every lane takes part)
            float add = here ? te.q[t] : 0.f;
            const bool lead = sum_of_equal(te.id, te.q, n, t, id, here && repeats(turn).mark[t], add);
            if (lead && v != absent<TYPE>()) {
                fix = entry_grad<TYPE>(c, v, x, -add);
                fix_at = out.p + id * out.cs;
            }
        }
        // (small jobs, each on its own warp: the slowest warp of a cluster is
        // what its barrier waits for)
        if (warp == kWarps - 1 && rank == 0) {
            const float loss = teacher_loss<TYPE>(n, a.r, te, norm);
            if (lane == 0) {
                a.loss[row] = loss;
                a.logz[row] = norm.logz(a.r);
            }
        }
        if (warp == kWarps - 2 && more) then.normalise(a.teacher);
        if (!more) break;
        row = next_row;
        s = next;
        turn ^= 1;
    }
    __syncthreads();
    if (fix_at) *fix_at = fix;
}

// Lets the kernel use shared memory up to what any step needs (one value for
// all calls: it is the kernel's, not the launch's), unless that was done on
// this device.
template <class Kernel>
cudaError_t allow_memory(Kernel *kernel, int done, int *device) {
    cudaError_t e = cudaGetDevice(device);
    if (e != cudaSuccess || *device == done) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kStepMemory);
}

template <int TYPE, int G, bool MASK, bool UNIT>
cudaError_t launch_clusters(const OutStep &a, cudaStream_t stream) {
    auto *kernel = outcomes_step<TYPE, G, MASK, UNIT>;
    const size_t row_bytes = (size_t)a.r.seg_vecs * kOutVecBytes + step_lists(a.teacher.count);
    thread_local struct {      // what costs as much as the launch to set or ask
        int device = -1;
        size_t bytes = 0;
        int64_t segs = 0;
        int most = 0;
    } known;
    int device;
    cudaError_t e = allow_memory(kernel, known.device, &device);
    if (e != cudaSuccess) return e;
    if (known.device != device) known.bytes = 0;
    known.device = device;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(G);
    cfg.dynamicSmemBytes = row_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.r.segs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // as many clusters as run at once: each goes through its share of the rows
    int64_t clusters = a.r.rows;
    if (clusters * a.r.segs > kOutSms) {
        if (known.bytes != row_bytes || known.segs != a.r.segs) {
            cfg.numAttrs = 1;
            cfg.gridDim = dim3((unsigned)a.r.segs);
            e = cudaOccupancyMaxActiveClusters(&known.most, kernel, &cfg);
            if (e != cudaSuccess) return e;
            known.bytes = row_bytes;
            known.segs = a.r.segs;
        }
        if (known.most > 0 && clusters > known.most) clusters = known.most;
    }
    cfg.gridDim = dim3((unsigned)(clusters * a.r.segs));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int TYPE, bool MASK, bool UNIT>
cudaError_t launch_step(const OutStep &a, bool warp_rows, cudaStream_t stream) {
    size_t row_bytes = (size_t)a.r.seg_vecs * kOutVecBytes;
    if (warp_rows) {
        const int groups = kOutThreads / 32;
        auto *kernel = outcomes_step_warps<TYPE, MASK, UNIT>;
        row_bytes += teacher_bytes(a.teacher.count) + repeat_bytes(a.teacher.count) + repeat_sums(a.teacher.count);
        thread_local int ready = -1;
        const cudaError_t e = allow_memory(kernel, ready, &ready);
        if (e != cudaSuccess) {
            ready = -1;
            return e;
        }
        return launch_pdl(kernel, dim3((unsigned)((a.r.rows + groups - 1) / groups)),
                          dim3(kOutThreads), groups * row_bytes, stream, a);
    }
    return a.wide ? launch_clusters<TYPE, 2 * kStepThreads, MASK, UNIT>(a, stream)
                  : launch_clusters<TYPE, kStepThreads, MASK, UNIT>(a, stream);
}

}  // namespace

template <int TYPE>
cudaError_t outcomes_step_of(const OutStep &a, bool warp_rows, cudaStream_t stream) {
    if constexpr (TYPE == TN_TYPE_C64) {
        if (a.r.scale == 1.f)
            return a.r.mask ? launch_step<TYPE, true, true>(a, warp_rows, stream)
                            : launch_step<TYPE, false, true>(a, warp_rows, stream);
    }
    return a.r.mask ? launch_step<TYPE, true, false>(a, warp_rows, stream)
                    : launch_step<TYPE, false, false>(a, warp_rows, stream);
}

}  // namespace tn
