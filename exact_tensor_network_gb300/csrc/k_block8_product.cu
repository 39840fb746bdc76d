// Products of 8-bit matrices with a scale for each block of 128 (tcgen05, TMA,
// TMEM).
//
// out[p, q] = sum over blocks b of k of sP[p, b] sQ[q, b] (sum of the codes'
// products in b).  The tensor core knows no scales that differ from block to
// block of k, so a block (128 of k: four instructions) is accumulated in TMEM
// from zero and then added, scaled, to fp32 sums in registers; TMEM holds
// several such accumulators, so that the tensor core works on the next blocks
// meanwhile.  Per block and entry that is one packed multiply-add for two
// entries where Q's scale is the same for 128 rows (weights), a
// multiplication more where every row has its own.
//
// A CTA computes a tile of 128 rows of P by BN rows of Q.  One thread loads blocks
// of both operands by TMA into a ring of shared-memory stages (rows of 128
// bytes, 128-byte swizzle), one issues the products, four or eight warps add
// up: warp w owns TMEM lanes 32 (w % 4) .. and, of eight, half of the columns.
//   BN 256: large products.  One persistent CTA an SM, 4 stages of 48 KB, two
//   accumulators that fill TMEM.
//   BN 16 .. 128: one tile a CTA, two CTAs an SM.  Where a has few rows its b is P:
//   the weights' 128 rows are the tensor core's and a's rows its columns, so
//   that nothing is padded to 128 rows and the weights stream at the memory's
//   rate.  Where tiles are fewer than SMs, a cluster of 2, 4 or 8 CTAs shares a tile's k;
//   their sums meet in shared memory, added in the order of k.
//
// Every wait on a barrier is bounded: after its limit the CTA's flag goes up, its
// roles leave, copies and products in flight are waited for (with a limit
// too), TMEM is released and the status word says ERR_TIMEOUT.
#include <cuda_fp16.h>

#include "block8.h"
#include "common.cuh"
#include "tensor_core.cuh"

namespace tn {

namespace {

__device__ DevStatus g_status;

template <int BN>
struct Shape {
    static constexpr bool kBig = BN == 256;
    static constexpr int kWarps = kBig ? 8 : 4;             // that add up
    static constexpr int kThreads = (kWarps + 2) * 32;
    static constexpr int kCols = kBig ? BN / 2 : BN;        // of one such warp
    static constexpr int kBytesP = kB8Tile * 128, kBytesQ = BN * 128;
    static constexpr int kStage = kBytesP + kBytesQ;
    static constexpr int kStages = kBig ? 4 : BN == 128 ? 3 : BN == 64 ? 4 : 5;
    static constexpr int kBufs = BN >= 128 ? 2 : BN == 64 ? 4 : 8;
    static constexpr int kTmem = BN * kBufs;
    static constexpr int kRing = kStage * kStages;
    // each adding warp's: scales of Q of two blocks; in large tiles also a 32 x 32 block on
    // its way to the output (others use the ring, which is free by then)
    static constexpr int kStaging = 32 * 33 * 4;
    static constexpr int kOwn = kBig ? kStaging : 2 * kCols * 4;
    static constexpr int kBars = 2 * kStages + 2 * kBufs + 1;
    static constexpr int kSmem = 1024 + kRing + kWarps * kOwn + kBars * 8 + 16;
    static constexpr int kCtas = kBig ? 1 : 2;              // on an SM
    static constexpr uint32_t kWhat = (1u << 4) | (static_cast<uint32_t>(BN) >> 3 << 17) | (128u >> 4 << 24);
    static constexpr int kPitch = kB8Tile + 1;              // of a column of shared sums
    static_assert(kSmem <= (kBig ? 232448 : 115712) && kTmem * kCtas <= 512, "an SM's memory");
    static_assert(kBig || (BN * kPitch * 4 <= kRing && kWarps * kStaging <= kRing), "the ring holds the sums");
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return reinterpret_cast<float2 &>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return reinterpret_cast<float2 &>(d);
}

__device__ __forceinline__ void store(void *out, int32_t type, int64_t at, float v) {
    if (type == TN_TYPE_F32) static_cast<float *>(out)[at] = v;
    else if (type == TN_TYPE_BF16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
    else static_cast<__half *>(out)[at] = __float2half_rn(v);
}

// Tile t: groups of eight row tiles, columns inside, so that the tiles that run
// at once share operands in L2.
__device__ __forceinline__ void tile_of(int64_t t, const ProductArgs &a, int64_t &pt, int64_t &qt) {
    const int64_t group = 8 * a.qtiles, g = t / group, first = g * 8;
    const int64_t n = a.ptiles - first < 8 ? a.ptiles - first : 8;
    const int64_t r = t - g * group;
    qt = r / n;
    pt = first + (r - qt * n);
}

template <int BN, bool EACH>
__global__ void __launch_bounds__(Shape<BN>::kThreads, Shape<BN>::kCtas)
    product_kernel(const __grid_constant__ ProductArgs a) {
    using S = Shape<BN>;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    unsigned char *own = smem + S::kRing;
    uint64_t *bars = reinterpret_cast<uint64_t *>(own + S::kWarps * S::kOwn);
    const uint32_t full = tc::smem_address(bars), empty = full + 8 * S::kStages;
    const uint32_t tfull = empty + 8 * S::kStages, tempty = tfull + 8 * S::kBufs, end = tempty + 8 * S::kBufs;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + S::kBars);
    volatile int *gave_up = reinterpret_cast<volatile int *>(slot + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            tc::bar_init(full + 8 * s, 1);
            tc::bar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < S::kBufs; ++b) {
            tc::bar_init(tfull + 8 * b, 1);
            tc::bar_init(tempty + 8 * b, S::kWarps);
        }
        tc::bar_init(end, 1);
        *gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == S::kWarps + 1) tc::tmem_alloc<S::kTmem>(tc::smem_address(slot));
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *slot;
    // Only now: a following grid that holds TMEM while it waits for this one
    // must not be able to take what this one's CTAs still need.
    pdl_trigger();
    pdl_wait();

    const int split = a.split;
    const uint32_t rank = split > 1 ? tc::cluster_rank() : 0;
    const int64_t tiles = a.ptiles * a.qtiles;
    const int64_t first = split > 1 ? blockIdx.x / split : blockIdx.x;
    const int64_t step = split > 1 ? gridDim.x / split : gridDim.x;
    // this CTA's blocks of k
    const int kb0 = static_cast<int>(static_cast<int64_t>(a.kbs) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(a.kbs) * (rank + 1) / split);

    if (warp == S::kWarps) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0, parity = 0;
            bool ok = true;
            for (int64_t t = first; t < tiles && ok; t += step) {
                int64_t pt, qt;
                tile_of(t, a, pt, qt);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!tc::bar_wait(empty + 8 * stage, phase ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full + 8 * stage, to = tc::smem_address(smem) + stage * S::kStage;
                    tc::bar_expect(bar, S::kStage);
                    tc::load_2d(to, &a.tmP, bar, kb * 128, static_cast<int32_t>(pt * kB8Tile));
                    tc::load_2d(to + S::kBytesP, &a.tmQ, bar, kb * 128, static_cast<int32_t>(qt * BN));
                    issued |= 1u << stage;
                    parity = (parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)
                for (int s = 0; s < S::kStages; ++s)
                    if (issued & (1u << s)) tc::bar_wait_end(full + 8 * s, (parity >> s) & 1);
        }
    } else if (warp == S::kWarps + 1) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
            bool ok = true;
            for (int64_t t = first; t < tiles && ok; t += step) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!tc::bar_wait(tempty + 8 * buf, bphase ^ 1, gave_up) ||
                        !tc::bar_wait(full + 8 * stage, phase, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t at = tc::smem_address(smem) + stage * S::kStage;
                    const uint32_t da = tc::desc_lo(at), db = tc::desc_lo(at + S::kBytesP), d = tmem + buf * BN;
                    tc::mma8<false>(d, da, db, S::kWhat);
#pragma unroll
                    for (int i = 1; i < 4; ++i) tc::mma8<true>(d, da + 2 * i, db + 2 * i, S::kWhat);
                    tc::mma_commit(empty + 8 * stage);
                    tc::mma_commit(tfull + 8 * buf);
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    if (++buf == S::kBufs) {
                        buf = 0;
                        bphase ^= 1;
                    }
                }
            }
            if (!ok) {      // TMEM is not released under products in flight
                tc::mma_commit(end);
                tc::bar_wait_end(end, 0);
            }
        }
    } else {
        const int quad = warp % 4, col0 = (warp / 4) * S::kCols;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
        float *mine = reinterpret_cast<float *>(own + warp * S::kOwn);
        uint32_t buf = 0, bphase = 0;
        bool ok = true;
        for (int64_t t = first; t < tiles && ok; t += step) {
            int64_t pt, qt;
            tile_of(t, a, pt, qt);
            const int64_t p = pt * kB8Tile + quad * 32 + lane, q0 = qt * BN + col0;
            const float *sp = a.scaleP + ((p < a.p ? p : a.p - 1) >> a.shiftP) * a.strideP;
            // scales of Q: of the warp's columns lane, lane + 32, .., or of all
            constexpr int kScales = EACH ? (S::kCols + 31) / 32 : 1;
            const float *sq[kScales];
#pragma unroll
            for (int i = 0; i < kScales; ++i) {
                int64_t q = q0 + (EACH ? (lane + 32 * i) % S::kCols : 0);
                q = q < a.q ? q : a.q - 1;
                sq[i] = a.scaleQ + (q >> a.shiftQ) * a.strideQ;
            }
            float2 acc[S::kCols / 2];
#pragma unroll
            for (int i = 0; i < S::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            float next_p = 0.f, next_q[kScales] = {};
            if (kb0 < kb1) {
                next_p = __ldcg(sp + kb0);
#pragma unroll
                for (int i = 0; i < kScales; ++i) next_q[i] = __ldcg(sq[i] + kb0);
            }
            for (int kb = kb0; kb < kb1; ++kb) {
                float s = next_p;
                float *qs = mine + (kb & 1) * S::kCols;
                if constexpr (EACH) {
#pragma unroll
                    for (int i = 0; i < kScales; ++i)
                        if (lane + 32 * i < S::kCols) qs[lane + 32 * i] = next_q[i];
                    __syncwarp();
                } else {
                    // 0 times a product beyond fp32's range is 0 all the same
                    const float both = s * next_q[0];
                    s = isinf(both) && !isinf(s) && !isinf(next_q[0]) ? copysignf(3.402823466e38f, both) : both;
                }
                if (kb + 1 < kb1) {
                    next_p = __ldcg(sp + kb + 1);
#pragma unroll
                    for (int i = 0; i < kScales; ++i) next_q[i] = __ldcg(sq[i] + kb + 1);
                }
                if (!tc::bar_wait(tfull + 8 * buf, bphase, gave_up)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t from = tbase + buf * BN;
                const float2 s2 = make_float2(s, s);
                uint32_t r[2][16];
                tc::tmem_load(from, r[0]);
#pragma unroll
                for (int c = 0; c < S::kCols / 16; ++c) {
                    uint32_t(&v)[16] = r[c & 1];
                    tc::tmem_wait(v);
                    if (c + 1 < S::kCols / 16) {
                        tc::tmem_load(from + 16 * (c + 1), r[(c + 1) & 1]);
                    } else {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) tc::bar_arrive(tempty + 8 * buf);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 x = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        if constexpr (EACH) x = mul2(x, *reinterpret_cast<const float2 *>(qs + 16 * c + 2 * i));
                        acc[8 * c + i] = fma2(x, s2, acc[8 * c + i]);
                    }
                }
                if (++buf == S::kBufs) {
                    buf = 0;
                    bphase ^= 1;
                }
            }
            if (!ok) break;
            if (!S::kBig && split > 1) {
                // column q of the tile at q * kPitch; the ring is free, as the last
                // products have been read
                float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int i = 0; i < S::kCols / 2; ++i) {
                    part[(2 * i) * S::kPitch + quad * 32 + lane] = acc[i].x;
                    part[(2 * i + 1) * S::kPitch + quad * 32 + lane] = acc[i].y;
                }
            } else if (a.sp == 1) {
#pragma unroll
                for (int i = 0; i < S::kCols; ++i)
                    if (p < a.p && q0 + i < a.q)
                        store(a.out, a.type, p + (q0 + i) * a.sq, i & 1 ? acc[i / 2].y : acc[i / 2].x);
            } else {
                // 32 x 32 blocks turned in shared memory: a row's 32 columns are stored at once
                float *block = S::kBig ? mine : reinterpret_cast<float *>(smem) + warp * 32 * 33;
                const int64_t p0 = pt * kB8Tile + quad * 32;
                const int rows = static_cast<int>(a.p - p0 < 32 ? a.p - p0 : 32);
#pragma unroll
                for (int c = 0; c < (S::kCols + 31) / 32; ++c) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < (S::kCols < 32 ? S::kCols : 32); ++i)
                        block[lane * 33 + i] = i & 1 ? acc[16 * c + i / 2].y : acc[16 * c + i / 2].x;
                    __syncwarp();
                    const int64_t q = q0 + 32 * c + lane;
                    if (q < a.q && lane < S::kCols)
                        for (int r = 0; r < rows; ++r) store(a.out, a.type, (p0 + r) * a.sp + q, block[r * 33 + lane]);
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    if (!S::kBig && split > 1) {
        // CTA `rank` finishes its share of the tile: columns where p is the output's
        // inner axis, rows where q is
        tc::cluster_sync();
        int64_t pt, qt;
        tile_of(first, a, pt, qt);
        const uint32_t part = tc::smem_address(smem);
        const bool inner_p = a.sp == 1;
        const int lo = (inner_p ? BN : kB8Tile) * rank / split, hi = (inner_p ? BN : kB8Tile) * (rank + 1) / split;
        const int inner = inner_p ? kB8Tile : BN;
        for (int i = threadIdx.x; i < (hi - lo) * inner; i += S::kThreads) {
            const int o = lo + i / inner, n = i % inner;
            const int pp = inner_p ? n : o, qq = inner_p ? o : n;
            const int64_t p = pt * kB8Tile + pp, q = qt * BN + qq;
            if (p >= a.p || q >= a.q) continue;
            float sum = 0.f;
            for (int r = 0; r < split; ++r) sum += tc::cluster_load(tc::in_cta(part + (qq * S::kPitch + pp) * 4, r));
            store(a.out, a.type, p * a.sp + q * a.sq, sum);
        }
        tc::cluster_sync();     // others may still read this CTA's sums
    }
    tc::fence_before();
    __syncthreads();
    if (warp == S::kWarps + 1) {
        tc::fence_after();
        tc::tmem_free<S::kTmem>(tmem);
    }
    if (threadIdx.x == 0 && *gave_up) atomicCAS(&g_status.code, ERR_NONE, ERR_TIMEOUT);
}

template <int BN, bool EACH>
cudaError_t launch(const ProductArgs &a, cudaStream_t stream) {
    using S = Shape<BN>;
    auto kernel = product_kernel<BN, EACH>;
    static uint64_t ready = 0;      // devices whose limit is raised
    int device;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (!(__atomic_load_n(&ready, __ATOMIC_RELAXED) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&ready, bit, __ATOMIC_RELAXED);
    }
    const int64_t tiles = a.ptiles * a.qtiles;
    const int64_t ctas = S::kBig ? (tiles < kB8Sms ? tiles : kB8Sms) : tiles * a.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_product(const ProductArgs &a, int bn, bool each, cudaStream_t stream) {
    switch (bn) {
        case 256: return each ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
        case 128: return each ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
        case 64: return launch<64, true>(a, stream);
        case 32: return launch<32, true>(a, stream);
        default: return launch<16, true>(a, stream);
    }
}

cudaError_t block8_status(DevStatus *s) {
    cudaError_t e = cudaMemcpyFromSymbol(s, g_status, sizeof(*s));
    if (e != cudaSuccess || s->code == ERR_NONE) return e;
    const DevStatus none = {ERR_NONE, 0};
    return cudaMemcpyToSymbol(g_status, &none, sizeof(none));
}

}  // namespace tn
