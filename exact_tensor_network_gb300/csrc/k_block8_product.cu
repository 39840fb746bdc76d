// Products of 8-bit matrices with any fp32 scale for each block of 128 (tcgen05, TMA,
// TMEM).  Where scales are powers of two k_block8_scaled.cu has the faster way.
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
// A CTA computes tiles of 128 rows of P by BN rows of Q.  One thread loads blocks
// of both operands by TMA into a ring of shared-memory stages (rows of 128
// bytes, 128-byte swizzle), one issues the products, four or eight warps add up: warp w
// owns TMEM lanes 32 (w % 4) .. and, of eight, half of the columns.  The loader and the
// issuer run ahead of the adding warps from tile to tile.  A block costs one commit: it
// tells the adding warps that its sums stand, and they tell the loader that its stage
// is free (a commit costs the tensor core 130 cycles, a block's products 512; a
// second one made 170 us of nothing but products 205).
//   BN 256 and 128: large products.  One CTA an SM, a ring of 192 KB, accumulators
//   that fill TMEM, and registers moved to the adding warps.
//   BN 16 .. 64: two CTAs an SM.
// Where a has few rows its b is P: the weights' 128 rows are the tensor core's and
// a's rows its columns, so that nothing is padded to 128 rows and the weights
// stream at the memory's rate.  Where tiles are fewer than SMs, a cluster of 2, 4 or 8
// CTAs shares a tile's k; their sums meet in shared memory, added in the order of k.
//
// Every wait on a barrier is bounded: after its limit the CTA's flag goes up, its
// roles leave, copies and products in flight are waited for (with a limit
// too), TMEM is released and the device's count of timeouts goes up.
#include "block8_product.cuh"

namespace tn {

namespace {

template <int BN, bool EACH>
struct Shape {
    static constexpr bool kBig = BN >= 128;
    static constexpr int kWarps = kBig ? 8 : 4;             // that add up
    // Of large tiles the first warpgroup loads and issues, and gives registers to the
    // two that add up (128 fp32 sums a thread); of small ones the last.
    static constexpr int kFirst = kBig ? 4 : 0;             // of the adding warps
    static constexpr int kLoader = kBig ? 0 : kWarps, kIssuer = kLoader + 1;
    static constexpr int kThreads = kBig ? 384 : (kWarps + 2) * 32;
    static constexpr int kRegsLow = 56, kRegsHigh = 224;    // of 168 at launch
    static constexpr int kCols = kBig ? BN / 2 : BN;        // of an adding warp
    static constexpr int kStep = kCols < 32 ? 16 : 32;      // columns read from TMEM at once
    static constexpr int kBytesP = kB8Tile * 128, kBytesQ = BN * 128;
    static constexpr int kStage = kBytesP + kBytesQ;
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : BN == 64 ? 4 : 5;
    static constexpr int kBufs = BN == 256 ? 2 : BN >= 64 ? 4 : 8;
    static constexpr int kTmem = BN * kBufs;
    static constexpr int kRing = kStage * kStages;
    // words of each adding warp: the scales of its columns of two blocks, and at the end of a tile
    // kTurn bytes of its 32 rows on their way out
    static constexpr int kTurn = kBig ? 64 : 32;
    static constexpr int kOwn = 32 * (kTurn + 16) / 4;
    static constexpr int kBars = 2 * kStages + 2 * kBufs + 1;
    static constexpr int kSmem = 1024 + kRing + kWarps * kOwn * 4 + kBars * 8 + 16;
    static constexpr int kCtas = kBig ? 1 : 2;              // on an SM
    static constexpr uint32_t kWhat = (1u << 4) | (static_cast<uint32_t>(BN) >> 3 << 17) | (128u >> 4 << 24);
    static_assert(kSmem <= (kBig ? 232448 : 115712) && kTmem * kCtas <= 512, "an SM's memory");
    static_assert(3 * kCols <= kOwn, "scales of two blocks, and ones");
    static_assert(BN == 256 || part_bytes(BN) <= kRing, "the ring holds the sums");
    static_assert(!kBig || 4 * kRegsLow + 8 * kRegsHigh <= 12 * 168, "registers of the launch");
};

// acc += (sums of a block) * scales, of N columns
template <bool EACH, int N>
__device__ __forceinline__ void add_scaled(float2 *acc, const uint32_t (&v)[N], float s, const float *qs) {
    const float2 s2 = make_float2(s, s);
#pragma unroll
    for (int i = 0; i < N / 2; i += 2) {
        float2 x = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        float2 y = make_float2(__uint_as_float(v[2 * i + 2]), __uint_as_float(v[2 * i + 3]));
        if constexpr (EACH) {
            const float4 q = *reinterpret_cast<const float4 *>(qs + 2 * i);
            x = mul2(x, make_float2(q.x, q.y));
            y = mul2(y, make_float2(q.z, q.w));
        }
        acc[i] = fma2(x, s2, acc[i]);
        acc[i + 1] = fma2(y, s2, acc[i + 1]);
    }
}

// Where the product of two scales, or a block's sum (0, or 2^-18 .. 2^25) times Q's scale, is no normal number although
// the value may be one, sums are scaled before they are added: a scale is split into a number with half of its
// exponent and a power of two, and the sum times both of the first and then times both powers leaves fp32 only
// where the value does.
struct Halves {
    float part, power;
};
__device__ __forceinline__ Halves halves_of(float x) {
    if (x == 0.f || !(fabsf(x) <= 3.402823466e38f)) return {x, 1.f};
    int e;
    const float m = frexpf(x, &e);
    return {ldexpf(m, e - (e >> 1)), ldexpf(1.f, e >> 1)};
}
// N columns: row times col, or (EACH) times each column's.
template <bool EACH, int N>
__device__ __forceinline__ void scale_far(uint32_t (&v)[N], float row, float col, const float *each) {
    const Halves p = halves_of(row);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const Halves q = halves_of(EACH ? each[i] : col);
        v[i] = __float_as_uint(__uint_as_float(v[i]) * (p.part * q.part) * fminf(p.power * q.power, 0x1p127f));
    }
}
// Whether two scales have to go that way; whether Q's of a column of its own has to.
__device__ __forceinline__ bool far_product(float s, float q) {
    const float x = fabsf(s * q);
    return !(x >= 0x1p-126f && x <= 3.402823466e38f) && s != 0.f && q != 0.f && fabsf(s) <= 3.402823466e38f &&
           fabsf(q) <= 3.402823466e38f;
}
__device__ __forceinline__ bool far_scale(float q) {
    const float x = fabsf(q);
    return (x < 0x1p-100f && x > 0.f) || (x > 0x1p100f && x <= 3.402823466e38f);
}

template <int BN, bool EACH>
__global__ void __launch_bounds__(Shape<BN, EACH>::kThreads, Shape<BN, EACH>::kCtas)
    product_kernel(const __grid_constant__ ProductArgs a) {
    using S = Shape<BN, EACH>;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    float *own = reinterpret_cast<float *>(smem + S::kRing);
    uint64_t *bars = reinterpret_cast<uint64_t *>(own + S::kWarps * S::kOwn);
    const uint32_t full = tc::smem_address(bars), empty = full + 8 * S::kStages;
    const uint32_t tfull = empty + 8 * S::kStages, tempty = tfull + 8 * S::kBufs;
    const uint32_t end = tempty + 8 * S::kBufs;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + S::kBars);
    volatile int *gave_up = reinterpret_cast<volatile int *>(slot + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            tc::bar_init(full + 8 * s, 1);
            tc::bar_init(empty + 8 * s, S::kWarps);
        }
        for (int b = 0; b < S::kBufs; ++b) {
            tc::bar_init(tfull + 8 * b, 1);
            tc::bar_init(tempty + 8 * b, S::kWarps);
        }
        tc::bar_init(end, 1);
        *gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == S::kIssuer) tc::tmem_alloc<S::kTmem>(tc::smem_address(slot));
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

    const bool adds = S::kBig ? warp >= S::kFirst : warp < S::kWarps;
    if (!adds) {
        if constexpr (S::kBig) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsLow));
        if (warp == S::kLoader && lane == 0) {
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
        if (warp == S::kIssuer && lane == 0) {
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
        if constexpr (S::kBig) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsHigh));
        const int quad = warp % 4, col0 = (warp - S::kFirst) / 4 * S::kCols;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
        float *mine = own + (warp - S::kFirst) * S::kOwn;
        uint32_t buf = 0, bphase = 0, stage = 0;
        bool ok = true;
        for (int64_t t = first; t < tiles && ok; t += step) {
            int64_t pt, qt;
            tile_of(t, a, pt, qt);
            const int64_t p0 = pt * kB8Tile + quad * 32, q0 = qt * BN + col0;
            // scales, read two blocks ahead: of the lane's row of P, and of Q's columns lane,
            // lane + 32, .. or of all of the warp's
            constexpr int kQ = EACH ? (S::kCols + 31) / 32 : 1;
            const float *sp = a.scaleP + ((p0 + lane < a.p ? p0 + lane : a.p - 1) >> a.shiftP) * a.strideP;
            const float *sq[kQ];
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                const int64_t q = q0 + (EACH ? (lane + 32 * i) % S::kCols : 0);
                sq[i] = a.scaleQ + ((q < a.q ? q : a.q - 1) >> a.shiftQ) * a.strideQ;
            }
            float np[2] = {}, nq[2][kQ] = {};
#pragma unroll
            for (int n = 0; n < 2; ++n)
                if (kb0 + n < kb1) {
                    np[n] = __ldcg(sp + (kb0 + n) * a.blockP);
#pragma unroll
                    for (int i = 0; i < kQ; ++i) nq[n][i] = __ldcg(sq[i] + (kb0 + n) * a.blockQ);
                }
            float2 acc[S::kCols / 2];
#pragma unroll
            for (int i = 0; i < S::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int kb = kb0; kb < kb1; ++kb) {
                float s = np[0];
                const float *qs = mine + (kb & 1) * S::kCols;
                bool far = false;
                if constexpr (EACH) {
#pragma unroll
                    for (int i = 0; i < kQ; ++i) {
                        if (lane + 32 * i < S::kCols) mine[(kb & 1) * S::kCols + lane + 32 * i] = nq[0][i];
                        far |= far_scale(nq[0][i]);
                    }
                    __syncwarp();
                } else {
                    far = far_product(s, nq[0][0]);
                    s *= nq[0][0];
                }
                far = __any_sync(0xffffffffu, far);
                if (far) {      // scaled before they are added: with 1 from then on
                    s = 1.f;
                    if constexpr (EACH) {
#pragma unroll
                        for (int i = 0; i < kQ; ++i)
                            if (lane + 32 * i < S::kCols) mine[2 * S::kCols + lane + 32 * i] = 1.f;
                        __syncwarp();
                        qs = mine + 2 * S::kCols;
                    }
                }
                // (the scales are read again: kept until here they would cost every product registers)
                const auto if_far = [&](auto &r, int c) {
                    if (far) scale_far<EACH>(r, __ldcg(sp + kb * a.blockP), EACH ? 0.f : __ldcg(sq[0] + kb * a.blockQ),
                                             mine + (kb & 1) * S::kCols + c);
                };
                np[0] = np[1];
#pragma unroll
                for (int i = 0; i < kQ; ++i) nq[0][i] = nq[1][i];
                if (kb + 2 < kb1) {
                    np[1] = __ldcg(sp + (kb + 2) * a.blockP);
#pragma unroll
                    for (int i = 0; i < kQ; ++i) nq[1][i] = __ldcg(sq[i] + (kb + 2) * a.blockQ);
                }
                if (!tc::warp_wait(tfull + 8 * buf, bphase, gave_up)) {
                    ok = false;
                    break;
                }
                tc::bar_arrive_once(empty + 8 * stage);
                if (++stage == S::kStages) stage = 0;
                tc::fence_after();
                const uint32_t from = tbase + buf * BN;
                const auto loaded = [&] {       // all of the accumulator is in registers
                    tc::fence_before();
                    __syncwarp();
                    tc::bar_arrive_once(tempty + 8 * buf);
                };
                if constexpr (!S::kBig) {
                    uint32_t r[S::kStep];
#pragma unroll
                    for (int c = 0; c < S::kCols; c += S::kStep) {
                        tc::tmem_load(from + c, r);
                        tc::tmem_wait(r);
                        if (c + S::kStep == S::kCols) loaded();
                        if_far(r, c);
                        add_scaled<EACH>(acc + c / 2, r, s, qs + c);
                    }
                } else {
                    // two loads in flight; the next pair starts as its registers come free
                    uint32_t r0[32], r1[32];
                    tc::tmem_load(from, r0);
                    tc::tmem_load(from + 32, r1);
                    tc::tmem_wait(r0, r1);
#pragma unroll
                    for (int c = 0; c < S::kCols; c += 64) {
                        const bool more = c + 64 < S::kCols;
                        if (!more) loaded();
                        if_far(r0, c);
                        if_far(r1, c + 32);
                        add_scaled<EACH>(acc + c / 2, r0, s, qs + c);
                        if (more) tc::tmem_load(from + c + 64, r0);
                        add_scaled<EACH>(acc + c / 2 + 16, r1, s, qs + c + 32);
                        if (more) {
                            tc::tmem_load(from + c + 96, r1);
                            tc::tmem_wait(r0, r1);
                        }
                    }
                }
                if (++buf == S::kBufs) {
                    buf = 0;
                    bphase ^= 1;
                }
            }
            if (!ok) break;
            // (shared: the ring is free, as the last products have been read)
            if (BN < 256 && split > 1)
                keep_part<BN, S::kCols>(a, reinterpret_cast<float *>(smem), acc, quad * 32 + lane, col0);
            else
                store_sums<S::kCols, BN == 256, S::kTurn>(a, acc, mine, p0, q0, (qt + 1) * BN);
        }
    }
    __syncwarp();
    if (BN < 256 && split > 1) join_parts<BN, S::kThreads>(a, reinterpret_cast<const float *>(smem), first, rank);
    tc::fence_before();
    __syncthreads();
    if (warp == S::kIssuer) {
        tc::fence_after();
        tc::tmem_free<S::kTmem>(tmem);
    }
    if (threadIdx.x == 0 && *gave_up) atomicAdd(&a.status->timeouts, 1ull);
}

template <int BN, bool EACH>
cudaError_t launch(const ProductArgs &a, cudaStream_t stream) {
    using S = Shape<BN, EACH>;
    static uint64_t ready = 0;
    return launch_tiles(product_kernel<BN, EACH>, a, S::kThreads, S::kSmem, S::kCtas * kB8Sms, &ready, stream);
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

}  // namespace tn
