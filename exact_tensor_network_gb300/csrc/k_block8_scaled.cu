// Products of 8-bit matrices whose scales are powers of two (tcgen05 with block
// scales, TMA, TMEM).
//
// out[p, q] = sum over blocks b of k of sP[p, b] sQ[q, b] (sum of the codes' products in
// b).  The tensor core takes a power of two for each 32 of k of each row of both
// operands, so it can add up scaled blocks by itself, and a row's scale is the same
// for the four instructions of a block.  What is left for the other warps are the sums of
// four blocks at a time: its additions round towards zero, a loss of up to 2^-24 each
// that all go one way, so after 16 of them (512 of k) the sums are added to fp32
// registers, rounded to nearest.  (With any fp32 scale, k_block8_product.cu, every block
// goes that way, which costs more than the products.)
//
// A CTA computes tiles of 128 rows of P by BN rows of Q.  One thread loads blocks of
// both operands by TMA into a ring of shared-memory stages, one issues the products, two
// warps turn four blocks' scales into bytes (biased exponents) in the order that TMEM
// wants, four or eight warps add up and store.  All run ahead of each other from tile to
// tile.
//   BN 240: large products; two accumulators and the scales fill TMEM (256 would
//   leave no room for scales).  One CTA an SM, four stages of 46 KB.
//   BN 128: fewer rows, or tiles too few: clusters of 2, 4 or 8 CTAs share a tile's k.
//   BN 16 .. 64: two CTAs an SM, for a few rows of a: its b is P then (see
//   k_block8_product.cu), and the weights' bytes are what bounds them.
#include "block8_product.cuh"

namespace tn {

namespace {

__device__ Block8Status g_status;

constexpr int kGroup = 4;       // blocks of k that are added up by the tensor core

template <int BN>
struct Shape {
    static constexpr bool kBig = BN >= 128;
    static constexpr int kWarps = kBig ? 8 : 4;             // that add up
    static constexpr int kFirst = kBig ? 4 : 0;
    static constexpr int kLoader = kBig ? 0 : kWarps, kIssuer = kLoader + 1, kScaler = kLoader + 2;
    static constexpr int kThreads = (kWarps + 4) * 32;
    static constexpr int kRegsLow = 72, kRegsHigh = 216;    // of 168 at launch, large tiles
    static constexpr int kCols = BN == 240 ? 128 : kBig ? BN / 2 : BN;     // of an adding warp (240: 128 and 112)
    static constexpr int kStep = kCols < 32 ? 16 : 32;
    static constexpr int kBytesP = kB8Tile * 128, kBytesQ = BN * 128;
    static constexpr int kStage = kBytesP + kBytesQ;
    static constexpr int kStages = BN == 240 ? 4 : BN == 128 ? 5 : BN == 64 ? 4 : 5;
    static constexpr int kRing = kStage * kStages;
    // accumulators of two groups, then their scales: four columns for P's 128 rows, four
    // for each 128 of Q's
    static constexpr int kBufs = 2, kScales = BN > 128 ? 12 : 8;
    static constexpr int kScaleAt = kBufs * BN;
    static constexpr int kTmem = BN == 240 ? 512 : BN == 128 ? 512 : BN == 64 ? 256 : BN == 32 ? 128 : 64;
    static constexpr int kSlot = kScales * 128, kSlots = 2;         // bytes in shared memory
    static constexpr int kTurn = kBig ? 128 : 32;           // bytes of its 32 rows that an adding warp stores at once
    static constexpr int kOwn = 32 * (kTurn + 16) / 4;
    static constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kSlots + 1;
    static constexpr int kSmem = 1024 + kRing + kSlots * kSlot + kWarps * kOwn * 4 + kBars * 8 + 16;
    static constexpr int kCtas = kBig ? 1 : 2;
    // e4m3 both, N, M = 128, scales of 8 exponent bits
    static constexpr uint32_t kWhat = (static_cast<uint32_t>(BN) >> 3 << 17) | (1u << 23) | (128u >> 7 << 27);
    static_assert(kScaleAt + 16 * kBufs <= kTmem && kScaleAt % 16 == 0, "columns of TMEM");
    static_assert(kSmem <= (kBig ? 232448 : 115712) && kTmem * kCtas <= 512, "an SM's memory");
    static_assert(BN == 240 || part_bytes(BN) <= kRing, "the ring holds the sums");
    static_assert(!kBig || 4 * kRegsLow + 8 * kRegsHigh <= 12 * 168, "registers of the launch");
};

template <int N>
__device__ __forceinline__ void add_sums(float2 *acc, const uint32_t (&v)[N]) {
    const float2 one = make_float2(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        acc[i] = fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), one, acc[i]);
}

template <int BN>
__global__ void __launch_bounds__(Shape<BN>::kThreads, Shape<BN>::kCtas)
    scaled_kernel(const __grid_constant__ ProductArgs a) {
    using S = Shape<BN>;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    unsigned char *scales = smem + S::kRing;
    float *own = reinterpret_cast<float *>(scales + S::kSlots * S::kSlot);
    uint64_t *bars = reinterpret_cast<uint64_t *>(own + S::kWarps * S::kOwn);
    const uint32_t full = tc::smem_address(bars), empty = full + 8 * S::kStages;
    const uint32_t tfull = empty + 8 * S::kStages, tempty = tfull + 8 * S::kBufs;
    const uint32_t sfull = tempty + 8 * S::kBufs, sempty = sfull + 8 * S::kSlots, end = sempty + 8 * S::kSlots;
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
        for (int b = 0; b < S::kSlots; ++b) {
            tc::bar_init(sfull + 8 * b, 2);
            tc::bar_init(sempty + 8 * b, S::kWarps);
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
            uint32_t stage = 0, phase = 0, buf = 0, bphase = 0, place = 0, sphase = 0;
            bool ok = true;
            for (int64_t t = first; t < tiles && ok; t += step) {
                for (int g = kb0; g < kb1 && ok; g += kGroup) {
                    if (!tc::bar_wait(tempty + 8 * buf, bphase ^ 1, gave_up) ||
                        !tc::bar_wait(sfull + 8 * place, sphase, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t d = tmem + buf * BN, sa = tmem + S::kScaleAt + 16 * buf, sb = sa + 4;
                    const uint32_t from = tc::smem_address(scales) + place * S::kSlot;
#pragma unroll
                    for (int i = 0; i < S::kScales / 4; ++i) tc::copy_scales(sa + 4 * i, from + 512 * i);
                    const int n = kb1 - g < kGroup ? kb1 - g : kGroup;
                    for (int j = 0; j < n; ++j) {
                        if (!tc::bar_wait(full + 8 * stage, phase, gave_up)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        const uint32_t at = tc::smem_address(smem) + stage * S::kStage;
                        const uint32_t da = tc::desc_lo(at), db = tc::desc_lo(at + S::kBytesP);
                        const uint32_t what = S::kWhat | static_cast<uint32_t>(j) << 4 | static_cast<uint32_t>(j) << 29;
                        if (j == 0) tc::mma8_scaled<false>(d, da, db, what, sa, sb);
                        else tc::mma8_scaled<true>(d, da, db, what, sa, sb);
#pragma unroll
                        for (int i = 1; i < 4; ++i) tc::mma8_scaled<true>(d, da + 2 * i, db + 2 * i, what, sa, sb);
                        tc::mma_commit(empty + 8 * stage);
                        if (++stage == S::kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    tc::mma_commit(tfull + 8 * buf);
                    if (++buf == S::kBufs) {
                        buf = 0;
                        bphase ^= 1;
                    }
                    if (++place == S::kSlots) {
                        place = 0;
                        sphase ^= 1;
                    }
                }
            }
            if (!ok) {      // TMEM is not released under products in flight
                tc::mma_commit(end);
                tc::bar_wait_end(end, 0);
            }
        }
        if (warp >= S::kScaler) {
            // Row r of 128: four blocks' bytes at 16 (r % 32) + 4 (r / 32).  This warp has every other
            // 32 rows, of P (the first 128) and then of Q; the next group's scales are on
            // their way while a place is waited for.
            constexpr int kSets = (kB8Tile + (BN + 31) / 32 * 32 + 32) / 64, kSetsP = kB8Tile / 64;
            const int odd = warp - S::kScaler;
            uint32_t place = 0, phase = 0;
            bool ok = true, wrong = false;
            for (int64_t t = first; t < tiles && ok; t += step) {
                int64_t pt, qt;
                tile_of(t, a, pt, qt);
                const float *from[kSets];
                float v[kSets][kGroup];
#pragma unroll
                for (int i = 0; i < kSets; ++i) {
                    const int r = (2 * i + odd) * 32 + lane;
                    int64_t at = i < kSetsP ? pt * kB8Tile + r : qt * BN + r - kB8Tile;
                    const int64_t last = (i < kSetsP ? a.p : a.q) - 1;
                    if (at > last) at = last;
                    from[i] = i < kSetsP ? a.scaleP + (at >> a.shiftP) * a.strideP + kb0 * a.blockP
                                         : a.scaleQ + (at >> a.shiftQ) * a.strideQ + kb0 * a.blockQ;
                }
                const auto load = [&](int g) {
#pragma unroll
                    for (int i = 0; i < kSets; ++i) {
                        const int64_t block = i < kSetsP ? a.blockP : a.blockQ;
#pragma unroll
                        for (int j = 0; j < kGroup; ++j) {
                            v[i][j] = g + j < kb1 ? __ldcg(from[i]) : 1.f;
                            from[i] += block;
                        }
                    }
                };
                load(kb0);
                for (int g = kb0; g < kb1; g += kGroup) {
                    uint32_t w[kSets];
#pragma unroll
                    for (int i = 0; i < kSets; ++i) {
                        w[i] = 0;
#pragma unroll
                        for (int j = 0; j < kGroup; ++j) {
                            const uint32_t b = __float_as_uint(v[i][j]);
                            // a power of two, or NaN; whatever else it is, it is told
                            const bool power = (b & 0x007fffffu) == 0 && b - 0x00800000u < 0x7f000000u;
                            wrong |= !power && (b & 0x7fffffffu) <= 0x7f800000u;
                            w[i] |= (power ? b >> 23 : 0xffu) << (8 * j);
                        }
                    }
                    if (g + kGroup < kb1) load(g + kGroup);
                    if (!tc::warp_wait(sempty + 8 * place, phase ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < kSets; ++i) {
                        const int r = (2 * i + odd) * 32 + lane, q = r % kB8Tile;
                        if (r < kB8Tile + BN)
                            *reinterpret_cast<uint32_t *>(scales + place * S::kSlot + (r / kB8Tile) * 512 + q % 32 * 16 +
                                                          q / 32 * 4) = w[i];
                    }
                    tc::fence_async();
                    __syncwarp();
                    if (lane == 0) tc::bar_arrive(sfull + 8 * place);
                    if (++place == S::kSlots) {
                        place = 0;
                        phase ^= 1;
                    }
                }
            }
            if (wrong) atomicAdd(&a.status->scales, 1ull);
        }
    } else {
        if constexpr (S::kBig) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsHigh));
        const int quad = warp % 4, col0 = (warp - S::kFirst) / 4 * S::kCols;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
        float *mine = own + (warp - S::kFirst) * S::kOwn;
        uint32_t buf = 0, bphase = 0, place = 0;
        bool ok = true;
        for (int64_t t = first; t < tiles && ok; t += step) {
            float2 acc[S::kCols / 2];
#pragma unroll
            for (int i = 0; i < S::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int g = kb0; g < kb1; g += kGroup) {
                if (!tc::warp_wait(tfull + 8 * buf, bphase, gave_up)) {
                    ok = false;
                    break;
                }
                tc::bar_arrive_once(sempty + 8 * place);
                if (++place == S::kSlots) place = 0;
                tc::fence_after();
                const uint32_t from = tbase + buf * BN;
                uint32_t r[S::kStep];
#pragma unroll
                for (int c = 0; c < S::kCols; c += S::kStep) {
                    // (the last of 240 columns: 16 of the 32 behind them are the next accumulator's or scales)
                    tc::tmem_load(from + c, r);
                    tc::tmem_wait(r);
                    if (c + S::kStep == S::kCols) {
                        tc::fence_before();
                        __syncwarp();
                        tc::bar_arrive_once(tempty + 8 * buf);
                    }
                    add_sums(acc + c / 2, r);
                }
                if (++buf == S::kBufs) {
                    buf = 0;
                    bphase ^= 1;
                }
            }
            if (!ok) break;
            int64_t pt, qt;
            tile_of(t, a, pt, qt);
            const int64_t p0 = pt * kB8Tile + quad * 32, q0 = qt * BN + col0;
            // (shared: the ring is free, as the last products have been read)
            if (BN < 240 && split > 1) {
                keep_part<BN, S::kCols>(a, reinterpret_cast<float *>(smem), acc, quad * 32 + lane, col0);
            } else {
                store_sums<S::kCols, BN == 240, S::kTurn>(a, acc, mine, p0, q0, (qt + 1) * BN);
            }
        }
    }
    __syncwarp();
    if (BN < 240 && split > 1) join_parts<BN, S::kThreads>(a, reinterpret_cast<const float *>(smem), first, rank);
    tc::fence_before();
    __syncthreads();
    if (warp == S::kIssuer) {
        tc::fence_after();
        tc::tmem_free<S::kTmem>(tmem);
    }
    if (threadIdx.x == 0 && *gave_up) atomicAdd(&a.status->timeouts, 1ull);
}

template <int BN>
cudaError_t launch(const ProductArgs &a, cudaStream_t stream) {
    using S = Shape<BN>;
    static uint64_t ready = 0;
    return launch_tiles(scaled_kernel<BN>, a, S::kThreads, S::kSmem, S::kCtas * kB8Sms, &ready, stream);
}

}  // namespace

cudaError_t launch_scaled(const ProductArgs &a, int bn, cudaStream_t stream) {
    switch (bn) {
        case 240: return launch<240>(a, stream);
        case 128: return launch<128>(a, stream);
        case 64: return launch<64>(a, stream);
        case 32: return launch<32>(a, stream);
        default: return launch<16>(a, stream);
    }
}

cudaError_t block8_status(Block8Status **p) {
    static Block8Status *known[64] = {};
    int device;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    Block8Status **place = device < 64 ? &known[device] : p;
    *p = device < 64 ? __atomic_load_n(place, __ATOMIC_RELAXED) : nullptr;
    if (*p) return cudaSuccess;
    e = cudaGetSymbolAddress(reinterpret_cast<void **>(p), g_status);
    if (e == cudaSuccess && device < 64) __atomic_store_n(place, *p, __ATOMIC_RELAXED);
    return e;
}

}  // namespace tn
