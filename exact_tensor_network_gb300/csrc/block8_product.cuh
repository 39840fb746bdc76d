// What the kernels of 8-bit products share: the order of tiles, clusters that share a
// tile's k, outputs.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "block8.h"
#include "common.cuh"
#include "tensor_core.cuh"

namespace tn {

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

template <typename T>
__device__ __forceinline__ T rounded(float v) {
    if constexpr (std::is_same<T, float>::value) return v;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(v);
    else return __float2half_rn(v);
}

// An adding warp's sums (32 rows of P, a lane each, by COLS of Q, those below `q_end`) to their
// place.
template <typename T, int COLS, bool ROWS, int TURN>
__device__ __forceinline__ void store_tile(const ProductArgs &a, const float2 *acc, float *block, int64_t p0, int64_t q0,
                                           int64_t q_end) {
    const int lane = threadIdx.x % 32;
    T *out = static_cast<T *>(a.out);
    const int rows = static_cast<int>(a.p - p0 < 32 ? a.p - p0 : 32);
    if (q_end > a.q) q_end = a.q;
    const int cols = static_cast<int>(q_end - q0 < COLS ? q_end - q0 : COLS);
    if (!ROWS && a.sp == 1) {       // lanes are neighbours in the output
        T *to = out + q0 * a.sq + p0 + lane;
#pragma unroll
        for (int i = 0; i < COLS; ++i)
            if (lane < rows && i < cols) to[i * a.sq] = rounded<T>(i & 1 ? acc[i / 2].y : acc[i / 2].x);
        return;
    }
    // TURN bytes of 32 rows at a time, turned in shared memory so that neighbouring lanes store a
    // row's (rows there are an odd number of 16 bytes apart: eight lanes meet all banks)
    constexpr int E = 16 / sizeof(T), FULL = TURN / sizeof(T), STEP = FULL < COLS ? FULL : COLS;
    constexpr int PITCH = (TURN + 16) / sizeof(T);
    T *turned = reinterpret_cast<T *>(block);
    const bool whole = reinterpret_cast<uintptr_t>(out + p0 * a.sp + q0) % 16 == 0 && (a.sp * sizeof(T)) % 16 == 0;
#pragma unroll
    for (int b = 0; b < COLS; b += STEP) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < STEP; i += E) {
            union {
                uint4 w;
                T v[E];
            } u;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = b + i + e;
                u.v[e] = rounded<T>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
            }
            *reinterpret_cast<uint4 *>(turned + lane * PITCH + i) = u.w;
        }
        __syncwarp();
        const int n = cols - b < STEP ? cols - b : STEP;
        T *to = out + p0 * a.sp + q0 + b;
        if (whole && n == STEP) {
            constexpr int LANES = STEP / E;         // of a row
            const int c = lane % LANES * E;
#pragma unroll
            for (int r = lane / LANES; r < 32; r += 32 / LANES)
                if (r < rows) *reinterpret_cast<uint4 *>(to + r * a.sp + c) = *reinterpret_cast<const uint4 *>(turned + r * PITCH + c);
        } else {
            for (int c = lane; c < n; c += 32)
#pragma unroll 4
                for (int r = 0; r < rows; ++r) to[r * a.sp + c] = turned[r * PITCH + c];
        }
    }
    __syncwarp();
}

// An adding warp's sums by the output's type.
template <int COLS, bool ROWS, int TURN>
__device__ __forceinline__ void store_sums(const ProductArgs &a, const float2 *acc, float *block, int64_t p0, int64_t q0,
                                           int64_t q_end) {
    if (a.type == TN_TYPE_F32) store_tile<float, COLS, ROWS, TURN>(a, acc, block, p0, q0, q_end);
    else if (a.type == TN_TYPE_BF16) store_tile<__nv_bfloat16, COLS, ROWS, TURN>(a, acc, block, p0, q0, q_end);
    else store_tile<__half, COLS, ROWS, TURN>(a, acc, block, p0, q0, q_end);
}

// Clusters that share a tile's k.  A CTA's sums lie as the output does, its inner axis with four
// words behind it: neighbouring lanes read 16 bytes each of another CTA's lines.
constexpr int kPartPad = 4;
constexpr int part_bytes(int bn) { return (bn > kB8Tile ? bn : kB8Tile) * (kB8Tile + kPartPad) * 4; }
template <int BN, int COLS>
__device__ __forceinline__ void keep_part(const ProductArgs &a, float *part, const float2 *acc, int row, int col) {
    if (a.sp == 1) {
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) {
            part[(col + 2 * i) * (kB8Tile + kPartPad) + row] = acc[i].x;
            part[(col + 2 * i + 1) * (kB8Tile + kPartPad) + row] = acc[i].y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < COLS / 2; i += 2)
            *reinterpret_cast<float4 *>(part + row * (BN + kPartPad) + col + 2 * i) =
                make_float4(acc[i].x, acc[i].y, acc[i + 1].x, acc[i + 1].y);
    }
}
// All threads of all CTAs: CTA `rank` finishes its share of the tile, lines of the output's inner
// axis.
template <int BN, int THREADS>
__device__ __forceinline__ void join_parts(const ProductArgs &a, const float *mine, int64_t tile, uint32_t rank) {
    tc::cluster_sync();
    const int split = a.split;
    int64_t pt, qt;
    tile_of(tile, a, pt, qt);
    const uint32_t part = tc::smem_address(mine);
    const bool inner_p = a.sp == 1;
    const int lines = inner_p ? BN : kB8Tile, quads = (inner_p ? kB8Tile : BN) / 4;
    const int shift = inner_p ? 5 : BN == 128 ? 5 : BN == 64 ? 4 : BN == 32 ? 3 : 2;    // quads = 2^shift
    const int lo = lines * rank / split, hi = lines * (rank + 1) / split;
    for (int i = threadIdx.x; i < (hi - lo) << shift; i += THREADS) {
        const int o = lo + (i >> shift), n = (i & (quads - 1)) * 4;
        const uint32_t at = part + (o * (quads * 4 + kPartPad) + n) * 4;
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < split) v[r] = tc::cluster_load4(tc::in_cta(at, r));
        float4 sum = v[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
            if (r < split) {
                sum.x += v[r].x;
                sum.y += v[r].y;
                sum.z += v[r].z;
                sum.w += v[r].w;
            }
        const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t p = pt * kB8Tile + (inner_p ? n + e : o), q = qt * BN + (inner_p ? o : n + e);
            if (p < a.p && q < a.q) store(a.out, a.type, p * a.sp + q * a.sq, out[e]);
        }
    }
    tc::cluster_sync();     // others may still read this CTA's sums
}

// Launch of a kernel with `smem` bytes of shared memory, `most` CTAs at most where no clusters share
// tiles; `ready` has a bit for each device whose limit is raised.
template <class Kernel>
cudaError_t launch_tiles(Kernel kernel, const ProductArgs &a, int threads, int smem, int64_t most, uint64_t *ready,
                         cudaStream_t stream) {
    int device;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (!(__atomic_load_n(ready, __ATOMIC_RELAXED) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(ready, bit, __ATOMIC_RELAXED);
    }
    const int64_t tiles = a.ptiles * a.qtiles;
    const int64_t ctas = a.split == 1 && tiles > most ? most : tiles * a.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
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

}  // namespace tn
