// Quantisation to 8 bits with a scale for each block of 128.
//
// A CTA reads one tile of 128 x 128 entries once, each of its eight warps 16 rows
// with four neighbouring entries a lane, and holds it in registers: the largest
// magnitudes along rows are one warp reduction a row, those along columns
// go from warp to warp through shared memory, and codes of the transposed
// matrix leave through a shared tile so that both layouts are written in whole
// lines.  Magnitudes are compared as integers (the bits of |x| have its order, and
// infinities and NaN are the largest of all).  Bound by memory.
#include <cuda_fp16.h>

#include <type_traits>

#include "block8.h"
#include "common.cuh"

namespace tn {

namespace {

constexpr int THREADS = 256;
constexpr int WARP_ROWS = kB8Tile / (THREADS / 32);     // 16

// The bits of a magnitude as fp32's.
template <typename T>
__device__ __forceinline__ uint32_t as_float(uint32_t raw) {
    if constexpr (sizeof(T) == 4) return raw;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return raw << 16;
    else return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(raw))));
}

// Neighbouring entries as they lie in memory, and their values.
template <typename T, int N>
struct Raw {
    static constexpr int kWords = N * sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p) {      // all at once
        if constexpr (kWords == 4) {
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(p));
            w[0] = u.x;
            w[1] = u.y;
            w[2] = u.z;
            w[3] = u.w;
        } else {
            const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(p));
            w[0] = u.x;
            w[1] = u.y;
        }
    }
    // `n` of them one by one, the others 0 (neighbours share lines: through the L1 cache)
    __device__ __forceinline__ void load(const T *p, int64_t stride, int64_t n) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= n) continue;
            if constexpr (sizeof(T) == 4) w[i] = *reinterpret_cast<const uint32_t *>(p + i * stride);
            else w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p + i * stride)) << (16 * (i % 2));
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i / 2]));
            return i % 2 ? f.y : f.x;
        }
    }
    __device__ __forceinline__ uint32_t size(int i) const { return __float_as_uint((*this)[i]) & 0x7fffffffu; }
    // The largest of all sizes, of 16-bit types as they lie (two at a time; their bits have the same order).
    __device__ __forceinline__ uint32_t largest_raw() const {
        uint32_t m = w[0] & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
#pragma unroll
        for (int i = 1; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) m = max(m, w[i] & 0x7fffffffu);
            else m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        }
        return sizeof(T) == 4 ? m : max(m & 0xffffu, m >> 16);
    }
    __device__ __forceinline__ uint32_t largest() const { return as_float<T>(largest_raw()); }
};

// The scale of a block whose largest magnitude has the bits `top`, and what
// entries are multiplied by (0 with a NaN or an infinity among them).
struct Scale {
    float s, inverse;
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    if (top > 0x7f7fffffu) return {__uint_as_float(0x7fc00000u), 0.f};
    if (top == 0) return {1.f, 1.f};
    // top = m 2^e with 1 <= m < 2, and 448 = 1.75 2^8
    int e = static_cast<int>(top >> 23) - 127 - ((top & 0x7fffffu) > 0x600000u ? 7 : 8);
    if (e < -126) e = -126;
    return {__uint_as_float(static_cast<uint32_t>(e + 127) << 23),
            __uint_as_float(static_cast<uint32_t>(127 - e) << 23)};
}

// Four codes in a word, the first in its lowest byte.  A scaled entry is exact
// (but where it underflows, far below the smallest code).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}
// a b, packed
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// Codes of four entries (0 where there is a NaN or an infinity in the block: 0 times those is not 0).
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d, float inverse) {
    const float2 by = make_float2(inverse, inverse), x = mul2(make_float2(a, b), by), y = mul2(make_float2(c, d), by);
    return inverse == 0.f ? 0 : codes4(x.x, x.y, y.x, y.y);
}

// Few rows in the layout of x alone, with a scale for 128 entries of a row: 16 bytes of
// a row a lane, four loads in flight, no shared memory.
template <typename T>
__global__ void __launch_bounds__(THREADS) quantize_rows_kernel(const QuantArgs a) {
    constexpr int N = 16 / sizeof(T), LANES = TN_BLOCK8 / N, LOADS = 4;
    const int lane = threadIdx.x % 32;
    pdl_trigger();
    pdl_wait();
    // items of 32 vectors: `per` of them a row (sides are below 2^31 - 1024)
    const uint32_t rows = static_cast<uint32_t>(a.rows);
    const int cols = static_cast<int>(a.cols), per = (cols + 32 * N - 1) / (32 * N);
    const int step = gridDim.x * (THREADS / 32), first = blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
    // (one division each; from item to item by sums, which stay below 2^32)
    const int step_rows = step / per, step_rest = step - step_rows * per;
    uint32_t at_row = first / per;
    int at = first - first / per * per;
    while (at_row < rows) {
        Raw<T, N> v[LOADS];
        uint32_t row[LOADS];
        int col[LOADS];
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            row[l] = at_row;
            col[l] = (at * 32 + lane) * N;
            at_row = min(at_row, rows) + step_rows;
            at += step_rest;
            if (at >= per) {
                at -= per;
                ++at_row;
            }
            v[l].clear();
            if (row[l] >= rows || col[l] >= cols) continue;
            const T *p = static_cast<const T *>(a.x) + row[l] * a.row_stride;
            if (a.vec && col[l] + N <= cols) v[l].load(p + col[l]);
            else v[l].load(p + col[l] * a.col_stride, a.col_stride, cols - col[l]);
        }
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            if (row[l] >= rows) break;              // the warp's
            uint32_t top = v[l].largest();
#pragma unroll
            for (int o = LANES / 2; o; o /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (col[l] >= cols) continue;
            const Scale s = scale_of(top);
            if (lane % LANES == 0) a.r.scales[row[l] * a.r.scale_stride + col[l] / TN_BLOCK8 * a.r.scale_block] = s.s;
            uint32_t w[N / 4];
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                w[i] = codes_of(v[l][4 * i], v[l][4 * i + 1], v[l][4 * i + 2], v[l][4 * i + 3], s.inverse);
            uint8_t *to = a.r.codes + row[l] * a.r.row_stride + col[l];
            if (col[l] + N <= cols) {
                if constexpr (N == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t *>(to) = w[0];
            } else {
#pragma unroll
                for (int i = 0; i < N - 1; ++i)
                    if (col[l] + i < cols) to[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
            }
        }
    }
}

template <typename T, bool SQUARE>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 4 ? 2 : 3) quantize_kernel(const QuantArgs a) {
    __shared__ __align__(16) uint4 turned[kB8Tile * (kB8Tile / 16)];
    __shared__ uint32_t tops[THREADS / 32][kB8Tile];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_trigger();
    pdl_wait();
    const int64_t rt = blockIdx.x / a.col_tiles, ct = blockIdx.x - rt * a.col_tiles;
    const int64_t r0 = rt * kB8Tile + warp * WARP_ROWS, c0 = ct * kB8Tile + lane * 4;
    const T *x = static_cast<const T *>(a.x) + r0 * a.row_stride + c0 * a.col_stride;

    const int here = static_cast<int>(a.rows - r0 < WARP_ROWS ? a.rows - r0 : WARP_ROWS);    // rows (none if below 0)
    const int left = static_cast<int>(a.cols - c0 < 4 ? a.cols - c0 : 4);                    // entries of a row

    Raw<T, 4> v[WARP_ROWS];
    if (a.vec && left == 4) {
#pragma unroll
        for (int i = 0; i < WARP_ROWS; ++i, x += a.row_stride) {
            if (i < here) v[i].load(x);
            else v[i].clear();
        }
    } else {
#pragma unroll
        for (int i = 0; i < WARP_ROWS; ++i, x += a.row_stride) v[i].load(x, a.col_stride, i < here ? left : 0);
    }

    uint32_t ctop[4] = {0, 0, 0, 0};
    if (SQUARE || a.c.codes) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < WARP_ROWS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) ctop[j] = max(ctop[j], v[i].size(j));
        } else {
            uint32_t pair[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < WARP_ROWS; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) pair[j] = __vmaxu2(pair[j], v[i].w[j] & 0x7fff7fffu);
#pragma unroll
            for (int j = 0; j < 4; ++j) ctop[j] = as_float<T>(pair[j / 2] >> (16 * (j % 2)) & 0xffffu);
        }
    }
    Scale tile = {1.f, 1.f};
    if (SQUARE) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(ctop[0], ctop[1]), max(ctop[2], ctop[3])));
        if (lane == 0) tops[0][warp] = top;
        __syncthreads();
        tile = scale_of(__reduce_max_sync(0xffffffffu, lane < THREADS / 32 ? tops[0][lane] : 0u));
        if (threadIdx.x == 0) {
            if (a.r.codes) a.r.scales[rt * a.r.scale_stride + ct * a.r.scale_block] = tile.s;
            if (a.c.codes) a.c.scales[ct * a.c.scale_stride + rt * a.c.scale_block] = tile.s;
        }
    }
    if (a.r.codes) {
        // (a row's scale is made by the lane of its number, and handed to the others)
        Scale own = tile;
        if (!SQUARE) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < WARP_ROWS; ++i) {
                const uint32_t row_top = __reduce_max_sync(0xffffffffu, v[i].largest_raw());
                top = lane == i ? row_top : top;
            }
            own = scale_of(as_float<T>(top));
            if (lane < here) a.r.scales[(r0 + lane) * a.r.scale_stride + ct * a.r.scale_block] = own.s;
        }
        uint8_t *to = a.r.codes + r0 * a.r.row_stride + c0;
#pragma unroll
        for (int i = 0; i < WARP_ROWS; ++i, to += a.r.row_stride) {
            const float inverse = SQUARE ? tile.inverse : __shfl_sync(0xffffffffu, own.inverse, i);
            const uint32_t w = codes_of(v[i][0], v[i][1], v[i][2], v[i][3], inverse);
            if (i >= here) continue;
            if (left == 4) {
                *reinterpret_cast<uint32_t *>(to) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (j < left) to[j] = static_cast<uint8_t>(w >> (8 * j));
            }
        }
    }
    if (a.c.codes) {
        Scale s[4] = {tile, tile, tile, tile};
        if (!SQUARE) {
            *reinterpret_cast<uint4 *>(&tops[warp][lane * 4]) = make_uint4(ctop[0], ctop[1], ctop[2], ctop[3]);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                const uint4 t = *reinterpret_cast<const uint4 *>(&tops[w][lane * 4]);
                ctop[0] = max(ctop[0], t.x);
                ctop[1] = max(ctop[1], t.y);
                ctop[2] = max(ctop[2], t.z);
                ctop[3] = max(ctop[3], t.w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = scale_of(ctop[j]);
                if (warp == 0 && c0 + j < a.cols) a.c.scales[(c0 + j) * a.c.scale_stride + rt * a.c.scale_block] = s[j].s;
            }
        }
        // Piece `warp` (16 codes) of column 4 lane + j lies at place warp ^ (lane % 8)
        // of the column's eight: eight lanes write, and later read, all banks.
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = codes_of(v[4 * i][j], v[4 * i + 1][j], v[4 * i + 2][j], v[4 * i + 3][j], s[j].inverse);
            turned[(lane * 4 + j) * 8 + (warp ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncthreads();
        const int piece = threadIdx.x % 8;
        const int64_t row = rt * kB8Tile + piece * 16;
#pragma unroll
        for (int i = 0; i < kB8Tile * 8 / THREADS; ++i) {
            const int c = i * (THREADS / 8) + threadIdx.x / 8;
            const int64_t col = ct * kB8Tile + c;
            if (col >= a.cols || row >= a.rows) continue;
            const uint4 w = turned[c * 8 + (piece ^ ((c >> 2) & 7))];
            uint8_t *to = a.c.codes + col * a.c.row_stride + row;
            if (row + 16 <= a.rows) {
                *reinterpret_cast<uint4 *>(to) = w;
            } else {
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 15; ++k)
                    if (row + k < a.rows) to[k] = static_cast<uint8_t>(u[k / 4] >> (8 * (k % 4)));
            }
        }
    }
}

template <typename T>
cudaError_t launch(const QuantArgs &a, bool square, cudaStream_t stream) {
    if (a.few) {
        constexpr int64_t kItem = 32 * 16 / sizeof(T);
        const int64_t warps = (a.rows * ((a.cols + kItem - 1) / kItem) + 3) / 4, most = 8 * kB8Sms;
        const int64_t ctas = (warps + THREADS / 32 - 1) / (THREADS / 32);
        return launch_pdl(quantize_rows_kernel<T>, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(THREADS),
                          0, stream, a);
    }
    const dim3 grid(static_cast<unsigned>(a.row_tiles * a.col_tiles));
    return square ? launch_pdl(quantize_kernel<T, true>, grid, dim3(THREADS), 0, stream, a)
                  : launch_pdl(quantize_kernel<T, false>, grid, dim3(THREADS), 0, stream, a);
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs &a, int32_t type, bool square, cudaStream_t stream) {
    switch (type) {
        case TN_TYPE_F32: return launch<float>(a, square, stream);
        case TN_TYPE_BF16: return launch<__nv_bfloat16>(a, square, stream);
        default: return launch<__half>(a, square, stream);
    }
}

}  // namespace tn
