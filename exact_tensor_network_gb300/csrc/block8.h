// Matrices in 8 bits with a scale for each block of 128: the kernels'
// arguments and their launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tn_block8.h"
#include "kernels.h"

namespace tn {

constexpr int kB8Sms = 152;
constexpr int kB8Tile = 128;            // rows and columns of a quantised tile; rows of a product's

// One quantised matrix as an output; codes is null where it is not asked for.
struct Block8Out {
    uint8_t *codes;
    float *scales;
    int64_t row_stride, scale_stride, scale_block;
};

struct QuantArgs {
    const void *x;
    int64_t rows, cols, row_stride, col_stride;
    Block8Out r, c;
    int64_t row_tiles, col_tiles;
    int32_t vec;        // neighbouring entries of a row may be read at once
    // Few rows in the layout of x alone: more CTAs than there are tiles.  By rows and by tiles: 16 x 4096 bf16 2.2
    // and 2.3 us, 128 rows 2.3 and 2.5, 512 rows 3.6 and 3.4, 4096 rows 10.4 and 7.7 (f32 17.9 and 10.0).
    int32_t few;
};

// What the products of a device have reported so far: counts that only grow, so that no report is lost to
// another, or to a thread that asks at the same time.
struct Block8Status {
    unsigned long long timeouts;    // CTAs that gave up waiting
    unsigned long long scales;      // threads that met a scale that should be a power of two
};

// A product by tiles of 128 rows of operand P by BN rows of operand Q:
// out[p sp + q sq].  P is the call's a (sp the output's stride, sq 1) or, where a
// has few rows, its b (sp 1).
struct ProductArgs {
    CUtensorMap tmP, tmQ;
    const float *scaleP, *scaleQ;
    int64_t strideP, strideQ;       // of the scales' rows
    int64_t blockP, blockQ;         // and blocks
    int32_t shiftP, shiftQ;         // log2 of the rows a scale stands for
    int64_t p, q;
    int64_t sp, sq;
    void *out;
    int32_t type;
    int32_t kbs;                    // blocks of k
    int32_t split;                  // CTAs of a cluster that share a tile's blocks
    int64_t ptiles, qtiles;
    Block8Status *status;
};

cudaError_t launch_quantize(const QuantArgs &a, int32_t type, bool square, cudaStream_t stream);
// bn: 256, 128, 64, 32 or 16; each: whether every row of Q has a scale of its own
cudaError_t launch_product(const ProductArgs &a, int bn, bool each, cudaStream_t stream);
// The same of scales that are powers of two; bn: 240, 128, 64, 32 or 16
cudaError_t launch_scaled(const ProductArgs &a, int bn, cudaStream_t stream);
// The current device's counts.
cudaError_t block8_status(Block8Status **p);

}  // namespace tn
