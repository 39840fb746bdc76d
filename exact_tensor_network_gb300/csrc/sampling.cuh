// Drawing outcomes from rows: weights, filters and draws.
//
// An outcome is a whole number, and near a border between two outcomes any
// rounding decides it: a sum of 10^5 weights in fp32 is wrong by some 2^-22, and one
// draw in ten of a broad row lies that near to a border.  So weights are computed as
// pairs of fp32 numbers (2^-44) and summed as 64-bit integers, in
// units of 2^-shift of the largest, the shift chosen by an estimate of the row's
// sum so that it uses 61 bits.  Integer sums need no order: histograms by
// shared-memory atomics, partial sums of CTAs and of warps are all exact.
//
// Rows of up to 8 KiB stay in the registers of a warp or a CTA, a few longer ones (up to
// 32768 entries) in those of a cluster; all others are cut into segments and read twice, or three
// times where they are filtered.
#pragma once

#include "outcomes.cuh"
#include "sampling.h"

namespace tn {

// 2^(i/32) and 2^(j/1024), each as the sum of two fp32 numbers
static __device__ const float2 kCoarse[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9e0p+0f, -0x1.5c0424p-25f}, {0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.6247ecp+0f, -0x1.f8b550p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246eb0p-26f},
};
static __device__ const float2 kFine[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.002c60p+0f, 0x1.78ba34p-26f}, {0x1.0058c8p+0f, 0x1.b68702p-26f},
    {0x1.008538p+0f, 0x1.7d77c2p-27f}, {0x1.00b1b0p+0f, -0x1.6950d0p-26f}, {0x1.00de2ep+0f, 0x1.a1dc1ep-25f},
    {0x1.010ab6p+0f, -0x1.34d0bcp-26f}, {0x1.013744p+0f, 0x1.326d6ep-26f}, {0x1.0163dap+0f, 0x1.3f6666p-25f},
    {0x1.019078p+0f, 0x1.5ad434p-25f}, {0x1.01bd1ep+0f, 0x1.dc5c2ep-26f}, {0x1.01e9ccp+0f, -0x1.eec114p-32f},
    {0x1.021682p+0f, -0x1.789fb0p-25f}, {0x1.02433ep+0f, 0x1.252dd6p-26f}, {0x1.027004p+0f, -0x1.df89dep-25f},
    {0x1.029cd0p+0f, -0x1.98a37ep-26f}, {0x1.02c9a4p+0f, -0x1.887fa0p-28f}, {0x1.02f680p+0f, -0x1.626868p-30f},
    {0x1.032364p+0f, -0x1.5ea7ecp-27f}, {0x1.035050p+0f, -0x1.1421f2p-25f}, {0x1.037d42p+0f, 0x1.c2377ap-25f},
    {0x1.03aa3ep+0f, 0x1.70aafep-28f}, {0x1.03d742p+0f, -0x1.cdd4aep-25f}, {0x1.04044cp+0f, -0x1.76954ap-28f},
    {0x1.04315ep+0f, 0x1.0dcff0p-25f}, {0x1.045e78p+0f, 0x1.eac818p-25f}, {0x1.048b9cp+0f, -0x1.9534c4p-25f},
    {0x1.04b8c6p+0f, -0x1.6f70bcp-25f}, {0x1.04e5f8p+0f, -0x1.a1356ap-25f}, {0x1.051330p+0f, 0x1.d83408p-25f},
    {0x1.054072p+0f, 0x1.ff05d8p-26f}, {0x1.056dbcp+0f, -0x1.448794p-28f},
};

// 2^(k/1024), k = 0 .. 1023, in shared memory: the products of the two, what a pair adds to its
// larger number kRoots places behind that.
constexpr int kRoots = 1024;
template <int NT>
__device__ __forceinline__ void make_roots(float *roots) {
    for (int k = threadIdx.x; k < kRoots; k += NT) {
        const float2 c = kCoarse[k >> 5], f = kFine[k & 31];
        const float h = c.x * f.x, l = fmaf(c.x, f.x, -h) + fmaf(c.x, f.y, c.y * f.x), x = h + l;
        roots[k] = x;
        roots[kRoots + k] = (h - x) + l;
    }
}

// For c = 1 + (i + 1/2) / 128: a number of eight bits that is near 1 / c, and the logarithm of its inverse, to
// 16 bits and what is left.
static __device__ const float4 kLogs[128] = {
    {0x1.fep-1f, 0x1.01p-8f, -0x1.fea9aap-18f, 0.f}, {0x1.fap-1f, 0x1.828p-7f, -0x1.dbae3cp-18f, 0.f},
    {0x1.f6p-1f, 0x1.434p-6f, -0x1.56da68p-18f, 0.f}, {0x1.f2p-1f, 0x1.c64p-6f, -0x1.689f5ap-21f, 0.f},
    {0x1.eep-1f, 0x1.252p-5f, 0x1.e65f1ap-18f, 0.f}, {0x1.eap-1f, 0x1.67cp-5f, 0x1.29e5aap-18f, 0.f},
    {0x1.e8p-1f, 0x1.894p-5f, 0x1.54294p-18f, 0.f}, {0x1.e4p-1f, 0x1.cccp-5f, -0x1.186444p-18f, 0.f},
    {0x1.ep-1f, 0x1.086p-4f, -0x1.9d2988p-18f, 0.f}, {0x1.dcp-1f, 0x1.2aap-4f, 0x1.2911c6p-22f, 0.f},
    {0x1.dap-1f, 0x1.3bep-4f, -0x1.4b05c2p-21f, 0.f}, {0x1.d6p-1f, 0x1.5e9p-4f, 0x1.69365ep-18f, 0.f},
    {0x1.d2p-1f, 0x1.819p-4f, 0x1.f8bd04p-18f, 0.f}, {0x1.dp-1f, 0x1.933p-4f, 0x1.797566p-18f, 0.f},
    {0x1.ccp-1f, 0x1.b6bp-4f, -0x1.bb9296p-19f, 0.f}, {0x1.c8p-1f, 0x1.da7p-4f, 0x1.3b1c22p-19f, 0.f},
    {0x1.c6p-1f, 0x1.ec7p-4f, 0x1.cc185p-19f, 0.f}, {0x1.c2p-1f, 0x1.0858p-3f, 0x1.8b59e4p-19f, 0.f},
    {0x1.cp-1f, 0x1.1178p-3f, 0x1.d044fcp-20f, 0.f}, {0x1.bcp-1f, 0x1.23d8p-3f, -0x1.dab6c8p-20f, 0.f},
    {0x1.bap-1f, 0x1.2d18p-3f, -0x1.ef3798p-19f, 0.f}, {0x1.b6p-1f, 0x1.3fb8p-3f, -0x1.d2d336p-18f, 0.f},
    {0x1.b4p-1f, 0x1.491p-3f, 0x1.ec199ep-18f, 0.f}, {0x1.bp-1f, 0x1.5bf8p-3f, -0x1.fca55ep-18f, 0.f},
    {0x1.aep-1f, 0x1.6578p-3f, -0x1.8a0bap-18f, 0.f}, {0x1.aap-1f, 0x1.7898p-3f, 0x1.b0a88ap-20f, 0.f},
    {0x1.a8p-1f, 0x1.824p-3f, -0x1.f4d572p-18f, 0.f}, {0x1.a6p-1f, 0x1.8be8p-3f, 0x1.7f59c8p-18f, 0.f},
    {0x1.a2p-1f, 0x1.9f7p-3f, -0x1.dfc7bcp-18f, 0.f}, {0x1.ap-1f, 0x1.a94p-3f, -0x1.2c3752p-19f, 0.f},
    {0x1.9ep-1f, 0x1.b32p-3f, -0x1.3d4522p-18f, 0.f}, {0x1.9ap-1f, 0x1.c7p-3f, -0x1.0e43fcp-21f, 0.f},
    {0x1.98p-1f, 0x1.d1p-3f, 0x1.bf932ap-18f, 0.f}, {0x1.96p-1f, 0x1.db1p-3f, 0x1.ed86a4p-18f, 0.f},
    {0x1.94p-1f, 0x1.e53p-3f, 0x1.dffce2p-20f, 0.f}, {0x1.9p-1f, 0x1.f99p-3f, 0x1.c6cb3cp-19f, 0.f},
    {0x1.8ep-1f, 0x1.01ecp-2f, -0x1.1a9d94p-18f, 0.f}, {0x1.8cp-1f, 0x1.0714p-2f, -0x1.e7ecaap-20f, 0.f},
    {0x1.8ap-1f, 0x1.0c44p-2f, -0x1.2989eap-18f, 0.f}, {0x1.88p-1f, 0x1.1178p-2f, 0x1.d044fcp-19f, 0.f},
    {0x1.84p-1f, 0x1.1bf8p-2f, 0x1.9635a6p-18f, 0.f}, {0x1.82p-1f, 0x1.2144p-2f, 0x1.5b43aep-20f, 0.f},
    {0x1.8p-1f, 0x1.2698p-2f, -0x1.deecb2p-18f, 0.f}, {0x1.7ep-1f, 0x1.2bfp-2f, -0x1.f0646ep-19f, 0.f},
    {0x1.7cp-1f, 0x1.315p-2f, -0x1.c3c594p-19f, 0.f}, {0x1.7ap-1f, 0x1.36b8p-2f, -0x1.88941ep-18f, 0.f},
    {0x1.78p-1f, 0x1.3c24p-2f, 0x1.277334p-18f, 0.f}, {0x1.76p-1f, 0x1.419cp-2f, -0x1.7b8542p-19f, 0.f},
    {0x1.74p-1f, 0x1.4718p-2f, 0x1.b84e38p-19f, 0.f}, {0x1.72p-1f, 0x1.4cap-2f, -0x1.f61e8ep-18f, 0.f},
    {0x1.7p-1f, 0x1.522cp-2f, -0x1.1f8c76p-18f, 0.f}, {0x1.6ep-1f, 0x1.57cp-2f, -0x1.1586e6p-19f, 0.f},
    {0x1.6cp-1f, 0x1.5d5cp-2f, -0x1.10535p-21f, 0.f}, {0x1.6ap-1f, 0x1.63p-2f, 0x1.859d56p-21f, 0.f},
    {0x1.68p-1f, 0x1.68acp-2f, 0x1.07d38ep-19f, 0.f}, {0x1.66p-1f, 0x1.6e6p-2f, 0x1.dcd5e4p-19f, 0.f},
    {0x1.64p-1f, 0x1.741cp-2f, 0x1.876c68p-18f, 0.f}, {0x1.62p-1f, 0x1.79e4p-2f, -0x1.99783p-18f, 0.f},
    {0x1.6p-1f, 0x1.7fbp-2f, -0x1.7109fap-20f, 0.f}, {0x1.5ep-1f, 0x1.8584p-2f, 0x1.5776dcp-18f, 0.f},
    {0x1.5cp-1f, 0x1.8b64p-2f, -0x1.95dd34p-20f, 0.f}, {0x1.5ap-1f, 0x1.914cp-2f, -0x1.79ca4p-18f, 0.f},
    {0x1.58p-1f, 0x1.973cp-2f, -0x1.cbcecap-18f, 0.f}, {0x1.56p-1f, 0x1.9d34p-2f, -0x1.415ea2p-18f, 0.f},
    {0x1.54p-1f, 0x1.a334p-2f, 0x1.00893ep-20f, 0.f}, {0x1.52p-1f, 0x1.a94p-2f, -0x1.2c3752p-18f, 0.f},
    {0x1.5p-1f, 0x1.af54p-2f, -0x1.6adb74p-18f, 0.f}, {0x1.5p-1f, 0x1.af54p-2f, -0x1.6adb74p-18f, 0.f},
    {0x1.4ep-1f, 0x1.b57p-2f, -0x1.7eee76p-20f, 0.f}, {0x1.4cp-1f, 0x1.bb98p-2f, -0x1.ee47f2p-18f, 0.f},
    {0x1.4ap-1f, 0x1.c1c8p-2f, -0x1.f96c06p-18f, 0.f}, {0x1.48p-1f, 0x1.c8p-2f, -0x1.8e2eaap-20f, 0.f},
    {0x1.46p-1f, 0x1.ce44p-2f, -0x1.0e7f9cp-18f, 0.f}, {0x1.46p-1f, 0x1.ce44p-2f, -0x1.0e7f9cp-18f, 0.f},
    {0x1.44p-1f, 0x1.d49p-2f, 0x1.236f7ep-21f, 0.f}, {0x1.42p-1f, 0x1.dae8p-2f, -0x1.56f66ep-19f, 0.f},
    {0x1.4p-1f, 0x1.e148p-2f, 0x1.4344e4p-19f, 0.f}, {0x1.3ep-1f, 0x1.e7b4p-2f, 0x1.61eed6p-21f, 0.f},
    {0x1.3ep-1f, 0x1.e7b4p-2f, 0x1.61eed6p-21f, 0.f}, {0x1.3cp-1f, 0x1.ee2cp-2f, -0x1.ea94bep-18f, 0.f},
    {0x1.3ap-1f, 0x1.f4acp-2f, -0x1.811fcep-18f, 0.f}, {0x1.38p-1f, 0x1.fb34p-2f, 0x1.8af7a4p-18f, 0.f},
    {0x1.38p-1f, 0x1.fb34p-2f, 0x1.8af7a4p-18f, 0.f}, {0x1.36p-1f, 0x1.00e6p-1f, -0x1.46937ep-19f, 0.f},
    {0x1.34p-1f, 0x1.0436p-1f, 0x1.7cec08p-22f, 0.f}, {0x1.32p-1f, 0x1.078cp-1f, -0x1.f59876p-22f, 0.f},
    {0x1.32p-1f, 0x1.078cp-1f, -0x1.f59876p-22f, 0.f}, {0x1.3p-1f, 0x1.0ae8p-1f, -0x1.23a5f6p-18f, 0.f},
    {0x1.2ep-1f, 0x1.0e48p-1f, 0x1.30c23ap-18f, 0.f}, {0x1.2ep-1f, 0x1.0e48p-1f, 0x1.30c23ap-18f, 0.f},
    {0x1.2cp-1f, 0x1.11bp-1f, -0x1.f70e2ap-19f, 0.f}, {0x1.2ap-1f, 0x1.151cp-1f, 0x1.fb794cp-20f, 0.f},
    {0x1.2ap-1f, 0x1.151cp-1f, 0x1.fb794cp-20f, 0.f}, {0x1.28p-1f, 0x1.188ep-1f, 0x1.c81e48p-18f, 0.f},
    {0x1.26p-1f, 0x1.1c08p-1f, -0x1.ed9468p-19f, 0.f}, {0x1.26p-1f, 0x1.1c08p-1f, -0x1.ed9468p-19f, 0.f},
    {0x1.24p-1f, 0x1.1f86p-1f, 0x1.afe30cp-20f, 0.f}, {0x1.22p-1f, 0x1.230cp-1f, -0x1.e4e828p-18f, 0.f},
    {0x1.22p-1f, 0x1.230cp-1f, -0x1.e4e828p-18f, 0.f}, {0x1.2p-1f, 0x1.2696p-1f, 0x1.089a6ep-20f, 0.f},
    {0x1.1ep-1f, 0x1.2a28p-1f, -0x1.e4bc5p-19f, 0.f}, {0x1.1ep-1f, 0x1.2a28p-1f, -0x1.e4bc5p-19f, 0.f},
    {0x1.1cp-1f, 0x1.2dcp-1f, -0x1.5509e4p-18f, 0.f}, {0x1.1cp-1f, 0x1.2dcp-1f, -0x1.5509e4p-18f, 0.f},
    {0x1.1ap-1f, 0x1.315ep-1f, -0x1.6ef2fep-19f, 0.f}, {0x1.18p-1f, 0x1.3502p-1f, 0x1.15b3b2p-18f, 0.f},
    {0x1.18p-1f, 0x1.3502p-1f, 0x1.15b3b2p-18f, 0.f}, {0x1.16p-1f, 0x1.38aep-1f, 0x1.0b8cbcp-20f, 0.f},
    {0x1.16p-1f, 0x1.38aep-1f, 0x1.0b8cbcp-20f, 0.f}, {0x1.14p-1f, 0x1.3c6p-1f, 0x1.0186d8p-18f, 0.f},
    {0x1.12p-1f, 0x1.401ap-1f, -0x1.ef6d1ap-20f, 0.f}, {0x1.12p-1f, 0x1.401ap-1f, -0x1.ef6d1ap-20f, 0.f},
    {0x1.1p-1f, 0x1.43dap-1f, -0x1.a0db88p-26f, 0.f}, {0x1.1p-1f, 0x1.43dap-1f, -0x1.a0db88p-26f, 0.f},
    {0x1.0ep-1f, 0x1.47a2p-1f, -0x1.5b02ecp-18f, 0.f}, {0x1.0ep-1f, 0x1.47a2p-1f, -0x1.5b02ecp-18f, 0.f},
    {0x1.0cp-1f, 0x1.4b7p-1f, -0x1.48347ap-20f, 0.f}, {0x1.0ap-1f, 0x1.4f46p-1f, -0x1.5f296cp-19f, 0.f},
    {0x1.0ap-1f, 0x1.4f46p-1f, -0x1.5f296cp-19f, 0.f}, {0x1.08p-1f, 0x1.5322p-1f, 0x1.c4d0dp-18f, 0.f},
    {0x1.08p-1f, 0x1.5322p-1f, 0x1.c4d0dp-18f, 0.f}, {0x1.06p-1f, 0x1.5708p-1f, -0x1.76511cp-19f, 0.f},
    {0x1.06p-1f, 0x1.5708p-1f, -0x1.76511cp-19f, 0.f}, {0x1.04p-1f, 0x1.5af4p-1f, 0x1.70d928p-23f, 0.f},
    {0x1.04p-1f, 0x1.5af4p-1f, 0x1.70d928p-23f, 0.f}, {0x1.02p-1f, 0x1.5ee8p-1f, 0x1.55120cp-20f, 0.f},
    {0x1.02p-1f, 0x1.5ee8p-1f, 0x1.55120cp-20f, 0.f}, {0x1p-1f, 0x1.62e4p-1f, 0x1.7f7d1cp-20f, 0.f},
};
constexpr float kLn2Hi = 0x1.62e4p-1f, kLn2Lo = 0x1.7f7d1cp-20f;    // ln 2 likewise

// A difference beyond fp32 counts as this one; from this ch on it weighs nothing (2^-1024), as absent logits
// at -inf do then.
constexpr float kFarthest = -3.402823466e38f, kRareScale = 0x1p-118f;

// What a row's weights are computed from.
struct RowPlan {
    float m;            // largest order value
    float b;            // beta, as large as weights need it
    float ch;           // b log2(e), for estimates
    float low;          // lower order values weigh as much (next to nothing)
    // Weights are relative to m's (far), or to a number near it: e^(origin ln 2 / 1024), or of
    // amplitudes (2^n e^g)^beta with n + g = origin, n whole
    float origin;
    uint32_t first;     // what a rounded exponent's bits less this are the power of
    bool far;
    float down;         // amplitudes at beta = 1: 2^-x with weights up to 2^x
    int shift;          // a weight of 1 is 2^shift
    int down_log;       // x
    float beta;
    int state;          // kDraw, or how the row ends
    bool greedy;
    bool unit;          // beta is 1
    uint64_t bound;     // entries of at least this rank are left
};
enum { kDraw = 0, kEmpty = 1, kUndefined = 2 };

// Rank of an entry: by order value, then by index (lowest first); absent ones have
// none.  Any present entry's is at least kPresent.
constexpr uint64_t kPresent = 1ull << 32;
template <int TYPE>
__device__ __forceinline__ uint64_t rank_of(float v, int64_t e) {
    const uint32_t k = order_key<TYPE>(v);
    return k ? static_cast<uint64_t>(k) << 32 | (0xffffffffu - static_cast<uint32_t>(e)) : 0;
}

// ln 2 / 1024 as a pair, and 1.5 2^23, which rounds what it is added to.
constexpr float kStepHi = 0x1.62e43p-11f, kStepLo = -0x1.05c61p-39f, kMagic = 12582912.f;

// w + wl in units of 2^-44 (conversions of fp32 to 64-bit integers would run on the fp64 pipe): w,
// below 2, to 2^-22 from the mantissa of w + 2, what is left of it with wl from that of a sum
// with 1.5 2^23 (it is less than 2^-22); then times 2^(k / 1024 + shift).
__device__ __forceinline__ uint64_t whole_weight(float w, float wl, int k, int shift) {
    const float up = __fadd_rn(w, 2.f), rest = (w - __fadd_rn(up, -2.f)) + wl;
    const int low = static_cast<int>(__float_as_uint(fmaf(rest, 0x1p44f, kMagic)) - __float_as_uint(kMagic));
    const int64_t n = static_cast<int64_t>(static_cast<int>(__float_as_uint(up) - 0x40000000u)) * (1 << 22) + low;
    const int x = (k >> 10) + shift - 44;
    const uint64_t whole = x >= 0 ? static_cast<uint64_t>(n) << x : x > -64 ? static_cast<uint64_t>(n) >> -x : 0;
    return whole > 0 ? whole : 1;
}

// The weights of two present entries, e^(b v) relative to the row's origin, to some 2^-44: 2^(k / 1024)
// e^r from a table and the exponential series, |r| <= ln 2 / 2048.  As unnormalised pairs w + wl without
// the whole part of k / 1024, and k.  Packed fp32 (a pair's operations cost what two single ones do);
// the origin on the grid of the table leaves no difference v - m to be taken, which rows whose |b m| is
// large need (`far`: b v would be known to fewer bits).
struct Powers {
    float2 w, wl;
    uint32_t k0, k1;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }
__device__ __forceinline__ Powers powers_of(const RowPlan &p, const float *roots, float2 v) {
    v = make_float2(fmaxf(v.x, p.low), fmaxf(v.y, p.low));
    float2 h, l;                                            // b v (or b (v - m)) as a pair
    if (p.far) {
        const float2 d = add2(v, both(-p.m)), b = sub2(d, v);
        const float2 e = add2(sub2(v, sub2(d, b)), sub2(both(-p.m), b));    // d + e is the exact difference
        h = mul2(d, both(p.b));
        l = fma2(e, both(p.b), fma2(d, both(p.b), mul2(d, both(-p.b))));
    } else {
        h = mul2(v, both(p.b));
        l = fma2(v, both(p.b), mul2(v, both(-p.b)));
    }
    const float2 km = fma2(h, both(0x1.71547652b82fep+10f), both(kMagic)), kf = add2(km, both(-kMagic));
    const uint32_t k0 = __float_as_uint(km.x) - p.first, k1 = __float_as_uint(km.y) - p.first;
    const float2 q = fma2(kf, both(-kStepHi), h), ql = fma2(kf, both(-kStepLo), l);     // (the first exact)
    const float2 r = add2(q, ql), rl = add2(sub2(q, r), ql);
    const float2 lo = fma2(mul2(r, r), fma2(r, both(1.f / 6), both(0.5f)), rl);     // e^r - 1 = r + lo
    const uint32_t i0 = k0 & (kRoots - 1), i1 = k1 & (kRoots - 1);
    const float2 x = make_float2(roots[i0], roots[i1]), y = make_float2(roots[i0 + kRoots], roots[i1 + kRoots]);
    const float2 a = mul2(x, r), al = fma2(x, r, mul2(x, mul2(r, both(-1.f)))), w = add2(x, a);
    return {w, add2(add2(sub2(x, w), a), add2(al, fma2(x, lo, fma2(y, r, y)))), k0, k1};
}

// A number of 0 <= v < 4 in units of 2^-shift, the same way.
__device__ __forceinline__ uint64_t in_units(float v, int shift) {
    const uint32_t b = __float_as_uint(v);
    const uint64_t n = (b & 0x7fffffu) | 0x800000u;
    const int x = static_cast<int>(b >> 23) - 150 + shift;
    return x >= 0 ? n << x : x > -64 ? n >> -x : 0;
}

// Out of line, as what follows is wherever a kernel's steady loop does not need it: a
// kernel's first pass through its code costs more than what it computes there.
//
// An amplitude's weight at beta != 1, to some 2^-40 (2^-46 on average): ln v = e ln 2 - ln t + ln(1 + r) with
// r = t c - 1 exact, t from the table; the parts of 16 bits add up exactly, the series' first two
// terms are kept as a pair.  148 x 226333 amplitudes, with logarithms and exponentials in 64 bits 4.1 ms.
static __device__ __noinline__ uint64_t weight_power(float v, float b, float origin, int shift, const float *roots) {
    const float up = v < 0x1p-126f ? 0x1p24f : 1.f;
    const uint32_t u = __float_as_uint(v * up);
    const float e = static_cast<float>(static_cast<int>(u >> 23) - (up > 1.f ? 151 : 127));
    const float c = __uint_as_float((u & 0x7fffffu) | 0x3f800000u), n = floorf(origin);
    const float4 t = kLogs[u >> 16 & 127];
    const float r = fmaf(c, t.x, -1.f), s = r * r;
    const float d = fmaf(e - n, kLn2Hi, t.y - (origin - n));
    const float ph = fmaf(-0.5f, s, r);
    const float cube = r * s * fmaf(r, fmaf(r, fmaf(r, fmaf(r, 1.f / 7, -1.f / 6), 0.2f), -0.25f), 1.f / 3);
    const float pl = fmaf(-0.5f, s, r - ph) + (fmaf(e - n, kLn2Lo, t.z) + fmaf(-0.5f, fmaf(r, r, -s), cube));
    const float x = d + ph, y = x - d, xl = ((d - (x - y)) + (ph - y)) + pl;
    const float h = x * b, l = fmaf(xl, b, fmaf(x, b, -h));
    if (!(h > -62.f)) return 1;
    const float km = fmaf(h, 0x1.71547652b82fep+10f, kMagic), kf = __fadd_rn(km, -kMagic);
    const int k = static_cast<int>(__float_as_uint(km) - __float_as_uint(kMagic));
    const float q = fmaf(kf, -kStepHi, h), ql = fmaf(kf, -kStepLo, l), a = q + ql;
    const float lo = fmaf(a * a, fmaf(a, 1.f / 6, 0.5f), (q - a) + ql);
    const float g = roots[k & (kRoots - 1)], gl = roots[(k & (kRoots - 1)) + kRoots];
    const float w = g * a, wl = fmaf(g, a, -w), w0 = g + w;
    const float wm = ((g - w0) + w) + (wl + fmaf(g, lo, fmaf(gl, a, gl))), whole = w0 + wm;
    return whole_weight(whole, (w0 - whole) + wm, k, shift);
}
// In 64 bits, at a beta that makes more of the logarithm's error.
static __device__ __noinline__ uint64_t weight_far_power(float v, float m, float beta, int shift) {
    const double x = static_cast<double>(beta) * log(static_cast<double>(v) / m);
    return x < -60.0 ? 1 : static_cast<uint64_t>(__double2ll_rn(ldexp(exp(x), shift)));
}

template <int TYPE>
__device__ __forceinline__ uint64_t weight(const RowPlan &p, const float *roots, float v) {
    if constexpr (Entry<TYPE>::kReal) {
        const Powers o = powers_of(p, roots, both(v));
        const float w = o.w.x + o.wl.x;
        return whole_weight(w, (o.w.x - w) + o.wl.x, static_cast<int>(o.k0), p.shift);
    } else {
        const uint64_t n = p.unit  ? in_units(v * p.down, p.shift)
                           : p.far ? weight_far_power(v, p.m, p.beta, p.shift)
                                   : weight_power(v, p.b, p.origin, p.shift, roots);
        return n > 0 ? n : 1;
    }
}
template <int TYPE>
__device__ __noinline__ uint64_t weight_once(const RowPlan &p, const float *roots, float v) {
    return weight<TYPE>(p, roots, v);
}
// Sums of weights as pairs of fp32 numbers, the largest weight being 1: what several
// entries next to each other cost less by than by integers one by one.  Two entries at a time,
// in packed arithmetic, into two sums.
struct PairSum {
    // (from the first on larger than what is added, so that a difference's error is one itself)
    static constexpr float kFrom = 4.f;
    float2 hi = {kFrom, kFrom}, lo = {0.f, 0.f};
    __device__ __forceinline__ void add(float2 h, float2 l) {
        const float2 x = add2(hi, h);
        lo = add2(lo, add2(sub2(h, sub2(x, hi)), l));
        hi = x;
    }
    __device__ __forceinline__ uint64_t units(int shift) const {
        const float u0 = hi.x - kFrom, u1 = hi.y - kFrom, x = u0 + u1, b = x - u0;
        const float y = ((u0 - (x - b)) + (u1 - b)) + (lo.x + lo.y);
        const float h = x + y, l = (x - h) + y;
        const uint64_t u = in_units(h, shift), v = in_units(fabsf(l), shift);
        return h > 0.f ? (l < 0.f ? u - v : l > 0.f ? u + v : u) : 0;
    }
};
// Of two entries, as pairs; 0 where they do not count.
struct Weights {
    float2 hi, lo;
};
__device__ __forceinline__ Weights weight_pairs(const RowPlan &p, const float *roots, float v0, float v1, bool counts0,
                                                bool counts1) {
    const Powers o = powers_of(p, roots, make_float2(counts0 ? v0 : p.m, counts1 ? v1 : p.m));
    const float2 unit = make_float2(counts0 ? __uint_as_float((o.k0 & ~(kRoots - 1u)) * (1u << 13) + 0x3f800000u) : 0.f,
                                    counts1 ? __uint_as_float((o.k1 & ~(kRoots - 1u)) * (1u << 13) + 0x3f800000u) : 0.f);
    return {mul2(o.w, unit), mul2(o.wl, unit)};
}
// The weights of two present entries, 1 at least (so that a draw of u = 0 finds the first entry left).
template <int TYPE>
__device__ __forceinline__ void two_weights(const RowPlan &p, const float *roots, float v0, float v1, uint64_t &w0,
                                            uint64_t &w1) {
    if constexpr (Entry<TYPE>::kReal) {
        const Powers o = powers_of(p, roots, make_float2(v0, v1));
        const float2 w = add2(o.w, o.wl), wl = add2(sub2(o.w, w), o.wl);    // (t's low part makes o.wl up to 2^-19)
        w0 = whole_weight(w.x, wl.x, static_cast<int>(o.k0), p.shift);
        w1 = whole_weight(w.y, wl.y, static_cast<int>(o.k1), p.shift);
    } else {
        w0 = weight<TYPE>(p, roots, v0);
        w1 = weight<TYPE>(p, roots, v1);
    }
}

// log2 of an amplitude's order value, which may be subnormal (lg2 takes those for 0; at a high temperature
// they are not).
__device__ __forceinline__ float log2_of(float v) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
// The estimate of an amplitude's weight relative to the larger m's, as a power of two.  Logarithms in fp32 are known to
// 2^-18 only; where beta makes much of that, by ln(v / m) <= (v - m) / m, which is exact for what is close to m (what
// is not weighs next to nothing there).  ch is beta log2(e).
__device__ __forceinline__ float rough_power(float beta, float ch, float v, float m) {
    return beta > 64.f ? ch * ((v - m) / m) : beta * (log2_of(v) - log2_of(m));
}

// The same in fp32, relative to the largest: for an estimate of the sum.  It must not be far too small, or
// the sums would overflow.
template <int TYPE>
__device__ __forceinline__ float rough_weight(const RowPlan &p, float v) {
    if constexpr (Entry<TYPE>::kReal) return ex2(fmaxf(v - p.m, kFarthest) * p.ch);
    else if (p.unit) return v * p.down;
    else return ex2(rough_power(p.beta, p.ch, v, p.m));
}

template <int TYPE>
__device__ __forceinline__ void vector_values(const Row<TYPE> &r, int64_t j, float (&v)[Entry<TYPE>::E]) {
    using En = Entry<TYPE>;
    const int64_t e0 = j * En::E - r.head;
    if (r.inside(e0)) {
        uint4 q = r.raw(e0);
        if (r.m) En::blank(q, row_keep<TYPE>(r, e0));
        En::values(q, v);
    } else {
        const Values<En::E> o = row_vector<TYPE>(r, j);
#pragma unroll
        for (int i = 0; i < En::E; ++i) v[i] = o.v[i];
    }
}

// f(order values, vector, n) of vectors first, first + stride, .. below hi, N at a time with
// their loads in flight together; `edge` is the first vector behind those that the
// caller's threads read at a time (N stride further than the first of them), so that
// they all take the same way.
template <int TYPE, int N, class F>
__device__ __forceinline__ void vectors_at(const Row<TYPE> &r, int64_t in_lo, int64_t in_hi, int64_t from, int64_t edge,
                                           int64_t first, int stride, int64_t hi, F f) {
    using En = Entry<TYPE>;
    if (from >= in_lo && edge <= in_hi && edge <= hi) {
        uint4 q[N];
        const uint4 *p = r.vectors() + first;
#pragma unroll
        for (int n = 0; n < N; ++n) q[n] = __ldcg(p + n * stride);
        if (r.m) {
            typename Row<TYPE>::Keep keep[N];
#pragma unroll
            for (int n = 0; n < N; ++n) keep[n] = r.keep((first + n * stride) * En::E - r.head);
#pragma unroll
            for (int n = 0; n < N; ++n) En::blank(q[n], keep[n]);
        }
        if constexpr (En::E == 2) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float v[En::E];
                En::values(q[n], v);
                f(v, first + n * stride, n);
            }
        } else {
            // one copy of f's code
#pragma unroll 1
            for (int n = 0; n < N; ++n) {
                uint4 x = q[0];
#pragma unroll
                for (int i = 1; i < N; ++i)
                    if (n == i) x = q[i];
                float v[En::E];
                En::values(x, v);
                f(v, first + n * stride, n);
            }
        }
    } else {
#pragma unroll 1
        for (int n = 0; n < N; ++n) {
            const int64_t j = first + n * stride;
            if (j >= hi) break;
            float v[En::E];
            vector_values<TYPE>(r, j, v);
            f(v, j, n);
        }
    }
}
// The same of all vectors lo .. hi - 1, by NT threads of which this is t.
template <int TYPE, int NT, int N, class F>
__device__ __forceinline__ void each_vector(const Row<TYPE> &r, int64_t lo, int64_t hi, int t, F f) {
    int64_t in_lo, in_hi;
    r.inside_range(in_lo, in_hi);
    for (int64_t from = lo; from < hi; from += N * NT)
        vectors_at<TYPE, N>(r, in_lo, in_hi, from, from + N * NT, from + t, NT, hi, f);
}

__device__ __forceinline__ uint64_t shfl_up(uint64_t x, int o) {
    return __shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(x), o);
}
__device__ __forceinline__ uint64_t shfl_from(uint64_t x, int lane) {
    return __shfl_sync(0xffffffffu, static_cast<unsigned long long>(x), lane);
}
// (parts of 27 bits, whose sums over 32 lanes fit into 32)
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
    constexpr uint32_t kPart = (1u << 27) - 1u;
    const uint32_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x) & kPart);
    const uint32_t b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 27) & kPart);
    const uint32_t c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 54));
    return a + (static_cast<uint64_t>(b) << 27) + (static_cast<uint64_t>(c) << 54);
}
// inclusive
__device__ __forceinline__ uint64_t warp_scan(uint64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = shfl_up(x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// floor(u z) and ceil(u z) of a number 0 <= u <= 1, exact.
static __device__ __noinline__ uint64_t share(double u, uint64_t z, bool up) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(u));
    const int e = static_cast<int>(b >> 52 & 0x7ff);
    const uint64_t m = (b & ((1ull << 52) - 1)) | (e ? 1ull << 52 : 0);
    const int right = 1075 - (e ? e : 1);                   // u = m 2^-right
    const unsigned __int128 p = static_cast<unsigned __int128>(m) * z;
    if (right >= 128) return up && p != 0;
    uint64_t q = static_cast<uint64_t>(p >> right);
    if (up && (p & ((static_cast<unsigned __int128>(1) << right) - 1)) != 0) ++q;
    return q;
}

// Parameters of a row; false if one is invalid.
struct Filters {
    float beta, top_p, min_p;
    int32_t top_k;
    bool greedy;
};
__device__ __forceinline__ bool filters_of(const SampleArgs &a, int64_t row, Filters &f) {
    const float t = a.f.temperatures ? a.f.temperatures[row] : a.f.temperature;
    f.top_p = a.f.top_ps ? a.f.top_ps[row] : a.f.top_p;
    f.min_p = a.f.min_ps ? a.f.min_ps[row] : a.f.min_p;
    f.top_k = a.f.top_ks ? a.f.top_ks[row] : a.f.top_k;
    f.greedy = t == 0.f || f.top_k == 1;
    f.beta = t == 0.f ? 1.f : fminf(__fdiv_rn(a.r.scale, t), 3.402823466e38f);
    return t >= 0.f && t <= 3.402823466e38f && f.top_p == f.top_p && f.min_p <= 1.f;
}

// m < 2^x of amplitudes' largest order value, where both 2^x and 2^-x are numbers (m 2^-x may be up to 4); those.
__device__ __forceinline__ int exponent_of(float m) {
    const int x = static_cast<int>(__float_as_uint(m) >> 23) - 126;
    return x > 126 ? 126 : x;
}
__device__ __forceinline__ float up_of(float m) { return __uint_as_float(static_cast<uint32_t>(127 + exponent_of(m)) << 23); }
__device__ __forceinline__ float down_of(float m) { return __uint_as_float(static_cast<uint32_t>(127 - exponent_of(m)) << 23); }

// What follows from a row's largest order value.
template <int TYPE>
__device__ __forceinline__ void plan_row(RowPlan &p, float m, bool valid, const Filters &f) {
    p.m = m;
    p.beta = f.beta;
    p.unit = f.beta == 1.f;
    if constexpr (Entry<TYPE>::kReal) {
        // With this the number next to m weighs 2^-124 .. 2^-62: less than a unit already, and what the
        // table and fp32's exponents reach
        p.b = fminf(f.beta, __fdiv_rn(43.f * 0x1p24f, fabsf(m)));
        p.ch = fminf(p.b * kLog2E, 3.402823466e38f);
        // (2^-60 .. 2^-120, where m's neighbours are few; differences beyond fp32 count as the largest number)
        p.low = fmaxf(fminf(m - __fdiv_rn(62.4f, p.b), nextafterf(m, -__builtin_huge_valf())),
                      fmaxf(m, 0.f) - 3.402823466e38f);
        const float at = m * p.b;
        p.far = !(fabsf(at) <= 64.f);
        const float grid = __fadd_rn(__fadd_rn(p.far ? 0.f : at * 0x1.71547652b82fep+10f, kMagic), -kMagic);
        p.origin = p.far ? m : grid;
        p.first = __float_as_uint(kMagic) + static_cast<uint32_t>(static_cast<int>(grid));
    } else {
        p.b = f.beta;
        p.ch = fminf(p.b * kLog2E, 3.402823466e38f);
        p.far = f.beta > 2.f;           // (the errors of logarithms count beta times)
        int n;
        const float g = lg2(2.f * frexpf(m, &n)) * 0.693147181f;       // (an estimate will do)
        p.origin = p.far ? m : (n - 1) + rintf(fmaxf(g, 0.f) * 65536.f) * 0x1p-16f;
    }
    p.greedy = f.greedy;
    p.bound = kPresent;
    p.down_log = p.unit && !Entry<TYPE>::kReal ? exponent_of(m) : 0;
    p.down = Entry<TYPE>::kReal ? 1.f : down_of(m);
    p.shift = 0;
    p.state = !valid || m != m || m == __builtin_huge_valf() ? kUndefined : m == absent<TYPE>() ? kEmpty : kDraw;
}
// and from an estimate of its weights' sum
__device__ __forceinline__ int shift_of(float sum) {
    int x;
    frexpf(fminf(fmaxf(sum, 0.25f), 0x1p33f) * 1.001f, &x);
    return 61 - x;
}

// The lowest order value of a present entry.
template <int TYPE>
__device__ __forceinline__ constexpr float least_present() {
    return Entry<TYPE>::kReal ? -3.402823466e38f : 1.4e-45f;
}

// Lower order values count as this one.
__device__ __forceinline__ float farthest(const RowPlan &p) { return fmaxf(p.m, 0.f) + kFarthest; }

// Entries of weight >= min_p of the largest: those of order value >= this.  (At a high temperature all: the
// value may lie below any, where the absent entries are.)
template <int TYPE>
__device__ __noinline__ float least_value(const RowPlan &p, float min_p) {
    double x;
    if constexpr (Entry<TYPE>::kReal) x = p.m + log(static_cast<double>(min_p)) / p.beta;
    else if (p.unit) x = static_cast<double>(p.m) * min_p;
    else x = p.m * exp(log(static_cast<double>(min_p)) / p.beta);
    float v = static_cast<float>(x);
    if (v < x) v = nextafterf(v, __builtin_huge_valf());
    if (Entry<TYPE>::kReal && v <= farthest(p)) v = least_present<TYPE>();      // (lower ones weigh as much as that)
    return fminf(fmaxf(v, least_present<TYPE>()), p.m);
}

// What log p of a draw is computed from: its order value, and the row's sum of weights left.  In 64
// bits, which a row's warp is slow at: the warps that take row after row collect a draw a lane
// and do 32 at a time.
struct LogP {
    uint64_t total;
    float v, origin, beta;
    int shift;          // weights' unit: 2^-shift of the origin's (of 1 for amplitudes at beta = 1)
    bool greedy, unit, far;

    __device__ __forceinline__ void of(const RowPlan &p, uint64_t t, float value) {
        total = t;
        v = fmaxf(value, farthest(p));
        origin = p.origin;
        far = p.far;
        beta = p.beta;
        greedy = p.greedy;
        unit = p.unit;
        shift = p.shift - p.down_log;
    }
};
template <int TYPE>
__device__ __noinline__ float log_p(const LogP &l) {
    constexpr double kLn2d = 0.693147180559945309;
    if (l.greedy) return 0.f;
    const double z = log(static_cast<double>(l.total));
    double x;
    if constexpr (Entry<TYPE>::kReal)
        x = l.far ? l.beta * (static_cast<double>(l.v) - l.origin) : static_cast<double>(l.beta) * l.v - l.origin * (kLn2d / 1024);
    else if (l.unit) x = log(static_cast<double>(l.v));
    else if (l.far) x = l.beta * log(static_cast<double>(l.v) / l.origin);
    else x = l.beta * (log(static_cast<double>(l.v)) - floorf(l.origin) * kLn2d - (l.origin - floorf(l.origin)));
    return static_cast<float>(x - (z - l.shift * kLn2d));
}

// ---- a row, digit by digit ------------------------------------------

struct Select {
    uint32_t lo[256], hi[256], count[256];
    int digit;
    uint32_t in_digit;
    uint64_t above;
    bool whole;
};

__device__ __forceinline__ void add_digit(Select *sel, int d, uint64_t w, bool mass) {
    atomicAdd(&sel->count[d], 1u);
    if (!mass) return;
    const uint32_t l = static_cast<uint32_t>(w), old = atomicAdd(&sel->lo[d], l);
    const uint32_t h = static_cast<uint32_t>(w >> 32) + (old + l < l);
    if (h) atomicAdd(&sel->hi[d], h);
}
// One warp: the digit, from the top, at which sums (or numbers) that begin with `above` reach the
// target; -1 if they do not.
template <bool MASS>
__device__ __noinline__ void find_digit(Select *sel, uint64_t above, uint64_t target) {
    const int lane = threadIdx.x % 32;
    const auto at = [&](int i) -> uint64_t {        // eight digits a lane
        const int d = 255 - lane * 8 - i;
        return MASS ? static_cast<uint64_t>(sel->hi[d]) << 32 | sel->lo[d] : sel->count[d];
    };
    uint64_t own = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) own += at(i);
    uint64_t upto = above + warp_scan(own, lane);
    const uint32_t reached = __ballot_sync(0xffffffffu, upto >= target);
    if (lane == 0) sel->digit = -1;
    __syncwarp();
    if (!reached || lane != __ffs(reached) - 1) return;
    upto -= own;
    for (int i = 0; i < 8; ++i) {
        const uint64_t x = at(i);
        if (upto + x >= target) {
            const int d = 255 - lane * 8 - i;
            sel->digit = d;
            sel->in_digit = sel->count[d];
            sel->above = upto;
            sel->whole = upto + x == target;
            return;
        }
        upto += x;
    }
}

// A row that the CTA's threads share.
template <int TYPE>
struct RowCta {
    static constexpr int E = Entry<TYPE>::E;
    Row<TYPE> r;
    int64_t vecs;
    const RowPlan *p;
    const float *roots;
    Select *sel;
    uint64_t *sums;     // kDrawWarps

    // f(order value, index) of every entry of the row
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        each_vector<TYPE, kDrawThreads, 1>(r, 0, vecs, threadIdx.x, [&](const float (&v)[E], int64_t j, int) {
#pragma unroll
            for (int i = 0; i < E; ++i) f(v[i], j * E - r.head + i);
        });
    }
    __device__ __forceinline__ uint64_t sum(uint64_t x) const {
        x = warp_sum(x);
        __syncthreads();
        if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = x;
        __syncthreads();
        x = 0;
        for (int w = 0; w < kDrawWarps; ++w) x += sums[w];
        return x;
    }
    // Weights' sum (or the number) of the entries of at least that rank.
    template <bool MASS>
    __device__ __noinline__ uint64_t total(uint64_t bound) const {
        uint64_t s = 0;
        each([&](float v, int64_t e) {
            if (rank_of<TYPE>(v, e) >= bound) s += MASS ? weight_once<TYPE>(*p, roots, v) : 1;
        });
        return sum(s);
    }
    // The rank down to which entries, largest first, reach `target` in weight (or
    // number), of those of at least the rank `bound`; `bound` if all do not.  Eight
    // bits of the rank at a time, from the top: sums by digit, then on with the digit in
    // which the target is reached.
    template <bool MASS>
    __device__ __noinline__ uint64_t select(uint64_t target, uint64_t bound) const {
        uint64_t prefix = 0, above = 0;
        for (int shift = 56; shift >= 0; shift -= 8) {
            if (shift == 24 && r.cols <= 1 << 24) {         // the same digit in every index
                prefix |= 0xffull << 24;
                continue;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 256; i += kDrawThreads) sel->lo[i] = sel->hi[i] = sel->count[i] = 0;
            __syncthreads();
            each([&](float v, int64_t e) {
                const uint64_t k = rank_of<TYPE>(v, e);
                if (k < bound || k == 0 || (shift < 56 && (k ^ prefix) >> (shift + 8))) return;
                const int d = static_cast<int>(k >> shift & 255);
                add_digit(sel, d, MASS ? weight_once<TYPE>(*p, roots, v) : 0, MASS);
            });
            __syncthreads();
            if (threadIdx.x < 32) find_digit<MASS>(sel, above, target);
            __syncthreads();
            if (sel->digit < 0) return bound;
            above = sel->above;
            prefix |= static_cast<uint64_t>(sel->digit) << shift;
            if (sel->in_digit == 1 || sel->whole) break;    // all of the digit, whatever follows
        }
        return prefix > bound ? prefix : bound;
    }
};

// Which entries of a row are left: those of order value >= gate, and of those below it but
// >= list the ones of rank >= bound.
struct Cut {
    float gate, list;
    uint64_t bound;
    // (a second range for top_k, where top_p cuts far above it)
    float gate2, list2;
};
template <int TYPE>
__device__ __forceinline__ bool is_left(const Cut &c, float v, int64_t e) {
    return v >= c.gate || (v >= c.list && rank_of<TYPE>(v, e) >= c.bound);
}

// Weights' sum of a vector's entries that are left, 1 at least for each: of those
// above the gate together, of the others one by one.
template <int TYPE>
__device__ __noinline__ uint64_t vector_weight(const RowPlan &p, const Cut &c, const float *roots,
                                               const float (&v)[Entry<TYPE>::E], int64_t e0) {
    constexpr int E = Entry<TYPE>::E;
    uint64_t own = 0;
    if constexpr (Entry<TYPE>::kReal) {
        PairSum sum;
        uint32_t n = 0, some = 0;
#pragma unroll 1
        for (int k = 0; k < E; k += 2) {
            const bool above = v[k] >= c.gate, above1 = v[k + 1] >= c.gate;
            const Weights w = weight_pairs(p, roots, v[k], v[k + 1], above, above1);
            sum.add(w.hi, w.lo);
            n += above + above1;
            some |= (!above && v[k] >= c.list) || (!above1 && v[k + 1] >= c.list);
        }
        own = sum.units(p.shift) + n;
        if (some) {
#pragma unroll 1
            for (int k = 0; k < E; ++k)
                if (!(v[k] >= c.gate) && is_left<TYPE>(c, v[k], e0 + k)) own += weight_once<TYPE>(p, roots, v[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (is_left<TYPE>(c, v[k], e0 + k)) own += weight_once<TYPE>(p, roots, v[k]);
    }
    return own;
}

// The first of n sums at which their total exceeds `target`, which becomes what is
// left of it there; one warp.
__device__ __forceinline__ int64_t locate(const uint64_t *sums, int64_t n, uint64_t &target) {
    const int lane = threadIdx.x % 32;
    for (int64_t base = 0; base < n; base += 32) {
        const uint64_t own = base + lane < n ? __ldcg(sums + base + lane) : 0, upto = warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, upto > target);
        if (over) {
            const int l = __ffs(over) - 1;
            target -= shfl_from(upto - own, l);
            return base + l;
        }
        target -= shfl_from(upto, 31);
    }
    return 0;
}
// The same of sums that are added up already, upto(i): a search by 32.
template <class F>
__device__ __forceinline__ int64_t locate_upto(F upto, int64_t n, uint64_t &target) {
    const int lane = threadIdx.x % 32;
    int64_t lo = 0, len = n;
    while (len > 1) {
        const int64_t step = (len + 31) / 32, at = lo + (lane + 1) * step - 1;
        const bool over = lane * step < len && (at >= lo + len - 1 || upto(at) > target);
        const int l = __ffs(__ballot_sync(0xffffffffu, over)) - 1;
        len = len - l * step < step ? len - l * step : step;
        lo += l * step;
    }
    if (lo > 0) target -= upto(lo - 1);
    return lo;
}

__device__ __forceinline__ double random_number(const SampleArgs &a, int64_t at) {
    return a.wide ? static_cast<const double *>(a.u)[at] : static_cast<const float *>(a.u)[at];
}
// A draw with an invalid number.
__device__ __forceinline__ void bad_draw(const SampleArgs &a, int64_t at, int64_t row) {
    a.ids[at] = -1;
    a.logp[at] = __uint_as_float(0x7fc00000u);
    flag_bad_id(a.r, row);
}
// One thread: the draw falls into this vector, `left` behind its first entry's begin.  Its order value.
template <int TYPE>
__device__ __noinline__ float finish_draw(const SampleArgs &a, const RowPlan &p, const Cut &c, const float *roots,
                                          const float (&v)[Entry<TYPE>::E], int64_t e0, uint64_t left, int64_t at) {
    constexpr int E = Entry<TYPE>::E;
    // (the vector's sum may be some units more than its entries': the last one's then)
    float value = 0.f;
    int64_t id = -1;
    bool found = false;
#pragma unroll 1
    for (int k = 0; k < E; ++k) {
        if (found || !is_left<TYPE>(c, v[k], e0 + k)) continue;
        const uint64_t w = weight_once<TYPE>(p, roots, v[k]) + (Entry<TYPE>::kReal && v[k] >= c.gate ? 1 : 0);
        value = v[k];
        id = e0 + k;
        found = w > left;
        left -= w;
    }
    a.ids[at] = id;
    return value;
}

// One warp: a draw of row r that lies `target` behind the begin of piece `first`, within the next
// `pieces`.  Its order value, to all lanes.
template <int TYPE>
__device__ __noinline__ float warp_draw(const SampleArgs &a, const Row<TYPE> &r, int64_t vecs, const RowPlan &p, const Cut &c,
                                        const float *roots, const uint64_t *masses, int64_t first, int64_t pieces,
                                        uint64_t target, int64_t at) {
    constexpr int E = Entry<TYPE>::E;
    const int lane = threadIdx.x % 32;
    const int64_t piece = first + locate(masses + first, pieces, target);
#pragma unroll 1
    for (int i = 0; i < kPieceVecs / 32; ++i) {
        const int64_t j = piece * kPieceVecs + i * 32 + lane;
        float v[E];
        uint64_t own = 0;
        if (j < vecs) {
            vector_values<TYPE>(r, j, v);
            own = vector_weight<TYPE>(p, c, roots, v, j * E - r.head);
        }
        const uint64_t upto = warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, upto > target);
        if (!over) {
            target -= shfl_from(upto, 31);
            continue;
        }
        const int l = __ffs(over) - 1;
        float value = 0.f;
        if (lane == l) value = finish_draw<TYPE>(a, p, c, roots, v, j * E - r.head, target - (upto - own), at);
        return __shfl_sync(0xffffffffu, value, l);
    }
    return 0.f;
}
// Whether a random number is valid; what it aims at.
__device__ __forceinline__ bool aim(const SampleArgs &a, double u, bool greedy, uint64_t total, int64_t at, int64_t row,
                                    uint64_t &target) {
    if (!(u >= 0.0 && u < 1.0)) {
        if (threadIdx.x % 32 == 0) bad_draw(a, at, row);
        return false;
    }
    target = greedy ? 0 : share(u, total, false);
    return true;
}

// Draws of a warp whose log p is still to come, a lane each.
template <int TYPE>
struct Pending {
    LogP l;
    int64_t at;
    int n = 0;

    __device__ __forceinline__ void flush(const SampleArgs &a) {
        if (static_cast<int>(threadIdx.x % 32) < n) a.logp[at] = log_p<TYPE>(l);
        n = 0;
    }
    __device__ __forceinline__ void add(const SampleArgs &a, const RowPlan &p, uint64_t total, float v, int64_t where) {
        if (static_cast<int>(threadIdx.x % 32) == n) {
            l.of(p, total, v);
            at = where;
        }
        if (++n == 32) flush(a);
    }
};

// Outcomes of a row that has none, by thread t of n.
__device__ __forceinline__ void no_draws(const SampleArgs &a, int64_t row, int state, int t, int n) {
    for (int64_t d = t; d < a.draws; d += n) {
        a.ids[row * a.draws + d] = -1;
        a.logp[row * a.draws + d] = state == kEmpty ? -__builtin_huge_valf() : __uint_as_float(0x7fc00000u);
    }
    if (t == 0) a.kept[row] = 0;
}

// The rank where the filters of a row cut.
template <int TYPE>
__device__ __noinline__ uint64_t bound_of(const RowCta<TYPE> &c, const RowPlan &p, int64_t top_k, float top_p) {
    uint64_t bound = kPresent;
    if (top_k > 0 && top_k < c.r.cols) bound = c.template select<false>(top_k, bound);
    if (top_p < 1.f) {
        const uint64_t all = c.template total<true>(bound), t = share(fmaxf(top_p, 0.f), all, true);
        bound = c.template select<true>(t > 0 ? t : 1, bound);
    }
    return bound > p.bound ? bound : p.bound;
}

// ---- rows in registers ---------------------------------------------------------
//
// N entries a thread (4 or 8 for the shortest rows, or kHeldEntries), whose weights are kept too;
// a warp a row, or a CTA of NT threads.  Filters find where they cut by halves of the order
// values (how many, or how much, lies at or above the middle) until one entry, or one value, is
// left in question.  Bound by its chain of reductions where rows are filtered, by the weights'
// arithmetic where not: 20000 x 64 amplitudes 32 us (with top_p 48), 16384 x 2048 bf16 147 (372),
// 1 x 32768 bf16 in a cluster of eight 10 (24, with top_k and top_p 29).  With 16 entries a thread
// 20000 x 256 bf16 take as long as 20000 x 512 (52 us), with 8 32.  All draws of a row are made by the warp or CTA
// that holds it, 0.5 to 0.6 us each: 1000 of 64 amplitudes 0.54 ms, 10^6 0.52 s (of 1024 amplitudes, a row in
// segments, whose draws have a kernel over all SMs, 38 us and 1.8 ms).

constexpr int kHeldEntries = 16;

// Sums over a warp, a CTA or a cluster of up to kMostRanks CTAs; of more than a warp, one barrier each, with two sets
// of places in turn.  In a cluster every warp's part goes to a place in every CTA.
constexpr int kMostRanks = 8;
__device__ __forceinline__ uint32_t rank_address(const void *p, int rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
    return at;
}
__device__ __forceinline__ void ranks_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int NT, bool RANKS>
struct RowGroup {
    static constexpr int kWarps = NT / 32, kMost = RANKS ? kMostRanks * kWarps : kWarps;
    ulonglong2 *places;     // 2 * kMost (unused by a warp)
    int lane, warp, rank = 0, ranks = 1, half = 0;

    // Each warp's (x, y), given by its lanes alike: those of warp `i` at the place returned + i, all to be read
    // from then on by every warp.
    __device__ __forceinline__ const ulonglong2 *meet(uint64_t x, uint64_t y) {
        half ^= 1;
        ulonglong2 *s = places + half * kMost;
        if constexpr (RANKS) {
            if (lane < ranks)
                asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(rank_address(s + rank * kWarps + warp, lane)),
                             "l"(x), "l"(y) : "memory");
            ranks_sync();
        } else {
            if (lane == 0) s[warp] = make_ulonglong2(x, y);
            __syncthreads();
        }
        return s;
    }
    // f(x, y) of every warp's part; in a cluster of 32nds of the parts by lane
    template <class F>
    __device__ __forceinline__ void each(const ulonglong2 *s, F f) const {
        if constexpr (RANKS) {
            for (int i = lane; i < ranks * kWarps; i += 32) f(s[i]);
        } else {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) f(s[w]);
        }
    }
    __device__ __forceinline__ float max(float x) {
        x = warp_max_nan(x);
        if constexpr (NT > 32) {
            each(meet(__float_as_uint(x), 0), [&](ulonglong2 y) { x = max_nan(x, __uint_as_float(static_cast<uint32_t>(y.x))); });
            if constexpr (RANKS) x = warp_max_nan(x);
        }
        return x;
    }
    __device__ __forceinline__ uint64_t max(uint64_t x) {
        const auto over_warp = [&] {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const uint64_t y = __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(x), o);
                x = y > x ? y : x;
            }
        };
        over_warp();
        if constexpr (NT > 32) {
            each(meet(x, 0), [&](ulonglong2 y) { x = y.x > x ? y.x : x; });
            if constexpr (RANKS) over_warp();
        }
        return x;
    }
    __device__ __forceinline__ float sum(float x) {
        const auto over_warp = [&] {
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        };
        over_warp();
        if constexpr (NT > 32) {
            const ulonglong2 *s = meet(__float_as_uint(x), 0);
            x = 0.f;
            each(s, [&](ulonglong2 y) { x += __uint_as_float(static_cast<uint32_t>(y.x)); });
            if constexpr (RANKS) over_warp();
        }
        return x;
    }
    __device__ __forceinline__ void sum(uint64_t &x, uint32_t &n) {
        x = warp_sum(x);
        n = __reduce_add_sync(0xffffffffu, n);
        if constexpr (NT > 32) {
            const ulonglong2 *s = meet(x, n);
            x = n = 0;
            each(s, [&](ulonglong2 y) {
                x += y.x;
                n += static_cast<uint32_t>(y.y);
            });
            if constexpr (RANKS) {
                x = warp_sum(x);
                n = __reduce_add_sync(0xffffffffu, n);
            }
        }
    }
    __device__ __forceinline__ uint32_t sum(uint32_t n) {
        n = __reduce_add_sync(0xffffffffu, n);
        if constexpr (NT > 32) {
            const ulonglong2 *s = meet(n, 0);
            n = 0;
            each(s, [&](ulonglong2 y) { n += static_cast<uint32_t>(y.x); });
            if constexpr (RANKS) n = __reduce_add_sync(0xffffffffu, n);
        }
        return n;
    }
    // inclusive; all: the sum of all
    __device__ __forceinline__ uint64_t scan(uint64_t x, uint64_t &all) {
        x = warp_scan(x, lane);
        all = shfl_from(x, 31);
        if constexpr (NT > 32) {
            const ulonglong2 *s = meet(all, 0);
            uint64_t before = 0;
            all = 0;
            if constexpr (RANKS) {
                for (int i = lane; i < ranks * kWarps; i += 32) {
                    all += s[i].x;
                    before += i < rank * kWarps + warp ? s[i].x : 0;
                }
                all = warp_sum(all);
                before = warp_sum(before);
            } else {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    all += s[w].x;
                    before += w < warp ? s[w].x : 0;
                }
            }
            x += before;
        }
        return x;
    }
};

template <int TYPE, int N, int NT, bool RANKS>
__global__ void __launch_bounds__(NT == 32 ? kDrawThreads : NT, (N <= 8 ? 1024 : 512) / (NT == 32 ? kDrawThreads : NT))
held_rows_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E, V = N / E, THREADS = NT == 32 ? kDrawThreads : NT, ROWS = THREADS / NT;
    constexpr int WARPS = NT / 32;
    // bits below these are the same in all order values
    constexpr int LOWEST = TYPE == TN_TYPE_BF16 ? 16 : TYPE == TN_TYPE_F16 ? 13 : 0;
    __shared__ float roots[2 * kRoots];
    __shared__ ulonglong2 places[2 * RowGroup<NT, RANKS>::kMost];
    __shared__ float values[2][WARPS];
    pdl_trigger();
    if (Entry<TYPE>::kReal || a.powers) make_roots<THREADS>(roots);
    pdl_wait();
    __syncthreads();
    const int t = threadIdx.x % NT, lane = t % 32, warp = t / 32;
    RowGroup<NT, RANKS> g{places, lane, warp};
    if constexpr (RANKS) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(g.rank));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(g.ranks));
        ranks_sync();       // (all have started before any writes to another's memory)
    }
    const int rank = g.rank, ranks = g.ranks;
    // vector i of this thread
    const auto vector_at = [&](int i) { return (i * ranks + rank) * NT + t; };
    int turn = 0;
    Pending<TYPE> pending;
    for (int64_t row = static_cast<int64_t>(blockIdx.x / ranks) * ROWS + threadIdx.x / NT; row < a.r.rows;
         row += static_cast<int64_t>(gridDim.x / ranks) * ROWS) {
        const Row<TYPE> r(a.r, row);
        const int vecs = static_cast<int>((r.head + r.cols + E - 1) / E);
        Filters f;
        const bool valid = filters_of(a, row, f);
        float v[V][E];
        float m = absent<TYPE>();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (vector_at(i) < vecs) {
                vector_values<TYPE>(r, vector_at(i), v[i]);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) v[i][k] = absent<TYPE>();
            }
#pragma unroll
            for (int k = 0; k < E; ++k) m = max_nan(m, v[i][k]);
        }
        m = g.max(m);
        RowPlan p;
        plan_row<TYPE>(p, m, valid, f);
        if (!valid && t == 0) flag_bad_id(a.r, row);
        if (p.state != kDraw) {
            if (rank == 0) no_draws(a, row, p.state, t, NT);
            continue;
        }
        if (!p.greedy) {
            float s = 0.f;
            if (Entry<TYPE>::kReal && p.ch >= kRareScale) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < E; ++k) s += ex2((v[i][k] - m) * p.ch);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < E; ++k)
                        if (v[i][k] != absent<TYPE>()) s += rough_weight<TYPE>(p, v[i][k]);
            }
            p.shift = shift_of(g.sum(s));
        }
        uint64_t w[V][E];       // 0 of what is not left, 1 at least otherwise
        uint64_t total = 0;     // of the row's
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < E; k += 2) {
                two_weights<TYPE>(p, roots, v[i][k], v[i][k + 1], w[i][k], w[i][k + 1]);
#pragma unroll
                for (int h = k; h < k + 2; ++h) {
                    const bool here = p.greedy ? v[i][h] == m : v[i][h] != absent<TYPE>();
                    if (!here) {
                        v[i][h] = absent<TYPE>();
                        w[i][h] = 0;
                    }
                    total += w[i][h];
                    left += here;
                }
            }
        // Keep the entries, largest first, until `target` is reached.  What is left has keys of `bottom` on;
        // under: that is a bound found already.
        uint32_t bottom = order_key<TYPE>(least_present<TYPE>()) & ~((1u << LOWEST) - 1u);
        bool under = !Entry<TYPE>::kReal;
        const auto cut = [&](uint64_t target, bool by_mass) {
            // the entry where it is has a key of lo <= key < hi: halves (numbers: quarters) of the values between
            // them, from first steps below the largest on; of the keys where those would take too long
            constexpr uint32_t kUnit = 1u << LOWEST;
            uint32_t lo = bottom, hi = (order_key<TYPE>(m) & ~(kUnit - 1u)) + kUnit;
            uint32_t least = left, most = 0;    // entries of lo and above, of hi and above
            uint64_t above = 0;                 // what of hi and above amounts to
            float step = __fdiv_rn(8.f, p.beta);
            for (int probes = 0; hi - lo > kUnit && least - most > 1; ++probes) {
                const float lowest = key_value(lo), highest = key_value(hi), middle = 0.5f * lowest + 0.5f * highest;
                // the key of a value between lo and hi, or if there is none of `part` quarters of the way
                const auto between = [&](float value, uint32_t part) {
                    const uint32_t x = order_key<TYPE>(value) & ~(kUnit - 1u);
                    return x > lo && x < hi && probes < 20 ? x : lo + ((hi - lo) / 4 * part + (hi - lo) % 4 * part / 4 & ~(kUnit - 1u));
                };
                if (by_mass) {
                    const uint32_t x = between(under ? middle : m - step, 2);
                    const float from = key_value(x);
                    uint64_t s = 0;
                    uint32_t n = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int k = 0; k < E; ++k)
                            if (v[i][k] >= from) {
                                s += w[i][k];
                                ++n;
                            }
                    g.sum(s, n);
                    if (s >= target) {
                        lo = x;
                        least = n;
                        under = true;
                    } else {
                        hi = x;
                        above = s;
                        most = n;
                    }
                } else {
                    const uint32_t x2 = between(under ? middle : m - step, 2);
                    const uint32_t y1 = between(under ? 0.5f * lowest + 0.5f * middle : m - 8.f * step, 1);
                    const uint32_t y3 = between(under ? 0.5f * middle + 0.5f * highest : m - 0.125f * step, 3);
                    const uint32_t x1 = y1 < x2 ? y1 : x2, x3 = y3 > x2 ? y3 : x2;
                    const float from1 = key_value(x1), from2 = key_value(x2), from3 = key_value(x3);
                    uint64_t s = 0;             // three numbers of 21 bits
                    uint32_t n1 = 0, n2 = 0, n3 = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            n1 += v[i][k] >= from1;
                            n2 += v[i][k] >= from2;
                            n3 += v[i][k] >= from3;
                        }
                    s = n1 | static_cast<uint64_t>(n2) << 21 | static_cast<uint64_t>(n3) << 42;
                    uint32_t none = 0;
                    g.sum(s, none);
                    constexpr uint32_t kNumber = (1u << 21) - 1u;
                    n1 = static_cast<uint32_t>(s) & kNumber;
                    n2 = static_cast<uint32_t>(s >> 21) & kNumber;
                    n3 = static_cast<uint32_t>(s >> 42);
                    const auto reached = [&](uint32_t x, uint32_t n) {
                        if (n >= target && x > lo) {
                            lo = x;
                            least = n;
                            under = true;
                        }
                    };
                    const auto missed = [&](uint32_t x, uint32_t n) {
                        if (n < target && x < hi) {
                            hi = x;
                            above = most = n;
                        }
                    };
                    reached(x1, n1);
                    reached(x2, n2);
                    reached(x3, n3);
                    missed(x3, n3);
                    missed(x2, n2);
                    missed(x1, n1);
                }
            }
            bottom = lo;
            // of equal entries (which have equal weights) as many as it takes, the first ones
            uint64_t one = 0;
            uint32_t tied = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const uint32_t o = order_key<TYPE>(v[i][k]);
                    if (o >= lo && o < hi && w[i][k] > 0) {
                        one = by_mass ? w[i][k] : 1;
                        tied |= 1u << (i * E + k);
                    } else if (o < lo) {
                        v[i][k] = absent<TYPE>();
                        w[i][k] = 0;
                    }
                }
            if (least - most <= 1) return;
            one = g.max(one);       // (one weight only)
            uint32_t need = one > 0 && target > above ? static_cast<uint32_t>((target - above + one - 1) / one) : 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {       // in the order of indices
                const uint32_t mine = __popc(tied >> (i * E) & ((1u << E) - 1u));
                uint64_t all;
                uint32_t before = static_cast<uint32_t>(g.scan(mine, all)) - mine;
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (tied >> (i * E + k) & 1) {
                        if (before >= need) {
                            v[i][k] = absent<TYPE>();
                            w[i][k] = 0;
                        }
                        ++before;
                    }
                need = need > all ? need - static_cast<uint32_t>(all) : 0;
            }
        };
        // what is left after a filter
        const auto count = [&] {
            total = 0;
            left = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    total += w[i][k];
                    left += w[i][k] > 0;
                }
            g.sum(total, left);
        };
        if (!p.greedy && a.filtered) {
            g.sum(total, left);
            if (f.top_k > 0 && static_cast<uint32_t>(f.top_k) < left) {
                cut(f.top_k, false);
                count();
            }
            if (f.top_p < 1.f) {
                const uint64_t x = share(fmaxf(f.top_p, 0.f), total, true);
                cut(x > 0 ? x : 1, true);
            }
        }
        if (!p.greedy && f.min_p > 0.f) {
            const float least = least_value<TYPE>(p, f.min_p);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (v[i][k] < least) w[i][k] = 0;
        }
        left = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < E; ++k) left += w[i][k] > 0;
        left = g.sum(left);
        if (t == 0 && rank == 0) a.kept[row] = p.greedy ? 1 : left;
        // sums up to each of the thread's vectors
        uint64_t upto[V];
        total = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint64_t own = 0, all;
#pragma unroll
            for (int k = 0; k < E; ++k) own += w[i][k];
            upto[i] = total + g.scan(own, all);
            total += all;
        }
        // draws, in a CTA one for each warp between two barriers: the thread that has the outcome finds it
        for (int64_t d0 = 0; d0 < a.draws; d0 += WARPS) {
            bool drawn = false;         // this warp's
            float value = 0.f;
#pragma unroll
            for (int j = 0; j < WARPS; ++j) {
                if (d0 + j >= a.draws) break;
                const int64_t at = row * a.draws + d0 + j;
                uint64_t target;
                const bool good = aim(a, random_number(a, at), p.greedy, total, at, row, target);
                if (j == warp) drawn = good;
                if (!good) continue;
                bool owner = false;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    uint64_t own = 0;
#pragma unroll
                    for (int k = 0; k < E; ++k) own += w[i][k];
                    uint64_t before = upto[i] - own;
                    if (upto[i] <= target || before > target) continue;
                    owner = true;
                    bool found = false;
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        before += w[i][k];
                        if (found || before <= target) continue;
                        found = true;
                        a.ids[at] = vector_at(i) * E + k - r.head;
                        value = v[i][k];
                    }
                }
                if constexpr (NT == 32) {
                    const uint32_t who = __ballot_sync(0xffffffffu, owner);
                    value = __shfl_sync(0xffffffffu, value, __ffs(who) - 1);
                } else if (owner) {
                    if constexpr (RANKS)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(rank_address(&values[turn][j], 0)), "f"(value)
                                     : "memory");
                    else
                        values[turn][j] = value;
                }
            }
            if constexpr (NT > 32) {
                if constexpr (RANKS) ranks_sync();
                else __syncthreads();
                value = values[turn][warp];
                turn ^= 1;
            }
            if (drawn && rank == 0) pending.add(a, p, total, value, row * a.draws + d0 + warp);
        }
    }
    pending.flush(a);
}

// ---- rows in segments -------------------------------------------------------
//
// One CTA a segment, a kernel for each pass over the rows; the CTA that finishes a
// row's last segment does what follows for the row:
//   top_kernel    the largest entry and a rough sum of weights; then the row's plan
//   bins_kernel   where a row has a top_k or top_p: how many entries lie in bins of the
//                 order value; then a range of bins in which the filters cut (a bin's
//                 weight is about its number times that of its middle)
//   sums_kernel   sums of the weights above the range, by pieces and segments, and the
//                 range's entries in a list; then the list is sorted, the cut found among it
//                 by exact sums, what is left of it added to the pieces, and a few draws made
//   draws_kernel  many draws, a warp each
// The first two are bound by memory, the third by arithmetic (some 50 operations for a
// weight); launches hide behind each other's ends.  64 x 131072 bf16 44 us (with top_p 121), 1024 x 50001 f16
// with a mask 170, 4096 shots of 2^24 amplitudes 88.
//
// A range with more entries than are listed: rows of kLongRow entries on look once more into up to
// four bins, each slot a bin; where all of the range are equal (16-bit logits of long rows, uniform
// states), their numbers in the pieces say how far they are left; else the row's CTA goes digit by
// digit through the ranks.  That is the way of top_k above 2048 together with top_p whose last entry has
// thousands of equals (100 ms for 2^24 entries), and of shorter rows whose logits lie close together: a bin is 1/64 of a
// power of two in weight, and 64 x 131072 f32 with top_p 0.9 take 130 us at a standard deviation of
// 2 (times beta), 158 at 0.3, and 2.0 ms from 0.1 on; with top_k 1000 91, 96, 101 and from 0.02 on 640 to 840.

struct RowState {
    RowPlan plan;
    Cut cut;
    float top_p;
    int32_t top_k;
    int32_t narrow;         // bins are wanted (kBinned), the list decides (kListed), or neither
    float bin_scale, min_value;
    int32_t slot_lo, slot_hi;   // slots (see slot_of) of the range
    uint32_t expected;      // its entries
    uint32_t above;         // and those above it
    int32_t two;            // a second range, for top_k
    uint32_t above2;        // entries above that
    uint64_t total;         // weights left
    uint32_t arrived[3];
    uint32_t listed;
    uint32_t key_hi, key_not;       // of a range too full to be listed: largest key, largest complement of one
    // sums of estimates of all weights and of those above the bins looked into, in the bins' units
    unsigned long long rough, rough_above;
};
enum { kBinned = 1, kListed = 2 };

struct RowBins {
    uint32_t count[kBins];
};

// Place of an order value on a scale from the largest down, of kBins bins of kSlots
// slots: for logits linear, for amplitudes linear between powers of two.  A larger
// value's is never greater (roundings are monotone).
constexpr int kSlots = 1024, kLastSlot = kBins * kSlots - 1;
template <int TYPE>
__device__ __forceinline__ int slot_of(const RowPlan &p, float bin_scale, float v) {
    if constexpr (Entry<TYPE>::kReal) {
        const float t = (p.m - v) * bin_scale;
        return static_cast<int>(fminf(t, static_cast<float>(kLastSlot)));
    } else {
        const uint32_t d = (__float_as_uint(p.m) - __float_as_uint(v)) >> 7;
        return d < kLastSlot ? static_cast<int>(d) : kLastSlot;
    }
}
// The lowest order value whose slot is below `slot`.
template <int TYPE>
__device__ __noinline__ float slot_begin(const RowPlan &p, float bin_scale, int slot) {
    if (slot <= 0) return __builtin_huge_valf();
    uint32_t lo = order_key<TYPE>(least_present<TYPE>()), hi = order_key<TYPE>(p.m);    // hi's slot is 0
    if (Entry<TYPE>::kReal) {       // near where it should be, if it is there
        const uint32_t guess = order_key<TYPE>(p.m - slot / bin_scale);
        if (guess > lo + 64 && guess + 64 < hi && slot_of<TYPE>(p, bin_scale, key_value(guess - 64)) >= slot &&
            slot_of<TYPE>(p, bin_scale, key_value(guess + 64)) < slot) {
            lo = guess - 64;
            hi = guess + 64;
        }
    }
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (slot_of<TYPE>(p, bin_scale, key_value(mid)) < slot) hi = mid;
        else lo = mid + 1;
    }
    return key_value(hi);
}

template <int TYPE>
struct Segment {
    Row<TYPE> r;
    int64_t row, seg, vecs, lo, hi;     // vectors of the row and of the segment

    __device__ __forceinline__ explicit Segment(const SampleArgs &a)
        : r(a.r, static_cast<int64_t>(blockIdx.x / static_cast<uint32_t>(a.segs))) {
        row = blockIdx.x / static_cast<uint32_t>(a.segs);
        seg = blockIdx.x - row * a.segs;
        vecs = (r.head + r.cols + Entry<TYPE>::E - 1) / Entry<TYPE>::E;
        lo = seg * a.seg_pieces * kPieceVecs;
        hi = lo + a.seg_pieces * kPieceVecs;
        if (hi > vecs) hi = vecs;
    }
};

// Whether this CTA is the last of its row's to come here.  What the others wrote
// before is visible to it.
__device__ __forceinline__ bool last_of_row(const SampleArgs &a, RowState &s, int which) {
    __shared__ bool last;
    if (a.segs == 1) {
        __syncthreads();
        return true;
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomicAdd(&s.arrived[which], 1u) == a.segs - 1;
        if (last) s.arrived[which] = 0;
        __threadfence();
    }
    __syncthreads();
    return last;
}

template <int TYPE>
__global__ void __launch_bounds__(kDrawThreads) top_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ uint32_t red[4 * kDrawWarps];
    pdl_trigger();
    pdl_wait();
    Group<kDrawThreads> g(red);
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    Filters f;
    const bool valid = filters_of(a, c.row, f);
    // the sum relative to the largest entry so far (of amplitudes at beta = 1 times down_of it)
    const float ch = fminf(f.beta * kLog2E, 3.402823466e38f);
    float m = absent<TYPE>(), s = 0.f;
    const auto over = [&](auto f) { each_vector<TYPE, kDrawThreads, 4>(c.r, c.lo, c.hi, threadIdx.x, f); };
    if (!Entry<TYPE>::kReal && f.beta == 1.f) {
        float down = 1.f, limit = 0.f;      // which down_of(m) holds below
        over([&](const float (&v)[E], int64_t, int) {
            float top = v[0];
#pragma unroll
            for (int i = 1; i < E; ++i) top = max_nan(top, v[i]);
            if (!(top < limit)) {
                down = down_of(top);
                limit = up_of(top);
                s *= down * up_of(m);
            }
            m = max_nan(m, top);
#pragma unroll
            for (int i = 0; i < E; ++i) s = fmaf(v[i], down, s);
        });
    } else {
        // RARE: see kRareScale; amplitudes' logarithms: see rough_power
        const auto pass = [&](auto rare) {
            constexpr bool RARE = decltype(rare)::value;
            over([&](const float (&v)[E], int64_t, int) {
                float top = v[0];
#pragma unroll
                for (int i = 1; i < E; ++i) top = max_nan(top, v[i]);
                if (!(top <= m)) {
                    if constexpr (Entry<TYPE>::kReal) s *= ex2(fmaxf(m - top, kFarthest) * ch);
                    else s *= m > 0.f ? ex2(rough_power(f.beta, ch, m, top)) : 0.f;
                    m = max_nan(m, top);
                }
                if constexpr (Entry<TYPE>::kReal) {
                    if (top != absent<TYPE>()) {
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            if (!RARE) s += ex2((v[i] - m) * ch);
                            else if (v[i] != absent<TYPE>()) s += ex2(fmaxf(v[i] - m, kFarthest) * ch);
                        }
                    }
                } else if (!RARE && m >= 0x1p-60f) {    // (below 2^-126 less than 2^-33 of m's)
                    const float l = lg2(m);
#pragma unroll
                    for (int i = 0; i < E; ++i) s += ex2(f.beta * (lg2(v[i]) - l));
                } else if (m > 0.f) {
#pragma unroll
                    for (int i = 0; i < E; ++i) s += v[i] > 0.f ? ex2(rough_power(f.beta, ch, v[i], m)) : 0.f;
                }
            });
        };
        const bool rare = Entry<TYPE>::kReal ? ch < kRareScale : f.beta < 0.5f || f.beta > 64.f;
        if (rare) pass(std::true_type{});
        else pass(std::false_type{});
    }
    // threads', then segments'
    const auto moved = [&](float from, float to) {
        if (from == absent<TYPE>()) return 0.f;
        if constexpr (Entry<TYPE>::kReal) return ex2(fmaxf(from - to, kFarthest) * ch);
        else return f.beta == 1.f ? down_of(to) * up_of(from) : ex2(rough_power(f.beta, ch, from, to));
    };
    const float own = m;
    m = g.max(m);
    s = g.sum(own == absent<TYPE>() ? 0.f : s * moved(own, m));
    if (a.segs > 1) {
        ulonglong2 *parts = a.partials + c.row * a.segs;
        if (threadIdx.x == 0)
            __stcg(&parts[c.seg], make_ulonglong2(__float_as_uint(m), __float_as_uint(s)));
        if (!last_of_row(a, st, 0)) return;
        m = absent<TYPE>();
        for (int64_t i = threadIdx.x; i < a.segs; i += kDrawThreads)
            m = max_nan(m, __uint_as_float(static_cast<uint32_t>(__ldcg(&parts[i]).x)));
        m = g.max(m);
        s = 0.f;
        for (int64_t i = threadIdx.x; i < a.segs; i += kDrawThreads) {
            const ulonglong2 p = __ldcg(&parts[i]);
            s += __uint_as_float(static_cast<uint32_t>(p.y)) * moved(__uint_as_float(static_cast<uint32_t>(p.x)), m);
        }
        s = g.sum(s);
    }
    __shared__ int state;
    if (threadIdx.x == 0) {
        RowPlan p;
        plan_row<TYPE>(p, m, valid, f);
        if (!valid) flag_bad_id(a.r, c.row);
        state = p.state;
        st.narrow = 0;
        st.listed = 0;
        st.min_value = least_present<TYPE>();
        if (p.state == kDraw) {
            p.shift = p.greedy ? 0 : shift_of(s);
            if (p.greedy) {
                st.min_value = m;
            } else {
                if (f.min_p > 0.f) {
                    st.min_value = least_value<TYPE>(p, f.min_p);
                    p.bound = static_cast<uint64_t>(order_key<TYPE>(st.min_value)) << 32;
                }
                if ((f.top_k > 0 && f.top_k < a.r.cols) || f.top_p < 1.f) st.narrow = kBinned;
            }
        }
        st.plan = p;
        st.cut = {st.min_value, st.min_value, p.bound, 0.f, 0.f};
        st.top_p = fmaxf(f.top_p, 0.f);
        st.top_k = f.top_k;
        // 64 bins a power of two in weight; for top_k, whose place has nothing to do with weights, 128
        // a unit of the logits at most
        const float scale = 64.f * p.ch;
        st.bin_scale = kSlots * fminf(scale, f.top_k > 0 ? 128.f : 0x1p80f);
    }
    __syncthreads();
    if (state != kDraw) no_draws(a, c.row, state, threadIdx.x, kDrawThreads);
}

// exclusive prefix sums over the CTA's threads; `sums` has kDrawWarps + 1 places, the
// last for the total
static __device__ __noinline__ uint64_t cta_scan(uint64_t x, uint64_t *sums) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint64_t upto = warp_scan(x, lane);
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    uint64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kDrawWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    if (threadIdx.x == 0) sums[kDrawWarps] = total;
    __syncthreads();
    return before + upto - x;
}

// FINE: the bins are the slots of the range that the first pass found, where it has more
// entries than are sorted.
template <int TYPE, bool FINE>
__global__ void __launch_bounds__(kDrawThreads, 4) bins_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E, kOwn = kBins / kDrawThreads;
    // (absent entries count behind the last; at the end a thread's bins lie together, its neighbours' one
    // place further, so that they meet no bank twice)
    __shared__ uint32_t count[kBins + kDrawThreads];
    __shared__ uint64_t sums[kDrawWarps + 1], nums[kDrawWarps + 1];
    __shared__ int range[2];
    pdl_trigger();
    for (int i = threadIdx.x; i < kBins; i += kDrawThreads) count[i] = 0;
    pdl_wait();
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    if (st.narrow == 0 || (FINE && st.expected <= kSorted)) return;
    const RowPlan p = st.plan;
    const float bin_scale = st.bin_scale;
    const int64_t k = st.top_k > 0 && st.top_k < a.r.cols ? st.top_k : 0;
    const float top_p = st.top_p;
    const bool by_mass = top_p < 1.f && (!FINE || k == 0);
    // FINE: up to four bins, each slot a bin
    const int first = FINE ? st.slot_lo : 0, last = FINE ? st.slot_hi : kLastSlot;
    const uint32_t above0 = FINE ? st.above : 0;
    if (FINE && last - first >= kBins) return;
    __syncthreads();
    const float unit = !Entry<TYPE>::kReal && p.unit ? __fdiv_rn(1.f, p.m * p.down) : 1.f;
    float rough = 0.f, rough_above = 0.f;
    each_vector<TYPE, kDrawThreads, 4>(c.r, c.lo, c.hi, threadIdx.x, [&](const float (&v)[E], int64_t, int) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int s = slot_of<TYPE>(p, bin_scale, v[i]);
            if (FINE) {
                if (v[i] != absent<TYPE>() && s >= first && s <= last) atomicAdd(&count[s - first], 1u);
                if (by_mass && v[i] != absent<TYPE>()) {
                    const float w = rough_weight<TYPE>(p, v[i]) * unit;
                    rough += w;
                    rough_above += s < first ? w : 0.f;
                }
            } else {
                atomicAdd(&count[v[i] == absent<TYPE>() ? kBins + threadIdx.x % 32 : s / kSlots], 1u);
            }
        }
    });
    // numbers, and weights about: in units of which the row's largest possible sum takes 62 bits
    int log_cols;
    frexpf(static_cast<float>(a.r.cols) * 1.01f, &log_cols);
    if (FINE && by_mass) {
        atomicAdd(&st.rough, static_cast<unsigned long long>(in_units(rough, 61 - log_cols)));
        atomicAdd(&st.rough_above, static_cast<unsigned long long>(in_units(rough_above, 61 - log_cols)));
    }
    __syncthreads();
    RowBins *all = a.segs > 1 ? a.bins + c.row : nullptr;
    if (all) {
        for (int i = threadIdx.x; i < kBins; i += kDrawThreads)
            if (count[i]) atomicAdd(&all->count[i], count[i]);
        if (!last_of_row(a, st, 1)) return;
    }
    const auto middle = [&](int b) {
        if constexpr (Entry<TYPE>::kReal) {
            if (TYPE == TN_TYPE_BF16 && !FINE) {
                // a bin may hold one or two of the type's values only: those
                const float around = __bfloat162float(__float2bfloat16_rn(p.m - (b + 0.5f) * kSlots / bin_scale));
                float s = 0.f;
                int n = 0;
                for (int i = -2; i <= 2; ++i) {
                    const float v = key_value(order_key<TYPE>(around) + (i << 16));
                    if (slot_of<TYPE>(p, bin_scale, v) / kSlots != b) continue;
                    s += ex2((v - p.m) * p.ch);
                    ++n;
                }
                if (n > 0 && n < 5) return s / n;
            }
            return ex2(-(FINE ? first + b + 0.5f : (b + 0.5f) * kSlots) * p.ch / bin_scale);
        } else {
            const float d = (FINE ? first + b + 0.5f : (b + 0.5f) * kSlots) * 128.f;
            const uint32_t top = __float_as_uint(p.m), down = static_cast<uint32_t>(d);
            const float q = down < top ? __uint_as_float(top - down) / p.m : 0.f;
            return p.unit ? q : q > 0.f ? ex2(p.beta * log2_of(q)) : 0.f;
        }
    };
    // (rolled, and weights computed again, here and below: the streaming loop wants its registers)
    const auto number = [&](int b) { return count[b + b / kOwn]; };
    const auto mass_of = [&](int b) -> uint64_t {
        return by_mass && number(b) ? number(b) * in_units(middle(b), 61 - log_cols) : 0;
    };
    {
        uint32_t n[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int b = threadIdx.x + i * kDrawThreads;
            n[i] = all ? __ldcg(&all->count[b]) : count[b];
            if (all) all->count[b] = 0;     // left clear
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int b = threadIdx.x + i * kDrawThreads;
            count[b + b / kOwn] = n[i];
        }
        __syncthreads();
    }
    uint64_t own_mass = 0, own_count = 0;
#pragma unroll 1
    for (int i = 0; i < kOwn; ++i) {
        const int b = threadIdx.x * kOwn + i;
        own_mass += mass_of(b);
        own_count += number(b);
    }
    const uint64_t before_mass = cta_scan(own_mass, sums), before_count = cta_scan(own_count, nums);
    const uint64_t entries = nums[kDrawWarps];
    const bool cut_k = FINE ? k > 0 : k > 0 && static_cast<uint64_t>(k) < entries;
    // both filters: the second needs all that the first leaves, so all from the top is listed
    const bool both = cut_k && top_p < 1.f;
    if (!cut_k && !by_mass) {       // fewer entries than top_k
        if (threadIdx.x == 0) st.narrow = 0;
        return;
    }
    // FINE: the weights above the bins and of all, better known by now than from bins' middles
    const uint64_t total = FINE ? __ldcg(&st.rough) : sums[kDrawWarps];
    uint64_t target = cut_k ? k : share(top_p, total, false);
    const uint64_t base = cut_k ? above0 : FINE ? __ldcg(&st.rough_above) : 0;
    // the bins that meet the target give or take the error of their middles (that of exponentials
    // in fp32, where those do not count), less of it where those hold too many
    constexpr int kOff = FINE ? 17 : 10;
    const bool again = !FINE && a.r.cols >= kLongRow;       // (four bins are looked into once more)
    uint32_t expected = 0, above = 0;
    for (int round = 0; round < 4; ++round) {
        const uint64_t off = cut_k || round == 3 ? 0 : total >> (kOff + 2 * round);
        __syncthreads();
        if (threadIdx.x == 0) {
            range[0] = kBins;
            range[1] = -1;
        }
        __syncthreads();
        uint64_t x = base + (cut_k ? before_count : before_mass);
        int lo = kBins, hi = -1;
        if (x <= target + off && x + (cut_k ? own_count : own_mass) + off >= target) {
#pragma unroll 1
            for (int i = 0; i < kOwn; ++i) {
                const int b = threadIdx.x * kOwn + i;
                const uint64_t next = x + (cut_k ? number(b) : mass_of(b));
                if (number(b) && next + off >= target && x <= target + off && (cut_k ? x < target : true)) {
                    if (lo == kBins) lo = b;
                    hi = b;
                }
                x = next;
            }
        }
        if (lo < kBins) {
            atomicMin(&range[0], lo);
            atomicMax(&range[1], hi);
        }
        __syncthreads();
        if (range[1] < 0) range[1] = -1;        // (none: past all of them)
        const int r0 = both ? 0 : range[0], r1 = range[1];
        // what lies above the range and in it: the thread with its first and the one with its last bin know
        __shared__ uint64_t at_range[2];
        if (threadIdx.x == 0) at_range[0] = at_range[1] = 0;
        __syncthreads();
        if (r1 >= 0 && (threadIdx.x == r0 / kOwn || threadIdx.x == r1 / kOwn)) {
            uint64_t n = before_count;
            for (int b = threadIdx.x * kOwn; b < (static_cast<int>(threadIdx.x) + 1) * kOwn; ++b) {
                if (b == r0) at_range[0] = n;
                n += number(b);
                if (b == r1) at_range[1] = n;
            }
        }
        __syncthreads();
        above = static_cast<uint32_t>(at_range[0]);
        expected = static_cast<uint32_t>(at_range[1] - at_range[0]);
        if (cut_k || (range[1] >= 0 && (expected <= kSorted || (again && range[1] - range[0] < kBins / kSlots)))) break;
    }
    // Too many from the top to top_k's bin: a range of its own for top_p, whose whole is the weight of
    // top_k entries, and top_k's bin as a second one where that does not reach it.
    bool two = false;
    int k_bin = 0;
    uint32_t above2 = 0;
    if (both && !FINE && expected > kSorted) {
        k_bin = range[1];
        __shared__ uint64_t at_bin[2];
        if (threadIdx.x == k_bin / kOwn) {
            uint64_t n = before_count, w = before_mass;
            for (int b = threadIdx.x * kOwn; b < k_bin; ++b) {
                n += number(b);
                w += mass_of(b);
            }
            at_bin[0] = n;
            at_bin[1] = w + mass_of(k_bin) / number(k_bin) * (k - n);
        }
        __syncthreads();
        above2 = static_cast<uint32_t>(at_bin[0]);
        target = share(top_p, at_bin[1], false);
        for (int round = 0; round < 4; ++round) {
            const uint64_t off = round == 3 ? 0 : at_bin[1] >> (10 + 2 * round);
            __syncthreads();
            if (threadIdx.x == 0) {
                range[0] = kBins;
                range[1] = -1;
            }
            __syncthreads();
            uint64_t x = before_mass, n = before_count;
#pragma unroll 1
            for (int i = 0; i < kOwn; ++i) {
                const int b = threadIdx.x * kOwn + i;
                if (b > k_bin) break;
                const uint64_t next = x + mass_of(b);
                if (number(b) && ((next + off >= target && x <= target + off) || b == k_bin)) {
                    // (the range's ends with the entries before and through them)
                    if (b < k_bin || x <= target + off) {
                        atomicMin(&range[0], b);
                        atomicMax(&range[1], b);
                    }
                }
                x = next;
                n += number(b);
            }
            __syncthreads();
            const int r0 = range[0], r1 = range[1];
            if (r1 < 0) continue;
            __shared__ uint64_t ends[3];
            if (threadIdx.x == r0 / kOwn || threadIdx.x == r1 / kOwn || threadIdx.x == k_bin / kOwn) {
                n = before_count;
                for (int b = threadIdx.x * kOwn; b < (static_cast<int>(threadIdx.x) + 1) * kOwn; ++b) {
                    if (b == r0) ends[0] = n;
                    n += number(b);
                    if (b == r1) ends[1] = n;
                    if (b == k_bin) ends[2] = number(b);
                }
            }
            __syncthreads();
            above = static_cast<uint32_t>(ends[0]);
            two = r1 < k_bin;
            expected = static_cast<uint32_t>(ends[1] - ends[0] + (two ? ends[2] : 0));
            if (expected <= kSorted) break;
        }
        if (expected > kSorted) two = false;
    }
    const bool from_top = both && (FINE || expected > kSorted || above2 == 0);
    __shared__ int slots[2];
    if (threadIdx.x == 0) {
        const int r0 = from_top ? 0 : range[0], r1 = range[1];
        const bool none = r1 < 0 || r0 > r1;
        if (none) expected = 0xffffffffu;       // digit by digit
        st.slot_lo = slots[0] = none ? 0 : FINE ? (from_top ? 0 : first + r0) : r0 * kSlots;
        st.slot_hi = slots[1] = none ? kLastSlot : FINE ? first + r1 : r1 * kSlots + kSlots - 1;
        st.expected = both && FINE ? expected + above0 : expected;
        st.above = from_top ? 0 : above0 + above;
        st.two = two;
        st.above2 = above2;
        if (!cut_k) st.top_k = 0;
        st.narrow = kListed;
    }
    __syncthreads();
    // order values instead of slots; and where min_p cuts above the range, nothing else does
    __shared__ float values[4];
    const int lo = slots[0], hi = slots[1];
    if (threadIdx.x % 32 == 0 && threadIdx.x < 128) {
        const int which = threadIdx.x / 32;
        const int slot = which == 0 ? lo : which == 1 ? hi + 1 : (k_bin + which - 2) * kSlots;
        values[which] = which > 1 && !two ? 0.f : slot > kLastSlot ? least_present<TYPE>() : slot_begin<TYPE>(p, bin_scale, slot);
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    st.cut = {values[0], values[1], 0, values[2], values[3]};
    if (p.bound > kPresent && slot_of<TYPE>(p, bin_scale, st.min_value) < lo) {
        st.narrow = 0;
        st.cut = {st.min_value, st.min_value, p.bound, 0.f, 0.f};
    }
}

// Ranks in descending order, n (a power of two) of them; every warp has a part of its own, so that
// only the few steps that are longer need the CTA's barrier.
__device__ __forceinline__ void sort_ranks(uint64_t *x, int n) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int own = n / 2 / kDrawWarps;         // pairs of a warp
    bool far = true;
    __syncthreads();
    for (int size = 2; size <= n; size *= 2)
        for (int step = size / 2; step; step /= 2) {
            const bool now = own < 32 || step > own;
            if (now || far) __syncthreads();
            else __syncwarp();
            far = now;
            const auto pair = [&](int t) {
                const int i = 2 * t - (t & (step - 1)), j = i + step;
                const uint64_t y = x[i], z = x[j];
                if ((y < z) == ((i & size) == 0)) {
                    x[i] = z;
                    x[j] = y;
                }
            };
            if (own < 32) {
                if (threadIdx.x < n / 2) pair(threadIdx.x);
            } else {
                for (int t = lane; t < own; t += 32) pair(warp * own + t);
            }
        }
    __syncthreads();
}

// A row's list (in shared memory, room for a power of two): the rank where the filters cut, and what is
// left of the list joins its pieces (and segments).  Returns the bound, 0 where the cut
// does not lie in the list after all; `more` and `joined`: weight and number of what joined.
template <int TYPE>
__device__ __noinline__ uint64_t cut_list(const RowState &st, uint64_t *list, int n, const float *roots, uint64_t above,
                                          uint64_t below, int head, int64_t pieces, int64_t seg_pieces, uint64_t *masses,
                                          ulonglong2 *parts, uint64_t *sums, uint64_t &more, uint64_t &joined) {
    constexpr int E = Entry<TYPE>::E, kOwn = kSorted / kDrawThreads;
    const RowPlan p = st.plan;
    int room = 2;
    while (room < n) room *= 2;
    for (int i = n + threadIdx.x; i < room; i += kDrawThreads) list[i] = 0;
    sort_ranks(list, room);
    int64_t left = n, last = n;         // entries that top_k leaves, and among which top_p cuts
    if (st.two) {
        // the first range's, then as many of the second as top_k takes
        const uint64_t end = static_cast<uint64_t>(order_key<TYPE>(st.cut.list)) << 32;
        __shared__ int in_first;
        if (threadIdx.x == 0) in_first = 0;
        __syncthreads();
        int mine = 0;
        for (int i = threadIdx.x; i < n; i += kDrawThreads) mine += list[i] >= end;
        atomicAdd(&in_first, mine);
        __syncthreads();
        last = in_first;
        left = last + st.top_k - static_cast<int64_t>(st.above2);
        if (left > n || left <= last) return 0;
    } else if (st.top_k > 0) {
        last = left = st.top_k - static_cast<int64_t>(st.above);
        if (left > n || left < 1) return 0;
    }
    // of consecutive ranks, a thread each; equal keys have equal weights
    const int per = (n + kDrawThreads - 1) / kDrawThreads, lo = threadIdx.x * per;
    uint64_t w[kOwn], own = 0;
    uint32_t key = 0;
    uint64_t same = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        w[i] = 0;
        if (i >= per || lo + i >= n) continue;
        const uint32_t k = static_cast<uint32_t>(list[lo + i] >> 32);
        if (k != key) same = weight_once<TYPE>(p, roots, key_value(k));
        key = k;
        w[i] = same;
        if (lo + i < left) own += same;
    }
    uint64_t bound = left > 0 ? list[left - 1] : kPresent;
    if (st.top_p < 1.f) {
        __shared__ uint64_t found;
        if (threadIdx.x == 0) found = 0;
        uint64_t upto = above + cta_scan(own, sums);
        const uint64_t in = sums[kDrawWarps];
        // of all that top_k leaves, or of all (equal entries' weights as they are added up here)
        uint64_t target = share(st.top_p, above + in + below, true);
        if (target == 0) target = 1;
        if (target <= above || target > above + in) return 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (i >= per || lo + i >= last) continue;
            if (upto < target && upto + w[i] >= target) found = list[lo + i];
            upto += w[i];
        }
        __syncthreads();
        bound = found;
        if (bound == 0) return 0;
    }
    if (p.bound > bound) bound = p.bound;
    uint64_t mass = 0, num = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        if (i >= per || lo + i >= n || list[lo + i] < bound) continue;
        const int64_t e = 0xffffffffu - static_cast<uint32_t>(list[lo + i]);
        const int64_t q = (e + head) / E / kPieceVecs;
        if (q >= pieces) continue;      // (a workspace that others wrote to)
        atomicAdd(reinterpret_cast<unsigned long long *>(&masses[q]), static_cast<unsigned long long>(w[i]));
        if (parts) atomicAdd(reinterpret_cast<unsigned long long *>(&parts[q / seg_pieces].x), static_cast<unsigned long long>(w[i]));
        mass += w[i];
        ++num;
    }
    cta_scan(mass, sums);
    more = sums[kDrawWarps];
    cta_scan(num, sums);
    joined = sums[kDrawWarps];
    return bound;
}

// The same of a range whose entries all have the key `key`, by their numbers in the pieces (`ties`): of equal
// entries the first ones are left.  kept: how many lie above the range.
template <int TYPE>
__device__ __noinline__ uint64_t cut_ties(const RowState &st, const Segment<TYPE> &c, uint32_t key, const float *roots,
                                          uint64_t above, uint64_t below, uint64_t kept, int64_t pieces, int64_t seg_pieces,
                                          uint64_t *masses, const uint32_t *ties, ulonglong2 *parts, uint64_t *sums,
                                          uint64_t &more, uint64_t &joined) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ uint64_t cut_need, cut_bound;
    __shared__ int64_t cut_piece;
    if (st.two) return 0;
    const RowPlan p = st.plan;
    const int64_t per = (pieces + kDrawThreads - 1) / kDrawThreads, lo = threadIdx.x * per;
    const int64_t hi = lo + per < pieces ? lo + per : pieces;
    uint64_t own = 0;
    for (int64_t q = lo; q < hi; ++q) own += __ldcg(&ties[q]);
    uint64_t before = cta_scan(own, sums);
    uint64_t need = sums[kDrawWarps];
    const uint64_t w = weight_once<TYPE>(p, roots, key_value(key));
    if (st.top_k > 0) {
        if (static_cast<uint64_t>(st.top_k) <= kept || st.top_k - kept > need) return 0;
        need = st.top_k - kept;
    }
    if (st.top_p < 1.f) {
        uint64_t target = share(st.top_p, above + need * w + below, true);
        if (target == 0) target = 1;
        if (target <= above || target > above + need * w) return 0;
        need = (target - above + w - 1) / w;
    }
    if (p.bound > kPresent && p.bound >> 32 > key) return p.bound;      // (min_p leaves none of them)
    for (int64_t q = lo; q < hi && before < need; ++q) {
        const uint64_t n = __ldcg(&ties[q]), take = n < need - before ? n : need - before;
        if (take > 0) {
            // (past the L1 cache, which may hold the line as another row's CTA found it)
            atomicAdd(reinterpret_cast<unsigned long long *>(&masses[q]), static_cast<unsigned long long>(take * w));
            if (parts) atomicAdd(reinterpret_cast<unsigned long long *>(&parts[q / seg_pieces].x), static_cast<unsigned long long>(take * w));
        }
        before += n;
        if (before >= need) {
            cut_piece = q;
            cut_need = take;
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        uint64_t upto = 0;
        for (int i = 0; i < kPieceVecs / 32; ++i) {
            const int64_t j = cut_piece * kPieceVecs + i * 32 + threadIdx.x;
            float v[E];
            uint64_t n = 0;
            if (j < c.vecs) {
                vector_values<TYPE>(c.r, j, v);
#pragma unroll
                for (int k = 0; k < E; ++k) n += order_key<TYPE>(v[k]) == key;
            }
            uint64_t at = upto + warp_scan(n, threadIdx.x) - n;
            upto = shfl_from(at + n, 31);
            if (j < c.vecs) {
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (order_key<TYPE>(v[k]) == key && ++at == cut_need) cut_bound = rank_of<TYPE>(v[k], j * E - c.r.head + k);
            }
        }
    }
    __syncthreads();
    more = need * w;
    joined = need;
    return cut_bound;
}

// More equal (or nearly equal) entries than are sorted, or a cut elsewhere: digit by digit, and the
// row's sums by this CTA, whose totals are left in the scans' last places.
template <int TYPE>
__device__ __noinline__ Cut by_digits(const SampleArgs &a, const Segment<TYPE> &c, const RowState &st, const RowPlan &p,
                                      const float *roots, Select *sel, uint64_t *masses, ulonglong2 *parts,
                                      int64_t pieces, uint64_t *sums, uint64_t *nums) {
    constexpr int E = Entry<TYPE>::E;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const RowCta<TYPE> cta{c.r, c.vecs, &p, roots, sel, sums};
    const Cut cut = {__builtin_huge_valf(), least_present<TYPE>(),
                     bound_of<TYPE>(cta, p, st.top_k, st.top_p), 0.f, 0.f};
    uint64_t total = 0, kept = 0;
    for (int64_t q = warp; q < pieces; q += kDrawWarps) {
        uint64_t own = 0;
        for (int i = 0; i < kPieceVecs / 32; ++i) {
            const int64_t j = q * kPieceVecs + i * 32 + lane;
            if (j >= c.vecs) break;
            float v[E];
            vector_values<TYPE>(c.r, j, v);
            own += vector_weight<TYPE>(p, cut, roots, v, j * E - c.r.head);
#pragma unroll
            for (int k = 0; k < E; ++k) kept += is_left<TYPE>(cut, v[k], j * E - c.r.head + k);
        }
        total += own;
        own = warp_sum(own);
        if (lane == 0) __stcg(&masses[q], own);
    }
    if (parts) {
        __threadfence();
        __syncthreads();
        for (int i = threadIdx.x; i < a.segs; i += kDrawThreads) {
            uint64_t own = 0;
            for (int64_t q = i * a.seg_pieces; q < (i + 1) * a.seg_pieces && q < pieces; ++q) own += __ldcg(&masses[q]);
            __stcg(&parts[i], make_ulonglong2(own, 0));
        }
    }
    cta_scan(total, sums);
    cta_scan(kept, nums);
    return cut;
}

// FILTERED: rows may have lists.
template <int TYPE, bool FILTERED>
__global__ void __launch_bounds__(kDrawThreads, 4) sums_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = Entry<TYPE>::E;
    __shared__ float roots[2 * kRoots];
    __shared__ uint64_t list[FILTERED ? kSorted : 1];
    __shared__ Select sel;
    __shared__ uint64_t sums[kDrawWarps + 1], nums[kDrawWarps + 1];
    __shared__ uint32_t listed;
    pdl_trigger();
    if (Entry<TYPE>::kReal || a.powers) make_roots<kDrawThreads>(roots);
    if (threadIdx.x == 0) listed = 0;
    pdl_wait();
    const Segment<TYPE> c(a);
    RowState &st = a.state[c.row];
    const RowPlan p = st.plan;
    if (p.state != kDraw) return;
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // (on its way early: whichever CTA ends the row makes the draws)
    const double u = a.draws <= kFewDraws && warp < a.draws ? random_number(a, c.row * a.draws + warp) : 0.0;
    uint64_t *masses = a.masses + c.row * a.pieces;
    const bool lists = FILTERED && st.narrow == kListed, passes = !lists || st.expected != 0xffffffffu;
    // too many for a list: if all of the range are equal, pieces' numbers of them will do
    const bool tied = lists && st.expected > kSorted, sorted = passes && !tied;
    uint32_t *ties = FILTERED ? a.ties + c.row * a.pieces : nullptr;
    uint32_t key_hi = 0, key_not = 0;
    // the weight of what lies below the range is wanted, all of it or as far as the second range
    const bool two = lists && st.two, by_mass = lists && st.top_p < 1.f && (st.top_k <= 0 || two);
    Cut cut = st.cut;
    const float lowest = two ? cut.gate2 : least_present<TYPE>();
    uint64_t *to = a.segs > 1 ? a.lists + c.row * kSorted : list;
    uint32_t *counter = a.segs > 1 ? &st.listed : &listed;
    uint64_t total = 0, all = 0;
    uint32_t number = 0;
    if (passes) {
        int64_t in_lo, in_hi;
        c.r.inside_range(in_lo, in_hi);
#pragma unroll 1
        for (int64_t q = c.lo / kPieceVecs + 2 * warp; q * kPieceVecs < c.hi; q += 2 * kDrawWarps) {
            // two pieces, their loads in flight together
            uint64_t both[2] = {0, 0};
            uint32_t in_piece[2] = {0, 0};
            vectors_at<TYPE, 2 * kPieceVecs / 32>(
                c.r, in_lo, in_hi, q * kPieceVecs, (q + 2) * kPieceVecs, q * kPieceVecs + lane, 32, c.hi,
                [&](const float (&v)[E], int64_t j, int which) {
                    uint64_t own = 0;
                    uint32_t in = 0;
                    if constexpr (Entry<TYPE>::kReal) {
                        PairSum sum, whole;
                        uint32_t n = 0;
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            const bool above = v[k] >= cut.gate, below = !(v[k] >= cut.list);
                            n += above;
                            if constexpr (FILTERED)
                                in |= static_cast<uint32_t>(!above && (!below || (two && v[k] < cut.gate2 && v[k] >= cut.list2))) << k;
                        }
                        if (n || (FILTERED && by_mass)) {
#pragma unroll (FILTERED ? 4 : 8)
                            for (int k = 0; k < E; k += 2) {
                                const bool above0 = v[k] >= cut.gate, above1 = v[k + 1] >= cut.gate;
                                if constexpr (FILTERED) {
                                    const Weights w = weight_pairs(p, roots, v[k], v[k + 1], v[k] != absent<TYPE>(),
                                                                   v[k + 1] != absent<TYPE>());
                                    const float2 f = make_float2(above0 ? 1.f : 0.f, above1 ? 1.f : 0.f);
                                    sum.add(mul2(w.hi, f), mul2(w.lo, f));
                                    if (by_mass) {
                                        const float2 c = make_float2(v[k] < cut.list && v[k] >= lowest ? 1.f : 0.f,
                                                                     v[k + 1] < cut.list && v[k + 1] >= lowest ? 1.f : 0.f);
                                        whole.add(mul2(w.hi, c), mul2(w.lo, c));
                                    }
                                } else {
                                    const Weights w = weight_pairs(p, roots, v[k], v[k + 1], above0, above1);
                                    sum.add(w.hi, w.lo);
                                }
                            }
                            if (FILTERED && by_mass) all += whole.units(p.shift);
                        }
                        own += sum.units(p.shift) + n;
                        number += n;
                    } else {
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            const bool above = v[k] >= cut.gate, below = !(v[k] >= cut.list);
                            const bool second = FILTERED && two && v[k] < cut.gate2 && v[k] >= cut.list2;
                            if (FILTERED && !above && (!below || second)) in |= 1u << k;
                            const bool counts = FILTERED && by_mass && below && v[k] >= lowest;
                            if (!above && !counts) continue;
                            const uint64_t w = weight<TYPE>(p, roots, v[k]);
                            own += above ? w : 0;
                            number += above;
                            all += counts ? w : 0;
                        }
                    }
                    both[0] += which < kPieceVecs / 32 ? own : 0;
                    both[1] += which < kPieceVecs / 32 ? 0 : own;
                    if (!FILTERED || !lists || !in) return;
                    if (tied) {
                        in_piece[0] += which < kPieceVecs / 32 ? __popc(in) : 0;
                        in_piece[1] += which < kPieceVecs / 32 ? 0 : __popc(in);
#pragma unroll 1
                        for (uint32_t rest = in; rest; rest &= rest - 1) {
                            const int at = __ffs(rest) - 1;
                            float x = v[0];
#pragma unroll
                            for (int k = 1; k < E; ++k) x = k == at ? v[k] : x;
                            const uint32_t key = order_key<TYPE>(x);
                            key_hi = max(key_hi, key);
                            key_not = max(key_not, ~key);
                        }
                        return;
                    }
                    uint32_t at = atomicAdd(counter, static_cast<uint32_t>(__popc(in)));
#pragma unroll
                    for (int k = 0; k < E; ++k)
                        if (in >> k & 1) {
                            if (at < kSorted) to[at] = rank_of<TYPE>(v[k], j * E - c.r.head + k);
                            ++at;
                        }
                });
            total += both[0] + both[1];
            both[0] = warp_sum(both[0]);
            both[1] = warp_sum(both[1]);
            if (lane == 0) {
                __stcg(&masses[q], both[0]);
                if ((q + 1) * kPieceVecs < c.hi) __stcg(&masses[q + 1], both[1]);
            }
            if (FILTERED && tied) {
                in_piece[0] = __reduce_add_sync(0xffffffffu, in_piece[0]);
                in_piece[1] = __reduce_add_sync(0xffffffffu, in_piece[1]);
                if (lane == 0) {
                    __stcg(&ties[q], in_piece[0]);
                    if ((q + 1) * kPieceVecs < c.hi) __stcg(&ties[q + 1], in_piece[1]);
                }
            }
        }
    }
    if (FILTERED && tied && passes) {
        key_hi = __reduce_max_sync(0xffffffffu, key_hi);
        key_not = __reduce_max_sync(0xffffffffu, key_not);
        if (lane == 0) {
            atomicMax(&st.key_hi, key_hi);
            atomicMax(&st.key_not, key_not);
        }
    }
    cta_scan(total, sums);
    cta_scan(number, nums);
    total = sums[kDrawWarps];
    uint64_t kept = nums[kDrawWarps];
    if (by_mass) {
        cta_scan(all, sums);
        all = sums[kDrawWarps];
    }
    ulonglong2 *parts = nullptr;
    const int per = static_cast<int>((a.segs + kDrawThreads - 1) / kDrawThreads), s0 = threadIdx.x * per;
    if (a.segs > 1) {
        parts = a.partials + c.row * a.segs;
        uint64_t *alls = a.alls + c.row * a.segs;
        if (threadIdx.x == 0) {
            __stcg(&parts[c.seg], make_ulonglong2(total, kept));
            if (by_mass) __stcg(&alls[c.seg], all);
        }
        if (!last_of_row(a, st, 2)) return;
        total = kept = all = 0;
        for (int i = s0; i < s0 + per && i < a.segs; ++i) {
            const ulonglong2 x = __ldcg(&parts[i]);
            total += x.x;
            kept += x.y;
            if (by_mass) all += __ldcg(&alls[i]);
        }
        cta_scan(kept, nums);
        cta_scan(total, sums);
        total = sums[kDrawWarps];
        kept = nums[kDrawWarps];
        if (by_mass) {
            cta_scan(all, sums);
            all = sums[kDrawWarps];
        }
    } else {
        if (FILTERED && tied) __threadfence();
        __syncthreads();        // the pieces' sums and the list
    }
    const int64_t pieces = (c.vecs + kPieceVecs - 1) / kPieceVecs;
    if constexpr (FILTERED) if (lists) {
        uint64_t bound = 0;
        const uint32_t found = sorted ? (a.segs > 1 ? __ldcg(&st.listed) : listed) : 0;
        if (sorted && found <= kSorted) {
            if (a.segs > 1) {
                for (int i = threadIdx.x; i < found; i += kDrawThreads) list[i] = __ldcg(&to[i]);
                __syncthreads();
            }
            uint64_t more = 0, joined = 0;
            bound = cut_list<TYPE>(st, list, found, roots, total, all, c.r.head, pieces, a.seg_pieces, masses, parts, sums,
                                   more, joined);
            total += more;
            kept += joined;
            cut.bound = bound;
        }
        const uint32_t key = tied && passes ? __ldcg(&st.key_hi) : 0;
        if (key != 0 && key == ~__ldcg(&st.key_not)) {
            uint64_t more = 0, joined = 0;
            bound = cut_ties<TYPE>(st, c, key, roots, total, all, kept, pieces, a.seg_pieces, masses, ties, parts, sums, more,
                                   joined);
            total += more;
            kept += joined;
            cut.bound = bound;
        }
        if (bound == 0) {
            cut = by_digits<TYPE>(a, c, st, p, roots, &sel, masses, parts, pieces, sums, nums);
            total = sums[kDrawWarps];
            kept = nums[kDrawWarps];
        }
    }
    __threadfence();
    __syncthreads();
    if (FILTERED && threadIdx.x == 0) {
        st.key_hi = st.key_not = 0;
        st.rough = st.rough_above = 0;
    }
    // sums up to each segment, of consecutive ones by a thread each
    __shared__ uint64_t upto_segment[kDrawThreads];
    const bool few = a.segs <= kDrawThreads;
    if (parts) {
        uint64_t own = 0;
        for (int i = s0; i < s0 + per && i < a.segs; ++i) own += __ldcg(&parts[i]).x;
        uint64_t upto = cta_scan(own, sums);
        for (int i = s0; i < s0 + per && i < a.segs; ++i) {
            upto += few ? own : __ldcg(&parts[i]).x;
            if (few) upto_segment[i] = upto;
            if (!few || a.draws > kFewDraws) __stcg(&parts[i], make_ulonglong2(upto, 0));
        }
    }
    if (threadIdx.x == 0) {
        a.kept[c.row] = p.greedy ? 1 : static_cast<int64_t>(kept);
        st.total = total;
        st.cut = cut;
        st.listed = 0;
    }
    if (!few) __threadfence();
    __syncthreads();
    if (a.draws > kFewDraws) return;
    for (int64_t d = warp; d < a.draws; d += kDrawWarps) {
        const int64_t at = c.row * a.draws + d;
        uint64_t target;
        if (!aim(a, d < kDrawWarps ? u : random_number(a, at), p.greedy, total, at, c.row, target)) continue;
        int64_t first = 0, n = pieces;
        if (parts) {
            first = few ? locate_upto([&](int64_t i) { return upto_segment[i]; }, a.segs, target)
                        : locate_upto([&](int64_t i) -> uint64_t { return __ldcg(&parts[i]).x; }, a.segs, target);
            first *= a.seg_pieces;
            n = pieces - first < a.seg_pieces ? pieces - first : a.seg_pieces;
        }
        LogP l;
        l.of(p, total, warp_draw<TYPE>(a, c.r, c.vecs, p, cut, roots, masses, first, n, target, at));
        if (lane == 0) a.logp[at] = log_p<TYPE>(l);
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kDrawThreads) draws_kernel(const __grid_constant__ SampleArgs a) {
    __shared__ float roots[2 * kRoots];
    pdl_trigger();
    if (Entry<TYPE>::kReal || a.powers) make_roots<kDrawThreads>(roots);
    pdl_wait();
    __syncthreads();
    const int64_t ctas = (a.draws + kDrawWarps - 1) / kDrawWarps;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t row = blockIdx.x / ctas, d0 = (blockIdx.x - row * ctas) * kDrawWarps, d = d0 + warp;
    const RowState &st = a.state[row];
    const RowPlan p = st.plan;
    if (p.state != kDraw) return;
    __shared__ float values[kDrawWarps];
    __shared__ bool drawn[kDrawWarps];
    uint64_t target = 0;
    const int64_t at = row * a.draws + d;
    const bool valid = d < a.draws && aim(a, random_number(a, at), p.greedy, st.total, at, row, target);
    if (lane == 0) drawn[warp] = valid;
    if (valid) {
        const Row<TYPE> r(a.r, row);
        const int64_t vecs = (r.head + r.cols + Entry<TYPE>::E - 1) / Entry<TYPE>::E;
        int64_t first = 0, n = (vecs + kPieceVecs - 1) / kPieceVecs;
        if (a.segs > 1) {
            const ulonglong2 *parts = a.partials + row * a.segs;
            first = locate_upto([&](int64_t i) -> uint64_t { return __ldcg(&parts[i]).x; }, a.segs, target) * a.seg_pieces;
            n = n - first < a.seg_pieces ? n - first : a.seg_pieces;
        }
        const float v = warp_draw<TYPE>(a, r, vecs, p, st.cut, roots, a.masses + row * a.pieces, first, n, target, at);
        if (lane == 0) values[warp] = v;
    }
    __syncthreads();
    if (threadIdx.x < kDrawWarps && drawn[threadIdx.x]) {       // all logarithms in one warp
        LogP l;
        l.of(p, st.total, values[threadIdx.x]);
        a.logp[row * a.draws + d0 + threadIdx.x] = log_p<TYPE>(l);
    }
}

template <int TYPE, int N, int NT>
cudaError_t launch_held(const SampleArgs &a, cudaStream_t stream) {
    constexpr int THREADS = NT == 32 ? kDrawThreads : NT, ROWS = THREADS / NT;
    const int64_t groups = (a.r.rows + ROWS - 1) / ROWS, most = kDrawTarget * (kDrawThreads / THREADS);
    return launch_pdl(held_rows_kernel<TYPE, N, NT, false>, dim3(static_cast<unsigned>(groups < most ? groups : most)),
                      dim3(THREADS), 0, stream, a);
}
template <int TYPE>
cudaError_t launch_ranks(const SampleArgs &a, int ranks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.r.rows * ranks));
    cfg.blockDim = dim3(kDrawThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, held_rows_kernel<TYPE, kHeldEntries, kDrawThreads, true>, a);
}

template <int TYPE>
cudaError_t sample_of(const SampleArgs &a, cudaStream_t stream) {
    constexpr int E = Entry<TYPE>::E;
    const bool aligned = a.r.col_stride != 1 || (reinterpret_cast<uintptr_t>(a.r.data) % 16 == 0 &&
                                                 a.r.row_stride % E == 0);
    const int64_t entries = (a.r.cols + (aligned ? 0 : E - 1) + E - 1) / E * E;
    if (!a.state) {
        // a warp a row where its registers hold it, otherwise the least CTA that does
        constexpr int kFew = E == 8 ? 8 : 4, N = kHeldEntries;
        if (entries <= 32 * kFew) return launch_held<TYPE, kFew, 32>(a, stream);
        if (entries <= 32 * N) return launch_held<TYPE, N, 32>(a, stream);
        if (entries <= 64 * N) return launch_held<TYPE, N, 64>(a, stream);
        if constexpr (E > 2)
            if (entries <= 128 * N) return launch_held<TYPE, N, 128>(a, stream);
        if constexpr (E > 4)
            if (entries <= 256 * N) return launch_held<TYPE, N, 256>(a, stream);
        return cudaErrorInvalidValue;       // (rows of more than kRowVecs vectors have a state)
    }
    // Few rows that a cluster holds: one kernel instead of three, at the price of a barrier of the
    // cluster for every sum.  bf16, by clusters and in segments, us without filters, with top_k, top_p and
    // both: 40 x 32768 22, 44, 56, 62 and 28, 51, 76, 62; 154 x 8192 19, 37, 43, 60 and 28, 58, 80, 69;
    // 76 x 32768 33, 74, 89, 119 and 32, 57, 87, 68.
    int ranks = 2;
    while (ranks <= kMostRanks && entries > ranks * kDrawThreads * kHeldEntries) ranks *= 2;
    const bool both = (a.f.top_ks || a.f.top_k > 0) && (a.f.top_ps || a.f.top_p < 1.f);
    if (ranks <= kMostRanks && a.r.rows * ranks <= (both ? 2 : 3) * kOutSms && a.draws <= 2 * kFewDraws)
        return launch_ranks<TYPE>(a, ranks, stream);
    const dim3 block(kDrawThreads), grid(static_cast<unsigned>(a.r.rows * a.segs));
    cudaError_t e = launch_pdl(top_kernel<TYPE>, grid, block, 0, stream, a);
    if (e == cudaSuccess && a.filtered) {
        e = launch_pdl(bins_kernel<TYPE, false>, grid, block, 0, stream, a);
        if (e == cudaSuccess && a.r.cols >= kLongRow)
            e = launch_pdl(bins_kernel<TYPE, true>, grid, block, 0, stream, a);
    }
    if (e == cudaSuccess)
        e = a.filtered ? launch_pdl(sums_kernel<TYPE, true>, grid, block, 0, stream, a)
                       : launch_pdl(sums_kernel<TYPE, false>, grid, block, 0, stream, a);
    if (e == cudaSuccess && a.draws > kFewDraws) {
        const int64_t ctas = a.r.rows * ((a.draws + kDrawWarps - 1) / kDrawWarps);
        e = launch_pdl(draws_kernel<TYPE>, dim3(static_cast<unsigned>(ctas)), block, 0, stream, a);
    }
    return e;
}

}  // namespace tn
