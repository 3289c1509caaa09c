// Shared pieces of the tensor-core gated delta rule (la_tc_delta.cu, la_tc_delta_bwd.cu): the image of a
// chunk's matrices that the preparing kernel leaves for the scans, and small device helpers.
//
// In a chunk of C = 64 tokens with G the running sum of g and D_ij = exp(G_i - G_j) (j <= i), the
// errors E of the chunk's writes solve a unit lower triangular system,
//   E = T (V - exp(G) K S) = T V + W S,   T = (I + N diag(beta))^-1,  N = tril(D (K K^T), -1),  W = -T exp(G) K,
// and with U = beta E:  O = scale (exp(G) Q S + P U),  S' = exp(G_C) S + K^T exp(G_C - G) U,  P = tril(D (Q K^T))
// (exp(G) and exp(G_C - G) scale rows).  The way back through a chunk, of R = dL/dS', has the same form,
//   dX = Z^T dO + W2 R,   Z = scale P T2,  T2 = (I + diag(beta) N)^-1,  W2 = T2^T exp(G_C - G) K,
//   dL/dS = exp(G_C) R + scale (exp(G) Q)^T dO - K^T exp(G) beta dX,        dV = beta dX.
// Forward, O takes the operand that S' does: with U' = beta exp(r) E, r = G_C - G (at least -kClosed: P U = P' U' needs its
// inverse), P' = P exp(-r), S' = exp(G_C) S + K^T U'.
// All that does not depend on the states is prepared for all chunks at once, so that a step of a scan
// is two products: the errors from the state, the next state from the errors.
#pragma once

#include "la_delta.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace delta {

using namespace sm100;
using namespace tc;

constexpr int kChunk = 64;
constexpr uint32_t kSq = kChunk * 128;  // a [64 x 64] bf16 image, 128-byte swizzled: 8 KB
// Gates that close what a token writes to exp(-48) by its chunk's end close it no further in S' (1.4e-21 of it is left, 1e-14
// of what fp32 tells apart), so that its inverse, 7e20, leaves room for q.k up to 4e17, and a low part is a normal number for
// errors down to 1e-14.
constexpr float kClosed = 48.f;
constexpr uint64_t kDrainNs = 100000000ull;

// The scalars of a chunk, by token; a scan loads three of the first four.
struct Scalars {
    float beta[kChunk], write[kChunk], first[kChunk], back[kChunk];  // beta, beta exp(G_C - G) (forward: exp(r)), exp(G), -beta exp(G)
    // exp(G_C - G); G log2(e) as two floats (differences of the pairs carry no more than their own rounding)
    float last[kChunk], hi[kChunk], lo[kChunk], open[kChunk];  // (forward: open = exp(-r))
};
static_assert(sizeof(Scalars) == 2048, "");
constexpr uint32_t kScanScalars = 3 * kChunk * 4;

// A chunk's image: the scalars, then matrices in two bf16 parts (high, then low: the value within 2^-17) as 128-byte
// swizzled MMA operands: T [i][j]; W [i][d_k], in boxes of 64 columns; P' [i][j] for the forward pass, or Z [i][j]
// and W2 [j][d_k] for the backward.
template <int DK> struct Layout {
    static constexpr uint32_t w_bytes = 2 * (DK / 64) * kSq;
    static constexpr uint32_t t = sizeof(Scalars), w = t + 2 * kSq, p = w + w_bytes, z = p, w2 = z + 2 * kSq;
    static constexpr uint32_t forward_bytes = p + 2 * kSq, backward_bytes = w2 + w_bytes;
};

// Two values as bf16 high parts and the bf16 rounding of what is left: together within 2^-17 of each.
__device__ __forceinline__ void split2(uint64_t v, uint32_t &hi, uint32_t &lo)
{
    float a, b;
    unpair(v, a, b);
    hi = pack_bf16(a, b);
    const uint64_t h = pair(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
    unpair(fma2(h, pair(-1.f, -1.f), v), a, b);
    lo = pack_bf16(a, b);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) { split2(pair(a, b), hi, lo); }
__device__ __forceinline__ float bf16_at(const uint8_t *p) { return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16); }

__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// For the warp that issues MMAs, whose lanes must stay together: once a wait has run out the abort flag is set, every
// later wait returns at once, and the loop ends at its next check of the flag.
__device__ __forceinline__ void wait_or_abort(unsigned *status, int *abort_flag, uint64_t *bar, uint32_t parity)
{
    if (!mbar_try_wait(bar, parity)) wait_bar(status, abort_flag, bar, parity);
    __syncwarp();
}
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kDrainNs) {
    }
}
// Copies that may still be writing shared memory after an abort have landed long before this returns.
__device__ __forceinline__ void let_copies_land()
{
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kDrainNs) {
    }
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// D_ij = exp(G_i - G_j) of a row's 2 columns: hi, lo (G_i log2(e)) twice, and the columns' as they are.
__device__ __forceinline__ uint64_t decay2(uint64_t hi, uint64_t lo, float2 hj, float2 lj)
{
    float x, y;
    unpair(add2(add2(hi, pair(-hj.x, -hj.y)), add2(lo, pair(-lj.x, -lj.y))), x, y);
    return pair(ex2(x), ex2(y));
}

// Descriptors of a 64-row tile: K-major (rows M or N), k step kk; 64 columns a box of `box` bytes.
__device__ __forceinline__ uint64_t rows_k(uint32_t tile, int kk, uint32_t box = kSq)
{
    return desc_sw128(tile + (kk >> 2) * box + (kk & 3) * 32, 16, 1024);
}
// MN-major (rows K): k step kk of 16 rows; neighbouring boxes of 64 columns `lbo` bytes apart.
__device__ __forceinline__ uint64_t cols_mn(uint32_t tile, int kk, uint32_t lbo = kSq) { return desc_sw128(tile + kk * 2048, lbo, 1024); }

}  // namespace delta
}  // namespace la
