// Shared pieces of the gated delta rule's kernels (la_delta.cu, la_tc_delta.cu).
#pragma once

#include <stdint.h>

#include <type_traits>

#include "la_internal.h"

namespace la {
namespace delta {

struct Params {
    const void *q, *k, *v, *dout;
    const float *g, *beta, *S0, *dSN;
    void *o, *dq, *dk_out, *dv_out;
    float *SN, *dg, *dbeta, *dS0;
    int B, Hk, H, N, dk, dv;
    float scale;
    unsigned long long wait_ns;  // limit of a wait for a published chunk; the work item that is not published (a test's), or -1
    long long drop;
};

inline Params params_of(const DeltaProblem &p)
{
    return {p.q,  p.k,  p.v,     p.dout, p.g, p.beta, p.S0, p.dSN, p.o,  p.dq, p.dk_out,
            p.dv_out, p.SN, p.dg, p.dbeta, p.dS0, p.B, p.Hk, p.H, p.N, p.dk, p.dv, p.scale, test_wait_limit_ns(), test_drop_ticket()};
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

}  // namespace delta
}  // namespace la
