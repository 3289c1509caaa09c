// Shared pieces of the gated delta rule's kernels (la_delta.cu, la_tc_delta.cu).
#pragma once

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
};

inline Params params_of(const DeltaProblem &p)
{
    return {p.q,  p.k,  p.v,     p.dout, p.g, p.beta, p.S0, p.dSN, p.o,  p.dq, p.dk_out,
            p.dv_out, p.SN, p.dg, p.dbeta, p.dS0, p.B, p.Hk, p.H, p.N, p.dk, p.dv, p.scale};
}

}  // namespace delta
}  // namespace la
