// Gated delta rule on the CUDA cores: the token-by-token scan, its reverse, the gradients of a
// chunk, and the decode step.
//
//   D_t = a_t S_{t-1},  e_t = v_t - D_t^T k_t,  S_t = D_t + k_t (b_t e_t)^T,  o_t = scale S_t^T q_t
//
// with a_t = exp(g_t).  Columns of S (one per value feature) do not meet, so a scan's blocks take
// 32 columns each and hold them in registers.  The scans are bound by the chain of a token (a dot
// product over d_k, two shuffles, the update), not by memory; they serve fp32 and the widths that
// the tensor-core kernels are not built for.
#include "la_common.cuh"
#include "la_delta.cuh"
#include "la_internal.h"

namespace la {
namespace delta {
namespace {

constexpr int kTile = 16;   // tokens staged in shared memory at a time
constexpr int kCols = 32;   // columns of S per block: 4 warps of 8, four lanes to a column
constexpr int kC = 32;      // tokens of a chunk of the backward pass

template <typename T> struct Vec4;
template <> struct Vec4<float> {
    static __device__ __forceinline__ float4 get(const float *p) { return *reinterpret_cast<const float4 *>(p); }
};
template <> struct Vec4<__nv_bfloat16> {
    static __device__ __forceinline__ float4 get(const __nv_bfloat16 *p)
    {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    }
};

__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src));
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

// The rows of one tile: keys, queries, a slice of 32 values (forward: v, reverse: dO), gates.
template <typename T, int DK> struct alignas(16) Stage {
    T k[kTile][DK], q[kTile][DK], v[kTile][kCols];
    float alpha[kTile], beta[kTile];
};

template <typename T, int DK>
__device__ __forceinline__ void load_stage(Stage<T, DK> &s, const T *k, const T *q, const T *v, const float *g,
                                           const float *beta, int t0, int n, int dv, bool want_q)
{
    constexpr int kPer = 16 / sizeof(T);
    const int rows = min(kTile, n - t0), tid = threadIdx.x;
    for (int i = tid; i < rows * (DK / kPer); i += 128) {
        const int r = i / (DK / kPer), c = i % (DK / kPer) * kPer;
        copy16(&s.k[r][c], k + (size_t)(t0 + r) * DK + c);
        if (want_q) copy16(&s.q[r][c], q + (size_t)(t0 + r) * DK + c);
    }
    for (int i = tid; i < rows * (kCols / kPer); i += 128) {
        const int r = i / (kCols / kPer), c = i % (kCols / kPer) * kPer;
        copy16(&s.v[r][c], v + (size_t)(t0 + r) * dv + c);
    }
    copies_commit();
    if (tid < rows) {
        s.alpha[tid] = expf(g[t0 + tid]);
        s.beta[tid] = beta[t0 + tid];
    }
}

// Four lanes share a column: lane part p holds rows 16 m + 4 p .. + 3, so that a warp's reads of a
// key are 64 consecutive bytes (fp32).
template <typename T, int DK> __device__ __forceinline__ float dot_rows(const T *x, const float (&S)[DK / 4], int part)
{
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) {
        const float4 a = Vec4<T>::get(x + 16 * m + 4 * part);
        s[0] = fmaf(a.x, S[4 * m], s[0]);
        s[1] = fmaf(a.y, S[4 * m + 1], s[1]);
        s[2] = fmaf(a.z, S[4 * m + 2], s[2]);
        s[3] = fmaf(a.w, S[4 * m + 3], s[3]);
    }
    float r = (s[0] + s[1]) + (s[2] + s[3]);
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    return r + __shfl_xor_sync(0xffffffffu, r, 2);
}
// S = c S + x w
template <typename T, int DK> __device__ __forceinline__ void update_rows(float (&S)[DK / 4], float c, const T *x, float w, int part)
{
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) {
        const float4 a = Vec4<T>::get(x + 16 * m + 4 * part);
        S[4 * m] = fmaf(a.x, w, c * S[4 * m]);
        S[4 * m + 1] = fmaf(a.y, w, c * S[4 * m + 1]);
        S[4 * m + 2] = fmaf(a.z, w, c * S[4 * m + 2]);
        S[4 * m + 3] = fmaf(a.w, w, c * S[4 * m + 3]);
    }
}
template <int DK> __device__ __forceinline__ void state_out(float *at, const float (&S)[DK / 4], int part, int dv)
{
#pragma unroll
    for (int r = 0; r < DK / 4; ++r) at[(size_t)(r / 4 * 16 + part * 4 + r % 4) * dv] = S[r];
}
template <int DK> __device__ __forceinline__ void state_in(const float *at, float (&S)[DK / 4], int part, int dv)
{
#pragma unroll
    for (int r = 0; r < DK / 4; ++r) S[r] = at ? at[(size_t)(r / 4 * 16 + part * 4 + r % 4) * dv] : 0.f;
}

// kSave: instead of o, the errors e_t (fp32) and the state before each chunk of kC tokens.
template <typename T, int DK, bool kSave>
__global__ void __launch_bounds__(128) delta_scan(Params p, float *errors, float *before)
{
    __shared__ Stage<T, DK> stage[2];
    const int slices = p.dv / kCols, bh = blockIdx.x / slices, c0 = blockIdx.x % slices * kCols;
    const int part = threadIdx.x & 3, col = threadIdx.x >> 2;
    const int b = bh / p.H, bhk = b * p.Hk + bh % p.H / (p.H / p.Hk);
    const T *k = static_cast<const T *>(p.k) + (size_t)bhk * p.N * DK, *q = static_cast<const T *>(p.q) + (size_t)bhk * p.N * DK;
    const T *v = static_cast<const T *>(p.v) + (size_t)bh * p.N * p.dv + c0;
    const float *g = p.g + (size_t)bh * p.N, *beta = p.beta + (size_t)bh * p.N;
    const size_t at = (size_t)bh * DK * p.dv + c0 + col;
    float S[DK / 4];
    state_in<DK>(p.S0 ? p.S0 + at : nullptr, S, part, p.dv);
    const int tiles = (p.N + kTile - 1) / kTile, chunks = (p.N + kC - 1) / kC;
    if (tiles > 0) load_stage<T, DK>(stage[0], k, q, v, g, beta, 0, p.N, p.dv, !kSave);
    for (int i = 0; i < tiles; ++i) {
        if (i + 1 < tiles) {
            load_stage<T, DK>(stage[(i + 1) & 1], k, q, v, g, beta, (i + 1) * kTile, p.N, p.dv, !kSave);
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncthreads();
        const Stage<T, DK> &s = stage[i & 1];
        const int t0 = i * kTile, rows = min(kTile, p.N - t0);
        if (kSave && t0 % kC == 0)
            state_out<DK>(before + ((size_t)bh * chunks + t0 / kC) * DK * p.dv + c0 + col, S, part, p.dv);
        for (int t = 0; t < rows; ++t) {
            const float a = s.alpha[t];
            const float e = Elem<T>::to_f32(s.v[t][col]) - a * dot_rows<T, DK>(s.k[t], S, part);
            update_rows<T, DK>(S, a, s.k[t], s.beta[t] * e, part);
            const size_t row = ((size_t)bh * p.N + t0 + t) * p.dv + c0 + col;
            if (kSave) {
                if (part == 0) errors[row] = e;
            } else {
                const float o = p.scale * dot_rows<T, DK>(s.q[t], S, part);
                if (part == 0) static_cast<T *>(p.o)[row] = Elem<T>::from_f32(o);
            }
        }
        __syncthreads();
    }
    if (!kSave && p.SN) state_out<DK>(p.SN + at, S, part, p.dv);
}

// The reverse scan of R = dL/dS:  R += q (scale dO)^T;  dX = R^T k;  dv = b dX;  R = a (R - k dv^T).
// Writes dv, dX (fp32), R behind each chunk (before the chunk's own dO) and dS0.
template <typename T, int DK>
__global__ void __launch_bounds__(128) delta_reverse(Params p, float *dX, float *after)
{
    __shared__ Stage<T, DK> stage[2];
    const int slices = p.dv / kCols, bh = blockIdx.x / slices, c0 = blockIdx.x % slices * kCols;
    const int part = threadIdx.x & 3, col = threadIdx.x >> 2;
    const int b = bh / p.H, bhk = b * p.Hk + bh % p.H / (p.H / p.Hk);
    const T *k = static_cast<const T *>(p.k) + (size_t)bhk * p.N * DK, *q = static_cast<const T *>(p.q) + (size_t)bhk * p.N * DK;
    const T *dout = static_cast<const T *>(p.dout) + (size_t)bh * p.N * p.dv + c0;
    const float *g = p.g + (size_t)bh * p.N, *beta = p.beta + (size_t)bh * p.N;
    const size_t at = (size_t)bh * DK * p.dv + c0 + col;
    float R[DK / 4];
    state_in<DK>(p.dSN ? p.dSN + at : nullptr, R, part, p.dv);
    const int tiles = (p.N + kTile - 1) / kTile, chunks = (p.N + kC - 1) / kC;
    if (tiles > 0) load_stage<T, DK>(stage[(tiles - 1) & 1], k, q, dout, g, beta, (tiles - 1) * kTile, p.N, p.dv, true);
    for (int i = tiles - 1; i >= 0; --i) {
        if (i > 0) {
            load_stage<T, DK>(stage[(i - 1) & 1], k, q, dout, g, beta, (i - 1) * kTile, p.N, p.dv, true);
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncthreads();
        const Stage<T, DK> &s = stage[i & 1];
        const int t0 = i * kTile, rows = min(kTile, p.N - t0);
        if (i == tiles - 1 || (t0 + kTile) % kC == 0)
            state_out<DK>(after + ((size_t)bh * chunks + t0 / kC) * DK * p.dv + c0 + col, R, part, p.dv);
        for (int t = rows - 1; t >= 0; --t) {
            update_rows<T, DK>(R, 1.f, s.q[t], p.scale * Elem<T>::to_f32(s.v[t][col]), part);
            const float x = dot_rows<T, DK>(s.k[t], R, part), y = s.beta[t] * x, a = s.alpha[t];
            update_rows<T, DK>(R, a, s.k[t], -a * y, part);
            const size_t row = ((size_t)bh * p.N + t0 + t) * p.dv + c0 + col;
            if (part == 0) {
                dX[row] = x;
                static_cast<T *>(p.dv_out)[row] = Elem<T>::from_f32(y);
            }
        }
        __syncthreads();
    }
    if (p.dS0) state_out<DK>(p.dS0 + at, R, part, p.dv);
}

// Gradients within a chunk of kC tokens of one key head, over the heads that share it.  With
// U = b e, Y = b dX, G the running sum of g in the chunk, D_ij = exp(G_i - G_j) (j <= i), B and A the
// state before the chunk and its gradient behind it:
//   dP = tril(dO U^T),  dM = -tril(Y U^T, -1)
//   dq = exp(G) dO B^T + (D dP) k
//   dk = exp(G_end - G) U A^T - exp(G) Y B^T + (D dP)^T q + (D dM + (D dM)^T) k
//   dbeta = rowsum(dX e)
// and g_t stands in each decay that crosses from before t to t or later: dg_t sums, over the pairs i >= t > j,
// D_ij (q_i.k_j dP_ij + k_i.k_j dM_ij), the reads of B at i >= t, the writes into A at j < t, and
// exp(G_end) <B, A>.  Every term carries its own decay: nothing is taken as a difference of larger sums.
template <int DK, int DV> struct LocalSmem {
    float K[kC][DK + 4], Q[kC][DK + 4], O[kC][DV + 4], U[kC][DV + 4], Y[kC][DV + 4];
    float B[DK][33], A[DK][33];
    float P[kC][kC + 1], M[kC][kC + 1], R[kC][kC + 1];
    float hi[kC], lo[kC], first[kC], last[kC], beta[kC], reads[kC], writes[kC], sums[8];
};

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256) delta_local(Params p, const float *errors, const float *dX, const float *before,
                                                   const float *after)
{
    extern __shared__ float4 smem_raw[];
    LocalSmem<DK, DV> &s = *reinterpret_cast<LocalSmem<DK, DV> *>(smem_raw);
    constexpr int kKG = DK / 4, kI = DK / 32;  // threads along d_k; rows a thread
    const int chunks = (p.N + kC - 1) / kC, bhk = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int group = p.H / p.Hk, t0 = chunk * kC, rows = min(kC, p.N - t0), tid = threadIdx.x;
    const int kg = tid % kKG, i0 = tid / kKG * kI;
    for (int i = tid; i < kC * DK; i += 256) {
        const int r = i / DK, c = i % DK;
        const size_t at = ((size_t)bhk * p.N + t0 + r) * DK + c;
        s.K[r][c] = r < rows ? Elem<T>::to_f32(static_cast<const T *>(p.k)[at]) : 0.f;
        s.Q[r][c] = r < rows ? Elem<T>::to_f32(static_cast<const T *>(p.q)[at]) : 0.f;
    }
    float dq[kI][4] = {}, dk[kI][4] = {};
    for (int h = 0; h < group; ++h) {
        const int bh = bhk / p.Hk * p.H + bhk % p.Hk * group + h;
        __syncthreads();  // the previous head's tiles are read
        if (tid < 32) {  // the running sum of the gates, as two floats (a gate below -200 closes as well as -inf)
            const size_t at = (size_t)bh * p.N + t0 + tid;
            const float gt = tid < rows ? p.g[at] : 0.f;
            double G = gt < -200.f ? -200.f : gt;
            for (int d = 1; d < 32; d *= 2) {
                const double x = __shfl_up_sync(0xffffffffu, G, d);
                if (tid >= d) G += x;
            }
            const double end = __shfl_sync(0xffffffffu, G, 31);
            s.hi[tid] = (float)G;
            s.lo[tid] = (float)(G - (double)s.hi[tid]);
            s.first[tid] = expf((float)G);
            s.last[tid] = expf((float)(end - G));
            s.beta[tid] = tid < rows ? p.beta[at] : 0.f;
        }
        __syncthreads();
        {
            const int r = tid / 8;
            const float bt = s.beta[r];
            float db = 0.f;
            for (int c = tid % 8; c < DV; c += 8) {
                const size_t at = ((size_t)bh * p.N + t0 + r) * DV + c;
                const float e = r < rows ? errors[at] : 0.f, x = r < rows ? dX[at] : 0.f;
                s.O[r][c] = r < rows ? p.scale * Elem<T>::to_f32(static_cast<const T *>(p.dout)[at]) : 0.f;
                s.U[r][c] = bt * e;
                s.Y[r][c] = bt * x;
                db = fmaf(x, e, db);
            }
            for (int d = 1; d < 8; d *= 2) db += __shfl_xor_sync(0xffffffffu, db, d);
            if (tid % 8 == 0 && r < rows) p.dbeta[(size_t)bh * p.N + t0 + r] = db;
        }
        float rq[kI][4] = {}, rk[kI][4] = {}, wk[kI][4] = {}, whole = 0.f;
        const size_t st = ((size_t)bh * chunks + chunk) * DK * DV;
        for (int v0 = 0; v0 < DV; v0 += 32) {
            __syncthreads();
            for (int i = tid; i < DK * 32; i += 256) {
                const size_t at = st + (size_t)(i / 32) * DV + v0 + i % 32;
                const float x = before[at], y = after[at];
                s.B[i / 32][i % 32] = x;
                s.A[i / 32][i % 32] = y;
                whole = fmaf(x, y, whole);
            }
            __syncthreads();
#pragma unroll 4
            for (int v = 0; v < 32; ++v) {
                float b[4], a[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) b[m] = s.B[kg + m * kKG][v], a[m] = s.A[kg + m * kKG][v];
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    const float o = s.O[i0 + i][v0 + v], u = s.U[i0 + i][v0 + v], y = s.Y[i0 + i][v0 + v];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        rq[i][m] = fmaf(o, b[m], rq[i][m]);
                        rk[i][m] = fmaf(y, b[m], rk[i][m]);
                        wk[i][m] = fmaf(u, a[m], wk[i][m]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const float f = s.first[i0 + i], l = s.last[i0 + i];
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float kk = s.K[i0 + i][kg + m * kKG], qq = s.Q[i0 + i][kg + m * kKG];
                rq[i][m] *= f;
                rk[i][m] *= -f;
                wk[i][m] *= l;
                x = fmaf(qq, rq[i][m], fmaf(kk, rk[i][m], x));
                y = fmaf(kk, wk[i][m], y);
                dq[i][m] += rq[i][m];
                dk[i][m] += rk[i][m] + wk[i][m];
            }
#pragma unroll
            for (int d = 1; d < kKG; d *= 2) {
                x += __shfl_xor_sync(0xffffffffu, x, d);
                y += __shfl_xor_sync(0xffffffffu, y, d);
            }
            if (kg == 0) s.reads[i0 + i] = x, s.writes[i0 + i] = y;
        }
        for (int d = 1; d < 32; d *= 2) whole += __shfl_xor_sync(0xffffffffu, whole, d);
        if (tid % 32 == 0) s.sums[tid / 32] = whole;
        {
            const int i = tid / 8;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int j = tid % 8 + 8 * m;
                float dp = 0.f, dm = 0.f, qk = 0.f, kk = 0.f;
                if (j <= i) {
                    for (int c = 0; c < DV; ++c) {
                        const float u = s.U[j][c];
                        dp = fmaf(s.O[i][c], u, dp);
                        dm = fmaf(-s.Y[i][c], u, dm);
                    }
                    for (int c = 0; c < DK; ++c) {
                        const float x = s.K[j][c];
                        qk = fmaf(s.Q[i][c], x, qk);
                        kk = fmaf(s.K[i][c], x, kk);
                    }
                }
                const float D = j <= i ? expf((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j])) : 0.f;
                s.P[i][j] = D * dp;
                s.M[i][j] = j < i ? D * dm : 0.f;
                s.R[i][j] = j < i ? D * (qk * dp + kk * dm) : 0.f;
            }
        }
        __syncthreads();
        for (int j = 0; j < kC; ++j) {
            float kj[4], qj[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) kj[m] = s.K[j][kg + m * kKG], qj[m] = s.Q[j][kg + m * kKG];
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                const float pij = s.P[i0 + i][j], pji = s.P[j][i0 + i], mm = s.M[i0 + i][j] + s.M[j][i0 + i];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    dq[i][m] = fmaf(pij, kj[m], dq[i][m]);
                    dk[i][m] = fmaf(pji, qj[m], fmaf(mm, kj[m], dk[i][m]));
                }
            }
        }
        if (tid < 32) {
            float row = 0.f, pairs = 0.f;  // of row tid: R summed over j < t
            for (int t = 0; t < 32; ++t) {
                float x = tid >= t ? row : 0.f;
                for (int d = 1; d < 32; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
                if (tid == t) pairs = x;
                row += s.R[tid][t];
            }
            float reads = s.reads[tid], writes = s.writes[tid];
            for (int d = 1; d < 32; d *= 2) {
                const float x = __shfl_down_sync(0xffffffffu, reads, d), y = __shfl_up_sync(0xffffffffu, writes, d);
                if (tid + d < 32) reads += x;
                if (tid >= d) writes += y;
            }
            const float before_t = __shfl_up_sync(0xffffffffu, writes, 1);
            float sum = 0.f;
            for (int w = 0; w < 8; ++w) sum += s.sums[w];
            if (tid < rows)
                p.dg[(size_t)bh * p.N + t0 + tid] = pairs + reads + (tid ? before_t : 0.f) + s.first[31] * sum;
        }
    }
#pragma unroll
    for (int i = 0; i < kI; ++i)
        if (i0 + i < rows)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const size_t at = ((size_t)bhk * p.N + t0 + i0 + i) * DK + kg + m * kKG;
                static_cast<T *>(p.dq)[at] = Elem<T>::from_f32(dq[i][m]);
                static_cast<T *>(p.dk_out)[at] = Elem<T>::from_f32(dk[i][m]);
            }
}

// One decode step.  A block takes 32 columns of one head's state: 16 rows of eight lanes with four
// columns each, so that a warp reads four rows of 128 bytes and every thread has DK / 16 loads in flight.  The dot
// products with k and q are taken in the one pass that reads S, as S_t^T q = a S^T q + (k.q) u.
template <typename T, int DK>
__global__ void __launch_bounds__(128) delta_step_kernel(Params p, float *S)
{
    __shared__ float ks[DK], qs[DK];
    __shared__ float4 part[2][4][8];
    const int slices = p.dv / kCols, bh = blockIdx.x / slices, c0 = blockIdx.x % slices * kCols;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cg = tid & 7, r0 = tid >> 3;
    const int bhk = bh / p.H * p.Hk + bh % p.H / (p.H / p.Hk);
    float4 *at = reinterpret_cast<float4 *>(S + (size_t)bh * DK * p.dv + c0) + cg;
    const size_t row = p.dv / 4;
    float4 x[DK / 16];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) x[m] = __ldcs(at + (r0 + 16 * m) * row);
    const float a = expf(p.g[bh]), beta = p.beta[bh];
    const size_t vat = (size_t)bh * p.dv + c0 + 4 * cg;
    const float4 v = Vec4<T>::get(static_cast<const T *>(p.v) + vat);
    if (tid < DK) {
        ks[tid] = Elem<T>::to_f32(static_cast<const T *>(p.k)[(size_t)bhk * DK + tid]);
        qs[tid] = Elem<T>::to_f32(static_cast<const T *>(p.q)[(size_t)bhk * DK + tid]);
    }
    __syncthreads();
    float kq = 0.f;
#pragma unroll
    for (int m = 0; m < DK / 32; ++m) kq = fmaf(ks[lane + 32 * m], qs[lane + 32 * m], kq);
    float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) {
        const float kr = ks[r0 + 16 * m], qr = qs[r0 + 16 * m];
        sk.x = fmaf(kr, x[m].x, sk.x), sk.y = fmaf(kr, x[m].y, sk.y), sk.z = fmaf(kr, x[m].z, sk.z), sk.w = fmaf(kr, x[m].w, sk.w);
        sq.x = fmaf(qr, x[m].x, sq.x), sq.y = fmaf(qr, x[m].y, sq.y), sq.z = fmaf(qr, x[m].z, sq.z), sq.w = fmaf(qr, x[m].w, sq.w);
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        kq += __shfl_xor_sync(0xffffffffu, kq, d);
        if (d < 8) continue;
        sk.x += __shfl_xor_sync(0xffffffffu, sk.x, d), sk.y += __shfl_xor_sync(0xffffffffu, sk.y, d);
        sk.z += __shfl_xor_sync(0xffffffffu, sk.z, d), sk.w += __shfl_xor_sync(0xffffffffu, sk.w, d);
        sq.x += __shfl_xor_sync(0xffffffffu, sq.x, d), sq.y += __shfl_xor_sync(0xffffffffu, sq.y, d);
        sq.z += __shfl_xor_sync(0xffffffffu, sq.z, d), sq.w += __shfl_xor_sync(0xffffffffu, sq.w, d);
    }
    if (lane < 8) part[0][warp][lane] = sk, part[1][warp][lane] = sq;
    __syncthreads();
    auto total = [&](int w) {
        const float4 y0 = part[w][0][cg], y1 = part[w][1][cg], y2 = part[w][2][cg], y3 = part[w][3][cg];
        return make_float4((y0.x + y1.x) + (y2.x + y3.x), (y0.y + y1.y) + (y2.y + y3.y), (y0.z + y1.z) + (y2.z + y3.z),
                           (y0.w + y1.w) + (y2.w + y3.w));
    };
    sk = total(0);
    const float4 u = make_float4(beta * (v.x - a * sk.x), beta * (v.y - a * sk.y), beta * (v.z - a * sk.z), beta * (v.w - a * sk.w));
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) {
        const float kr = ks[r0 + 16 * m];
        __stcs(at + (r0 + 16 * m) * row, make_float4(fmaf(kr, u.x, a * x[m].x), fmaf(kr, u.y, a * x[m].y),
                                                     fmaf(kr, u.z, a * x[m].z), fmaf(kr, u.w, a * x[m].w)));
    }
    if (r0 == 0) {
        sq = total(1);
        T *o = static_cast<T *>(p.o) + vat;
        o[0] = Elem<T>::from_f32(p.scale * fmaf(kq, u.x, a * sq.x));
        o[1] = Elem<T>::from_f32(p.scale * fmaf(kq, u.y, a * sq.y));
        o[2] = Elem<T>::from_f32(p.scale * fmaf(kq, u.z, a * sq.z));
        o[3] = Elem<T>::from_f32(p.scale * fmaf(kq, u.w, a * sq.w));
    }
}

// Calls f with the element type and d_k as types.
template <typename F> la_status by_width(const DeltaProblem &p, F f)
{
    if (p.dtype == LA_F32)
        return p.dk == 32 ? f(0.f, std::integral_constant<int, 32>()) : p.dk == 64 ? f(0.f, std::integral_constant<int, 64>())
                                                                                   : f(0.f, std::integral_constant<int, 128>());
    const __nv_bfloat16 h{};
    return p.dk == 32 ? f(h, std::integral_constant<int, 32>()) : p.dk == 64 ? f(h, std::integral_constant<int, 64>())
                                                                             : f(h, std::integral_constant<int, 128>());
}

template <typename T, int DK, int DV>
la_status launch_local(const DeltaProblem &p, const Params &prm, const float *errors, const float *dX, const float *before,
                       const float *after)
{
    const int smem = (int)sizeof(LocalSmem<DK, DV>);
    const la_status st = ensure_smem(reinterpret_cast<const void *>(&delta_local<T, DK, DV>), smem);
    if (st != LA_OK) return st;
    const unsigned grid = (unsigned)p.B * p.Hk * ceil_div(p.N, kC);
    count_launches();
    delta_local<T, DK, DV><<<grid, 256, smem, p.stream>>>(prm, errors, dX, before, after);
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace delta

using namespace delta;

la_status delta_forward_simt(const DeltaProblem &p)
{
    const Params prm = params_of(p);
    return by_width(p, [&](auto t, auto dk) {
        count_launches();
        delta_scan<decltype(t), decltype(dk)::value, false>
            <<<(unsigned)(p.B * p.H * (p.dv / kCols)), 128, 0, p.stream>>>(prm, nullptr, nullptr);
        return cuda_status(cudaGetLastError());
    });
}

size_t delta_backward_simt_scratch(const DeltaProblem &p)
{
    const size_t rows = (size_t)p.B * p.H * p.N * p.dv, states = (size_t)p.B * p.H * ceil_div(p.N, kC) * p.dk * p.dv;
    return (rows + states) * 2 * sizeof(float);
}

la_status delta_backward_simt(const DeltaProblem &p)
{
    const Params prm = params_of(p);
    const size_t rows = (size_t)p.B * p.H * p.N * p.dv, states = (size_t)p.B * p.H * ceil_div(p.N, kC) * p.dk * p.dv;
    float *before = p.scratch, *after = before + states, *errors = after + states, *dX = errors + rows;
    return by_width(p, [&](auto t, auto dk) {
        using T = decltype(t);
        constexpr int DK = decltype(dk)::value;
        const unsigned grid = (unsigned)(p.B * p.H * (p.dv / kCols));
        if (p.N > 0) {
            count_launches();
            delta_scan<T, DK, true><<<grid, 128, 0, p.stream>>>(prm, errors, before);
        }
        count_launches();
        delta_reverse<T, DK><<<grid, 128, 0, p.stream>>>(prm, dX, after);
        const la_status st = cuda_status(cudaGetLastError());
        if (st != LA_OK || p.N == 0) return st;
        return p.dv == 32   ? launch_local<T, DK, 32>(p, prm, errors, dX, before, after)
               : p.dv == 64 ? launch_local<T, DK, 64>(p, prm, errors, dX, before, after)
                            : launch_local<T, DK, 128>(p, prm, errors, dX, before, after);
    });
}

la_status delta_step(const DeltaProblem &p, float *S)
{
    const Params prm = params_of(p);
    return by_width(p, [&](auto t, auto dk) {
        count_launches();
        delta_step_kernel<decltype(t), decltype(dk)::value>
            <<<(unsigned)(p.B * p.H * (p.dv / kCols)), 128, 0, p.stream>>>(prm, S);
        return cuda_status(cudaGetLastError());
    });
}

}  // namespace la
