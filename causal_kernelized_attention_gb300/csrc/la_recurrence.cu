// Gated recurrence, each channel on its own:
//
//   forward    h_t = alpha_t h_{t-1} + x_t                       (h_{-1} = h0, or 0)
//   backward   g_t = dh_t + alpha_{t+1} g_{t+1}                  (g_{N-1} = dh_{N-1} + dhN)
//              dx_t = g_t,  dalpha_t = g_t h_{t-1},  dh0 = alpha_0 g_0
//
// The backward pass is the forward's scan over reversed time with the gates moved by one
// token, so one kernel does both.  A run of tokens maps the state before it, c, to A c + H
// with A the product of its gates and H its result from zero; runs compose as
// (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2), without a division, so gates of 0 are exact.
//
// Bound by memory: alpha and x are read once, h written once (4 + 2 e bytes an element,
// e the size of x).  A thread holds a run of R tokens of kVec neighbouring channels in
// registers, a CTA a tile of consecutive runs; runs are joined by shuffles within a warp
// and through shared memory between warps.  A cluster of CTAs takes consecutive tiles of
// the same channels and exchanges its CTAs' (A, H) through distributed shared memory once a
// step, so a sequence is split over the machine when there are few channels, in one pass
// over the data and without a flag in global memory to wait for.
#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// V neighbouring elements of type T.
template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T x[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ld(const T *p) { return *reinterpret_cast<const Vec<T, V> *>(p); }
template <typename T, int V>
__device__ __forceinline__ void st(T *p, const Vec<T, V> &v) { *reinterpret_cast<Vec<T, V> *>(p) = v; }

template <typename T>
struct Args {
    const T *x;          // forward: x; backward: dh
    const float *alpha;
    const T *h_in;       // backward: h
    const float *h0;     // may be null
    const float *dhN;    // backward, may be null
    T *out;              // forward: h; backward: dx
    float *dalpha;       // backward
    float *last;         // forward: hN; backward: dh0; may be null
    int N, D, steps;
};

// kVec channels a thread, kCL lanes of a warp side by side over channels (the other
// 32 / kCL one after the other in time), kR tokens a thread.
template <typename T, int kVec, int kCL, int kR, bool kBack>
__global__ void __launch_bounds__(kThreads) recurrence_kernel(const __grid_constant__ Args<T> a)
{
    constexpr int kTL = 32 / kCL;
    constexpr int kC = kCL * kVec;               // channels of a CTA
    constexpr int kTile = kWarps * kTL * kR;     // tokens of a CTA's tile
    __shared__ __align__(16) float wA[kWarps][kC], wH[kWarps][kC];
    __shared__ __align__(16) float cA[2][kMaxCluster][kC], cH[2][kMaxCluster][kC];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cl = lane % kCL, tl = lane / kCL;
    const uint32_t S = cluster_size(), rank = S > 1 ? cluster_ctarank() : 0;
    const int groups = (a.D + kC - 1) / kC;
    const int unit = (int)(blockIdx.x / S);
    const int b = unit / groups, ch = (unit % groups) * kC + cl * kVec;
    const bool live = ch < a.D;
    const size_t base = (size_t)b * a.N * a.D + ch;

    float carry[kVec];  // the state before the cluster's step
#pragma unroll
    for (int v = 0; v < kVec; ++v) carry[v] = 0.f;
    const float *first = kBack ? a.dhN : a.h0;
    if (first && live) {
        const Vec<float, kVec> f = ld<float, kVec>(first + (size_t)b * a.D + ch);
#pragma unroll
        for (int v = 0; v < kVec; ++v) carry[v] = f.x[v];
    }

    if (S > 1) cluster_sync_all();  // every CTA of the cluster runs before its memory is written
    for (int step = 0; step < a.steps; ++step) {
        // scan index of this thread's first token; token t = i (forward), N - 1 - i (backward)
        const long long i0 = ((long long)step * S + rank) * kTile + (warp * kTL + tl) * kR;
        Vec<float, kVec> al[kR];
        Vec<T, kVec> xv[kR], hv[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const long long i = i0 + r;
            const bool in = live && i < a.N;
            const long long t = kBack ? a.N - 1 - i : i;
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                al[r].x[v] = 1.f;  // past the end: the identity
                xv[r].x[v] = Elem<T>::from_f32(0.f);
                hv[r].x[v] = Elem<T>::from_f32(0.f);
            }
            if (in) {
                const size_t o = base + (size_t)t * a.D;
                if (!kBack)
                    al[r] = ld<float, kVec>(a.alpha + o);
                else if (i > 0)
                    al[r] = ld<float, kVec>(a.alpha + o + a.D);
                xv[r] = ld<T, kVec>(a.x + o);
                if (kBack && t > 0) hv[r] = ld<T, kVec>(a.h_in + o - a.D);
            }
        }
        // this thread's run
        float A[kVec], H[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            A[v] = 1.f;
            H[v] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                H[v] = fmaf(al[r].x[v], H[v], Elem<T>::to_f32(xv[r].x[v]));
                A[v] *= al[r].x[v];
            }
        // inclusive scan over the warp's runs of the same channels
#pragma unroll
        for (int m = 1; m < kTL; m *= 2)
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const float pa = __shfl_up_sync(0xffffffffu, A[v], m * kCL);
                const float ph = __shfl_up_sync(0xffffffffu, H[v], m * kCL);
                if (tl >= m) {
                    H[v] = fmaf(A[v], ph, H[v]);
                    A[v] *= pa;
                }
            }
        if (tl == kTL - 1)
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                wA[warp][cl * kVec + v] = A[v];
                wH[warp][cl * kVec + v] = H[v];
            }
        __syncthreads();
        // the runs before this warp's in the CTA, and the whole CTA's
        float pA[kVec], pH[kVec], tA[kVec], tH[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            tA[v] = 1.f;
            tH[v] = 0.f;
            pA[v] = 1.f;
            pH[v] = 0.f;
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const Vec<float, kVec> xa = ld<float, kVec>(&wA[w][cl * kVec]), xh = ld<float, kVec>(&wH[w][cl * kVec]);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                if (w == warp) {
                    pA[v] = tA[v];
                    pH[v] = tH[v];
                }
                tH[v] = fmaf(xa.x[v], tH[v], xh.x[v]);
                tA[v] *= xa.x[v];
            }
        }
        float before[kVec];  // the state before this warp's runs
        if (S > 1) {
            const int slot = step & 1;
            // warp w sends to rank w; the slots alternate, so a CTA still reading this
            // step's is never overtaken (a writer of the slot after next has passed the
            // barrier of the next step)
            if (warp < (int)S && tl == 0) {
                const uint32_t da = mapa_shared(smem_u32(&cA[slot][rank][cl * kVec]), warp);
                const uint32_t dh = mapa_shared(smem_u32(&cH[slot][rank][cl * kVec]), warp);
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    st_dsmem_f32(da + 4 * v, tA[v]);
                    st_dsmem_f32(dh + 4 * v, tH[v]);
                }
            }
            cluster_sync_all();
            float at[kVec];
#pragma unroll
            for (int v = 0; v < kVec; ++v) at[v] = carry[v];
            for (uint32_t w = 0; w < S; ++w) {
                const Vec<float, kVec> xa = ld<float, kVec>(&cA[slot][w][cl * kVec]),
                                       xh = ld<float, kVec>(&cH[slot][w][cl * kVec]);
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    if (w == rank) at[v] = carry[v];
                    carry[v] = fmaf(xa.x[v], carry[v], xh.x[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < kVec; ++v) before[v] = fmaf(pA[v], at[v], pH[v]);
        } else {
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                before[v] = fmaf(pA[v], carry[v], pH[v]);
                carry[v] = fmaf(tA[v], carry[v], tH[v]);
            }
        }
        // the state before this thread's run: through the lanes before it
        float c[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const float pa = __shfl_up_sync(0xffffffffu, A[v], kCL % 32), ph = __shfl_up_sync(0xffffffffu, H[v], kCL % 32);
            c[v] = tl > 0 ? fmaf(pa, before[v], ph) : before[v];
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const long long i = i0 + r;
            const bool in = live && i < a.N;
            const long long t = kBack ? a.N - 1 - i : i;
            Vec<T, kVec> o;
            Vec<float, kVec> da;
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                c[v] = fmaf(al[r].x[v], c[v], Elem<T>::to_f32(xv[r].x[v]));
                o.x[v] = Elem<T>::from_f32(c[v]);
            }
            if (in) {
                const size_t at = base + (size_t)t * a.D;
                st<T, kVec>(a.out + at, o);
                if (kBack) {
                    Vec<float, kVec> hp;
#pragma unroll
                    for (int v = 0; v < kVec; ++v) hp.x[v] = Elem<T>::to_f32(hv[r].x[v]);
                    if (t == 0 && a.h0) hp = ld<float, kVec>(a.h0 + (size_t)b * a.D + ch);
#pragma unroll
                    for (int v = 0; v < kVec; ++v) da.x[v] = c[v] * hp.x[v];
                    st<float, kVec>(a.dalpha + at, da);
                }
            }
        }
        __syncthreads();  // wA, wH are rewritten by the next step
    }
    // the state after the last token (forward), or alpha_0 g_0 (backward)
    if (a.last && rank == 0 && warp == 0 && tl == 0 && live) {
        Vec<float, kVec> o;
#pragma unroll
        for (int v = 0; v < kVec; ++v) o.x[v] = carry[v];
        if (kBack && a.N > 0) {
            const Vec<float, kVec> f = ld<float, kVec>(a.alpha + base);
#pragma unroll
            for (int v = 0; v < kVec; ++v) o.x[v] *= f.x[v];
        }
        st<float, kVec>(a.last + (size_t)b * a.D + ch, o);
    }
}

template <typename T, int kVec, int kCL, int kR, bool kBack>
la_status launch(const RecurrenceProblem &p)
{
    constexpr int kTile = kWarps * (32 / kCL) * kR, kC = kCL * kVec;
    auto kern = recurrence_kernel<T, kVec, kCL, kR, kBack>;
    const long long units = (long long)p.B * ceil_div(p.D, kC);
    const int tiles = (int)(((long long)p.N + kTile - 1) / kTile);
    // Split a sequence over a cluster while its CTAs still all run at once: two resident
    // CTAs an SM are enough to keep the memory busy.
    int S = 1;
    while (S < kMaxCluster && S < tiles && units * S * 2 <= 2LL * tc::sm_count()) S *= 2;
    if (units * S > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    Args<T> a;
    a.x = static_cast<const T *>(kBack ? p.dh : p.x);
    a.alpha = p.alpha;
    a.h_in = static_cast<const T *>(p.h_in);
    a.h0 = p.h0;
    a.dhN = p.dhN;
    a.out = static_cast<T *>(kBack ? p.dx : p.h);
    a.dalpha = p.dalpha;
    a.last = kBack ? p.dh0 : p.hN;
    a.N = p.N;
    a.D = p.D;
    a.steps = (tiles + S - 1) / S;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(units * S));
    lc.blockDim = dim3(kThreads);
    lc.stream = p.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = S > 1 ? 1 : 0;
    count_launches();
    return cuda_status(cudaLaunchKernelEx(&lc, kern, a));
}

template <typename T, bool kBack>
la_status pick(const RecurrenceProblem &p)
{
    // Rows are whole 16-byte vectors of gates only when D is a multiple of 4.
    if (p.D % 4 == 0) return launch<T, 4, 8, 8, kBack>(p);
    return launch<T, 1, 32, 16, kBack>(p);
}

// ---------------------------------------------------------------- one token
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads)
step_kernel(float *state, const T *x, const float *alpha, T *h, long long n)
{
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * kVec;
    if (i >= n) return;
    Vec<float, kVec> s = ld<float, kVec>(state + i);
    const Vec<float, kVec> al = ld<float, kVec>(alpha + i);
    const Vec<T, kVec> xv = ld<T, kVec>(x + i);
    Vec<T, kVec> o;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
        s.x[v] = fmaf(al.x[v], s.x[v], Elem<T>::to_f32(xv.x[v]));
        o.x[v] = Elem<T>::from_f32(s.x[v]);
    }
    st<float, kVec>(state + i, s);
    st<T, kVec>(h + i, o);
}

template <typename T>
la_status step(float *state, const void *x, const float *alpha, void *h, long long n, cudaStream_t s)
{
    count_launches();
    if (n % 4 == 0)
        step_kernel<T, 4><<<(unsigned)((n / 4 + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            state, static_cast<const T *>(x), alpha, static_cast<T *>(h), n);
    else
        step_kernel<T, 1><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            state, static_cast<const T *>(x), alpha, static_cast<T *>(h), n);
    return cuda_status(cudaGetLastError());
}

}  // namespace

la_status recurrence(const RecurrenceProblem &p)
{
    if (p.dtype == LA_BF16) return p.backward ? pick<__nv_bfloat16, true>(p) : pick<__nv_bfloat16, false>(p);
    return p.backward ? pick<float, true>(p) : pick<float, false>(p);
}

la_status recurrence_step(float *state, const void *x, const float *alpha, void *h, int B, int D, la_dtype dtype,
                          cudaStream_t stream)
{
    const long long n = (long long)B * D;
    if (dtype == LA_BF16) return step<__nv_bfloat16>(state, x, alpha, h, n, stream);
    return step<float>(state, x, alpha, h, n, stream);
}

}  // namespace la
