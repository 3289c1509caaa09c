// Rotary positions of q and k.
//
// Feature pairs (a, b) of a token at position p turn by the angle p f_i:
//   a' = A (a cos - b sin),  b' = A (b cos + a sin)      (backward: the transpose, -sin)
// with f_i the pair's frequency and A an amplitude.  Pair i is features (i, i + rot/2)
// in the half layout, (2i, 2i + 1) in the interleaved one; features from `rot` on are copied.
//
// Angles.  The host passes F_i = f_i / (2 pi) 2^64 from a double, so p F_i modulo 2^64 --
// one integer multiplication -- is the angle's fraction of a turn: the reduction is exact,
// and what is left is the double's own rounding, |p f_i| 2^-47 at most with rot = 256 (8e-10
// at p = 10^5, where a 32-bit p f_i would be off by 4e-3).  The nearest quarter turn is
// taken off in integers too, and sincospif sees at most 1/4.
//
// Bound by memory: each element is read and written once.  A thread owns V pairs of one
// token (two vectors of up to 16 bytes), computes their sines once and applies them to a
// run of heads, so the ~40 instructions a sine and cosine cost are shared by the run.
#include <math.h>

#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

struct Args {
    const void *q, *k;
    void *oq, *ok;
    const int *positions;  // [B, N], or null: offset + n
    long long offset;
    int Hq, Hk, N, d, rot;
    long long tokens;      // B N
    int run;               // heads a thread turns; a token's runs are the grid's second dimension
    float amplitude, sign;
    uint64_t turns[kRotaryMaxPairs];
};

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T x[V]; };

template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args a)
{
    const int units = a.d / (2 * V);  // per token
    const long long u = (long long)blockIdx.x * kThreads + threadIdx.x, token = u / units;
    if (token >= a.tokens) return;
    const int c = (int)(u % units), n = (int)(token % a.N), g = (int)blockIdx.y;
    const long long b = token / a.N;
    const bool turned = c < a.rot / (2 * V);
    float cs[V], sn[V];
    if (turned) {
        const long long p = a.positions ? (long long)a.positions[token] : a.offset + n;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t t = (uint64_t)p * a.turns[c * V + i];
            const uint64_t quarter = (t + (1ull << 61)) >> 62;
            const float r = (float)(long long)(t - (quarter << 62)) * 0x1p-63f;  // half turns, |r| <= 1/4
            float s, co;
            sincospif(r, &s, &co);
            const float s1 = (quarter & 1) ? co : s, c1 = (quarter & 1) ? s : co;
            sn[i] = ((quarter & 2) ? -s1 : s1) * a.amplitude * a.sign;
            cs[i] = (((quarter + 1) & 2) ? -c1 : c1) * a.amplitude;
        }
    }
    // first and second vector of this unit
    const int e0 = turned ? (kInterleaved ? 2 * V * c : V * c) : 2 * V * c;
    const int e1 = turned && !kInterleaved ? e0 + a.rot / 2 : e0 + V;
    const int h0 = g * a.run, h1 = min(h0 + a.run, a.Hq + a.Hk);
    const size_t row = (size_t)a.N * a.d;
    const size_t at = (size_t)n * a.d;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const bool isq = h < a.Hq;
        const size_t off = (isq ? (size_t)b * a.Hq + h : (size_t)b * a.Hk + (h - a.Hq)) * row + at;
        const T *x = static_cast<const T *>(isq ? a.q : a.k) + off;
        T *y = static_cast<T *>(isq ? a.oq : a.ok) + off;
        Vec<T, V> v0 = *reinterpret_cast<const Vec<T, V> *>(x + e0);
        Vec<T, V> v1 = *reinterpret_cast<const Vec<T, V> *>(x + e1);
        if (turned) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // half: (v0[i], v1[i]); interleaved: consecutive elements of the two vectors in order
                T &xa = kInterleaved ? (2 * i < V ? v0.x[(2 * i) % V] : v1.x[(2 * i) % V]) : v0.x[i];
                T &xb = kInterleaved ? (2 * i + 1 < V ? v0.x[(2 * i + 1) % V] : v1.x[(2 * i + 1) % V]) : v1.x[i];
                const float fa = Elem<T>::to_f32(xa), fb = Elem<T>::to_f32(xb);
                xa = Elem<T>::from_f32(fa * cs[i] - fb * sn[i]);
                xb = Elem<T>::from_f32(fb * cs[i] + fa * sn[i]);
            }
        }
        *reinterpret_cast<Vec<T, V> *>(y + e0) = v0;
        *reinterpret_cast<Vec<T, V> *>(y + e1) = v1;
    }
}

template <typename T, int V>
la_status launch(const Args &a, bool interleaved, cudaStream_t s)
{
    const long long ctas = (a.tokens * (a.d / (2 * V)) + kThreads - 1) / kThreads;
    if (ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ctas, (unsigned)ceil_div(a.Hq + a.Hk, a.run));
    count_launches();
    if (interleaved)
        rotary_kernel<T, V, true><<<grid, kThreads, 0, s>>>(a);
    else
        rotary_kernel<T, V, false><<<grid, kThreads, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace

la_status rotary(const RotaryProblem &p)
{
    Args a;
    a.q = p.q; a.k = p.k; a.oq = p.oq; a.ok = p.ok;
    a.positions = p.positions;
    a.offset = p.offset;
    a.tokens = (long long)p.B * p.N;
    a.Hq = p.Hq; a.Hk = p.Hk; a.N = p.N; a.d = p.d; a.rot = p.spec.rot;
    a.amplitude = p.spec.amplitude;
    a.sign = p.backward ? -1.f : 1.f;
    for (int i = 0; i < p.spec.rot / 2; ++i) a.turns[i] = p.turns[i];
    // Widest vectors that both the turned and the copied part are whole numbers of.
    const int top = p.dtype == LA_BF16 ? 8 : 4;
    int V = top;
    while (V > 1 && (p.spec.rot % (2 * V) != 0 || p.d % (2 * V) != 0)) V /= 2;
    // Heads per thread: up to 8 share a thread's sines, fewer when the tokens alone do
    // not fill the machine (2048 threads an SM), down to one head per thread.
    const int heads = p.Hq + p.Hk;
    const long long threads = a.tokens * (p.d / (2 * V));
    int run = 8;
    while (run > 1 && threads * ceil_div(heads, run) < 2048LL * tc::sm_count()) run /= 2;
    a.run = max(run, ceil_div(heads, 65535));  // the grid's second dimension
    const bool il = p.spec.layout == LA_ROTARY_INTERLEAVED;
    if (p.dtype == LA_BF16) {
        if (V == 8) return launch<__nv_bfloat16, 8>(a, il, p.stream);
        if (V == 4) return launch<__nv_bfloat16, 4>(a, il, p.stream);
        if (V == 2) return launch<__nv_bfloat16, 2>(a, il, p.stream);
        return launch<__nv_bfloat16, 1>(a, il, p.stream);
    }
    if (V == 4) return launch<float, 4>(a, il, p.stream);
    if (V == 2) return launch<float, 2>(a, il, p.stream);
    return launch<float, 1>(a, il, p.stream);
}

}  // namespace la
