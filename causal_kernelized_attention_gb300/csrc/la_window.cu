// Softmax attention over a sliding window with sinks, on the CUDA cores in fp32.
//
//   forward   s_pj = scale q_p . k_j over the visible j,  lse_p = log sum_j exp(s_pj),
//             o_p = sum_j exp(s_pj - lse_p) v_j           (no visible j: o = 0, lse = -inf)
//   backward  P_pj = exp(s_pj - lse_p),  D_p = dO_p . o_p,
//             dS_pj = P_pj (dO_p . v_j - D_p) scale,
//             dq_p = sum_j dS_pj k_j,  dk_j = sum_p dS_pj q_p,  dv_j = sum_p P_pj dO_p
//             (key and value heads: summed over the query heads that share them)
//
// The forward and the dq blocks give a CTA 64 query rows and pass over the key tiles their
// window and the sinks reach (running maximum and sum of the softmax, the output rescaled as
// the maximum grows); the dk, dv blocks give a CTA 64 keys and pass over the query tiles
// that see them, of every head of the group.  Where those CTAs are few, or a tile of sinks is
// seen by every later row, a tile's query tiles are shared out over several CTAs, whose sums
// the last of them adds up; every sum is taken in a fixed order.  All products are fp32 fused
// multiply-adds on 4 x 4 register tiles fed by 16-byte shared-memory loads (8 loads for 64
// multiply-adds), rows padded by 4 floats so that the 8 threads of a quarter-warp meet 8
// different bank groups.  Bound by the shared-memory loads between the multiply-adds: 2048
// rows, window 512, d 128 run at 58% of the CUDA cores' fp32 rate (forward 43 TFLOP/s, backward
// 36 by the algorithm's 10 d operations a pair, about 50 executed).  fp32 calls run here; bf16
// calls run on the tensor cores.
#include <math.h>

#include <algorithm>

#include "la_tc_common.cuh"
#include "la_window.cuh"

namespace la {
namespace {

using namespace window;

constexpr int kT = 64;         // rows and keys of a tile
constexpr int kThreads = 256;  // 16 x 16: thread (ty, tx) owns rows ty + 16 i, keys tx + 16 j
constexpr int kPS = kT + 4;    // row stride of the probability tiles

template <int D> constexpr int stride() { return D + 4; }

// Rows [t0, t0 + 64) of x [N, D] into shared memory; rows at or past `rows` become zero.
template <int D>
__device__ __forceinline__ void load_tile(float *dst, const float *x, int t0, int rows)
{
    for (int u = threadIdx.x; u < kT * (D / 4); u += kThreads) {
        const int r = u / (D / 4), c = (u % (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + r < rows) v = *reinterpret_cast<const float4 *>(x + (size_t)(t0 + r) * D + c);
        *reinterpret_cast<float4 *>(dst + r * stride<D>() + c) = v;
    }
}

// The same in two halves, so that the next tile's loads run under this tile's products: one
// thread's part of a tile in registers, and its way into shared memory.
template <int D>
struct Part {
    static constexpr int kN = kT * (D / 4) / kThreads;
    float4 v[kN];
    __device__ __forceinline__ void load(const float *x, int t0, int rows)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int u = threadIdx.x + i * kThreads, r = u / (D / 4), c = (u % (D / 4)) * 4;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t0 + r < rows) v[i] = *reinterpret_cast<const float4 *>(x + (size_t)(t0 + r) * D + c);
        }
    }
    __device__ __forceinline__ void store(float *dst) const
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int u = threadIdx.x + i * kThreads, r = u / (D / 4), c = (u % (D / 4)) * 4;
            *reinterpret_cast<float4 *>(dst + r * stride<D>() + c) = v[i];
        }
    }
};

__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float c)
{
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

// acc[i][j] = A[ty + 16 i] . B[tx + 16 j] over D columns.
template <int D>
__device__ __forceinline__ void mul_nt(float (&acc)[4][4], const float *A, const float *B, int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * stride<D>() + c);
            b[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * stride<D>() + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = dot4(a[i], b[j], acc[i][j]);
    }
}

// acc[i][c] += sum_j P[ty + 16 i][j] X[j][col(c)] over the tile's 64 j; thread columns are
// 2 tx, 2 tx + 1 and the same 32 further on.
template <int D>
__device__ __forceinline__ void mul_nn(float (&acc)[4][D / 16], const float *P, const float *X, int ty, int tx)
{
#pragma unroll 2
    for (int j = 0; j < kT; j += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(P + (ty + 16 * i) * kPS + j);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float2 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = *reinterpret_cast<const float2 *>(X + (j + e) * stride<D>() + 32 * c + 2 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][2 * c] = fmaf(p[i].w, x[3].x, fmaf(p[i].z, x[2].x, fmaf(p[i].y, x[1].x, fmaf(p[i].x, x[0].x, acc[i][2 * c]))));
                acc[i][2 * c + 1] =
                    fmaf(p[i].w, x[3].y, fmaf(p[i].z, x[2].y, fmaf(p[i].y, x[1].y, fmaf(p[i].x, x[0].y, acc[i][2 * c + 1]))));
            }
        }
    }
}

__device__ __forceinline__ float max16(float v)
{
#pragma unroll
    for (int m = 8; m > 0; m /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}
__device__ __forceinline__ float sum16(float v)
{
#pragma unroll
    for (int m = 8; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// How the key tiles' query tiles are shared out: the first `sinks` tiles of a key head over
// `sink_parts` CTAs each, the others over `parts`.
struct Split {
    int sinks, sink_parts, parts, tiles;
    int shared_tiles, shared_units;  // of a key head: the tiles of several shares, which come first, and those shares
    __host__ __device__ int units() const { return sinks * sink_parts + (tiles - sinks) * parts; }
};

struct Args {
    const void *q, *k, *v, *o, *dout;
    void *out, *dq, *dk, *dv;
    float *lse, *delta;
    const int *lens;
    int B, Hq, Hk, Nq, Nk, window, sinks;
    float scale;
    Split sp;     // dk, dv
    unsigned dkv_blocks;
    float *part;  // [B Hk][shared units][dk, dv][64][D]
    int *left;    // [B Hk][shared tiles] shares left so far, zeroed by the delta kernel
    int shared;   // B Hk shared tiles
};

// ---------------------------------------------------------------- forward
template <int D>
__global__ void __launch_bounds__(kThreads) window_forward_kernel(const Args a)
{
    extern __shared__ __align__(16) float sm[];
    float *q = sm, *k = q + kT * stride<D>(), *v = k + kT * stride<D>(), *pr = v + kT * stride<D>();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles = (a.Nq + kT - 1) / kT;
    const int bh = (int)(blockIdx.x / tiles), t0 = (int)(blockIdx.x % tiles) * kT;
    const int b = bh / a.Hq, h = bh % a.Hq, off = a.Nk - a.Nq;
    const int n = valid(a.lens, b, a.Nk);
    const size_t kvrow = ((size_t)b * a.Hk + h / (a.Hq / a.Hk)) * a.Nk;
    const float *kp = static_cast<const float *>(a.k) + kvrow * D, *vp = static_cast<const float *>(a.v) + kvrow * D;
    load_tile<D>(q, static_cast<const float *>(a.q) + (size_t)bh * a.Nq * D, t0, a.Nq);
    const KeyTiles kt(t0 + off, min(t0 + kT, a.Nq) - 1 + off, a.window, a.sinks, n, kT);
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    Part<D> kn, vn;
    if (kt.count() > 0) {
        kn.load(kp, kt.tile(0) * kT, n);
        vn.load(vp, kt.tile(0) * kT, n);
    }
    for (int it = 0; it < kt.count(); ++it) {
        const int j0 = kt.tile(it) * kT;
        __syncthreads();
        kn.store(k);
        vn.store(v);
        __syncthreads();
        if (it + 1 < kt.count()) {
            kn.load(kp, kt.tile(it + 1) * kT, n);
            vn.load(vp, kt.tile(it + 1) * kT, n);
        }
        float s[4][4];
        mul_nt<D>(s, q, k, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = t0 + ty + 16 * i + off;
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = sees(p, j0 + tx + 16 * j, a.window, a.sinks, n) ? s[i][j] * a.scale : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            mx = max16(mx);
            const float safe = mx == -INFINITY ? 0.f : mx;  // nothing visible yet
            const float keep = expf(m[i] - safe);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = expf(s[i][j] - safe);
                sum += e;
                pr[(ty + 16 * i) * kPS + tx + 16 * j] = e;
            }
            l[i] = l[i] * keep + sum16(sum);
            m[i] = mx;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= keep;
        }
        __syncthreads();
        mul_nn<D>(o, pr, v, ty, tx);
    }
    float *op = static_cast<float *>(a.out) + (size_t)bh * a.Nq * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty + 16 * i;
        if (t >= a.Nq) continue;
        const float inv = t + off < n ? 1.f / l[i] : 0.f;  // padding gives zeros, a row of no finite score 0 / 0
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            op[(size_t)t * D + 32 * c + 2 * tx] = o[i][2 * c] * inv;
            op[(size_t)t * D + 32 * c + 2 * tx + 1] = o[i][2 * c + 1] * inv;
        }
        if (tx == 0) a.lse[(size_t)bh * a.Nq + t] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    }
}

// P and dS of one 64 x 64 block, rows of queries: s = scores, g = dO . v.
__device__ __forceinline__ void block_ds(float (&s)[4][4], float (&g)[4][4], const float *lse, const float *delta, int t0,
                                         int j0, int off, int n, const Args &a, int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i, p = t0 + r + off;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = t0 + r < a.Nq && sees(p, j0 + tx + 16 * j, a.window, a.sinks, n);
            const float e = in ? expf(s[i][j] * a.scale - lse[r]) : 0.f;
            s[i][j] = e;
            g[i][j] = in ? e * (g[i][j] - delta[r]) * a.scale : 0.f;
        }
    }
}

// ---------------------------------------------------------------- backward: D_p = dO . o
// D / 4 lanes a row; also zeroes the counters of the shared tiles.
template <int D>
__global__ void __launch_bounds__(kThreads) window_delta_kernel(const Args a)
{
    constexpr int L = D / 4;
    const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) / L;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < a.shared; i += (long long)gridDim.x * kThreads)
        a.left[i] = 0;
    const int c = threadIdx.x % L * 4;
    float x = 0.f;
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    if (row < rows)
        x = dot4(*reinterpret_cast<const float4 *>(static_cast<const float *>(a.dout) + row * D + c),
                 *reinterpret_cast<const float4 *>(static_cast<const float *>(a.o) + row * D + c), 0.f);
#pragma unroll
    for (int m = L / 2; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (row < rows && c == 0) a.delta[row] = x;
}

// ---------------------------------------------------------------- backward: dq
template <int D>
__device__ __forceinline__ void dq_block(const Args &a, const unsigned block, float *sm)
{
    float *q = sm, *go = q + kT * stride<D>(), *k = go + kT * stride<D>(), *v = k + kT * stride<D>();
    float *ds = v + kT * stride<D>();
    __shared__ float lse[kT], delta[kT];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles = (a.Nq + kT - 1) / kT;
    const int bh = (int)(block / tiles), t0 = (int)(block % tiles) * kT;
    const int b = bh / a.Hq, h = bh % a.Hq, off = a.Nk - a.Nq;
    const int n = valid(a.lens, b, a.Nk);
    const size_t kvrow = ((size_t)b * a.Hk + h / (a.Hq / a.Hk)) * a.Nk, qrow = (size_t)bh * a.Nq;
    const float *kp = static_cast<const float *>(a.k) + kvrow * D, *vp = static_cast<const float *>(a.v) + kvrow * D;
    const int rows = min(a.Nq, n - off);  // rows of tokens; the others are padding
    load_tile<D>(q, static_cast<const float *>(a.q) + qrow * D, t0, rows);
    load_tile<D>(go, static_cast<const float *>(a.dout) + qrow * D, t0, rows);
    if (threadIdx.x < kT) {
        const bool in = t0 + (int)threadIdx.x < rows;
        lse[threadIdx.x] = in ? a.lse[qrow + t0 + threadIdx.x] : 0.f;
        delta[threadIdx.x] = in ? a.delta[qrow + t0 + threadIdx.x] : 0.f;
    }
    float acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    const KeyTiles kt(t0 + off, min(t0 + kT, a.Nq) - 1 + off, a.window, a.sinks, n, kT);
    Part<D> kn, vn;
    if (kt.count() > 0) {
        kn.load(kp, kt.tile(0) * kT, n);
        vn.load(vp, kt.tile(0) * kT, n);
    }
    for (int it = 0; it < kt.count(); ++it) {
        const int j0 = kt.tile(it) * kT;
        __syncthreads();
        kn.store(k);
        vn.store(v);
        __syncthreads();
        if (it + 1 < kt.count()) {
            kn.load(kp, kt.tile(it + 1) * kT, n);
            vn.load(vp, kt.tile(it + 1) * kT, n);
        }
        float s[4][4], g[4][4];
        mul_nt<D>(s, q, k, ty, tx);
        mul_nt<D>(g, go, v, ty, tx);
        block_ds(s, g, lse, delta, t0, j0, off, n, a, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ds[(ty + 16 * i) * kPS + tx + 16 * j] = g[i][j];
        __syncthreads();
        mul_nn<D>(acc, ds, k, ty, tx);
    }
    float *dq = static_cast<float *>(a.dq) + qrow * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty + 16 * i;
        if (t >= a.Nq) continue;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            dq[(size_t)t * D + 32 * c + 2 * tx] = acc[i][2 * c];
            dq[(size_t)t * D + 32 * c + 2 * tx + 1] = acc[i][2 * c + 1];
        }
    }
}

// ---------------------------------------------------------------- backward: dk, dv
template <int D>
__device__ __forceinline__ void dkv_block(const Args &a, const unsigned block, float *sm)
{
    float *k = sm, *v = k + kT * stride<D>(), *q = v + kT * stride<D>(), *go = q + kT * stride<D>();
    float *pt = go + kT * stride<D>(), *dst = pt + kT * kPS;  // transposed: rows of keys
    __shared__ float lse[kT], delta[kT];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int units = a.sp.units(), bh = (int)(block / units), unit = (int)(block % units);
    const int u1 = unit - a.sp.sinks * a.sp.sink_parts;  // >= 0: not a tile of sinks
    const int parts = u1 < 0 ? a.sp.sink_parts : a.sp.parts, share = (u1 < 0 ? unit : u1) % parts;
    const int j0 = (u1 < 0 ? unit / parts : a.sp.sinks + u1 / parts) * kT;
    const int b = bh / a.Hk, hk = bh % a.Hk, off = a.Nk - a.Nq, group = a.Hq / a.Hk;
    const int n = valid(a.lens, b, a.Nk);
    const size_t kvrow = (size_t)bh * a.Nk;
    load_tile<D>(k, static_cast<const float *>(a.k) + kvrow * D, j0, n);
    load_tile<D>(v, static_cast<const float *>(a.v) + kvrow * D, j0, n);
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
    const QueryTiles qt(j0, min(j0 + kT, a.Nk) - 1, a.window, a.sinks, n, off, a.Nq, kT);
    const int rows = min(a.Nq, n - off);
    const int all = (qt.end - qt.begin) * group;
    const int first = (int)((long long)all * share / parts), end = (int)((long long)all * (share + 1) / parts);
    Part<D> qn, gn;
    float ln = 0.f, dn = 0.f;
    auto fetch = [&](int it) {
        const int t0 = (qt.begin + it / group) * kT;
        const size_t qrow = ((size_t)b * a.Hq + hk * group + it % group) * a.Nq;
        qn.load(static_cast<const float *>(a.q) + qrow * D, t0, rows);
        gn.load(static_cast<const float *>(a.dout) + qrow * D, t0, rows);
        if (threadIdx.x < kT) {
            const bool in = t0 + (int)threadIdx.x < rows;
            ln = in ? a.lse[qrow + t0 + threadIdx.x] : 0.f;
            dn = in ? a.delta[qrow + t0 + threadIdx.x] : 0.f;
        }
    };
    if (first < end) fetch(first);
    for (int it = first; it < end; ++it) {
        const int t0 = (qt.begin + it / group) * kT;
        __syncthreads();
        qn.store(q);
        gn.store(go);
        if (threadIdx.x < kT) {
            lse[threadIdx.x] = ln;
            delta[threadIdx.x] = dn;
        }
        __syncthreads();
        if (it + 1 < end) fetch(it + 1);
        float s[4][4], g[4][4];
        mul_nt<D>(s, q, k, ty, tx);
        mul_nt<D>(g, go, v, ty, tx);
        block_ds(s, g, lse, delta, t0, j0, off, n, a, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pt[(tx + 16 * j) * kPS + ty + 16 * i] = s[i][j];
                dst[(tx + 16 * j) * kPS + ty + 16 * i] = g[i][j];
            }
        __syncthreads();
        mul_nn<D>(dv, pt, go, ty, tx);
        mul_nn<D>(dk, dst, q, ty, tx);
    }
    if (parts > 1) {
        float *dst = a.part + (size_t)(bh * a.sp.shared_units + unit) * 2 * kT * D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const int at = (ty + 16 * i) * D + 32 * c + 2 * tx;
                *reinterpret_cast<float2 *>(dst + at) = make_float2(dk[i][2 * c], dk[i][2 * c + 1]);
                *reinterpret_cast<float2 *>(dst + kT * D + at) = make_float2(dv[i][2 * c], dv[i][2 * c + 1]);
            }
        // the block that is the last to leave its share adds all of them up, in order
        __shared__ int last;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last = atomicAdd(a.left + bh * a.sp.shared_tiles + j0 / kT, 1) == parts - 1;
        __syncthreads();
        if (!last) return;
        __threadfence();
        const float *src = a.part + (size_t)(bh * a.sp.shared_units + unit - share) * 2 * kT * D;
        for (int e = threadIdx.x; e < 2 * kT * (D / 4); e += kThreads) {
            const int c = e % (D / 4) * 4, r = e / (D / 4) % kT, which = e / (D / 4) / kT;
            if (j0 + r >= a.Nk) continue;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < parts; ++i) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + ((size_t)i * 2 + which) * kT * D + r * D + c));
                sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
            }
            *reinterpret_cast<float4 *>(static_cast<float *>(which ? a.dv : a.dk) + (kvrow + j0 + r) * D + c) = sum;
        }
        return;
    }
    float *dkp = static_cast<float *>(a.dk) + kvrow * D, *dvp = static_cast<float *>(a.dv) + kvrow * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + ty + 16 * i;
        if (j >= a.Nk) continue;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const size_t at = (size_t)j * D + 32 * c + 2 * tx;
            *reinterpret_cast<float2 *>(dkp + at) = make_float2(dk[i][2 * c], dk[i][2 * c + 1]);
            *reinterpret_cast<float2 *>(dvp + at) = make_float2(dv[i][2 * c], dv[i][2 * c + 1]);
        }
    }
}

// Both kinds of blocks in one launch, the dk, dv ones first: neither waits for the other, and the last
// wave is filled by either (padded batch of 3 x 509 rows: 42 -> 34 us by it, 30 with the shares added up here).
template <int D>
__global__ void __launch_bounds__(kThreads) window_backward_kernel(const Args a)
{
    extern __shared__ __align__(16) float sm[];
    if (blockIdx.x < a.dkv_blocks)
        dkv_block<D>(a, blockIdx.x, sm);
    else
        dq_block<D>(a, blockIdx.x - a.dkv_blocks, sm);
}

Args args_of(const WindowProblem &p)
{
    Args a;
    a.q = p.q; a.k = p.k; a.v = p.v; a.o = p.o; a.dout = p.dout;
    a.out = p.out; a.dq = p.dq; a.dk = p.dk; a.dv = p.dv;
    a.lse = p.lse; a.delta = p.delta; a.lens = p.lens;
    a.B = p.B; a.Hq = p.Hq; a.Hk = p.Hk; a.Nq = p.Nq; a.Nk = p.Nk;
    a.window = p.window; a.sinks = p.sinks; a.scale = p.scale;
    return a;
}

template <typename K>
la_status launch(K kern, long long ctas, size_t smem, const Args &a, cudaStream_t s)
{
    if (ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    la_status st = smem ? ensure_smem((const void *)kern, (int)smem) : LA_OK;
    if (st != LA_OK) return st;
    count_launches();
    kern<<<(unsigned)ctas, kThreads, smem, s>>>(a);
    return cuda_status(cudaGetLastError());
}

template <int D>
la_status forward(const WindowProblem &p)
{
    const size_t smem = (3 * kT * stride<D>() + kT * kPS) * sizeof(float);
    return launch(window_forward_kernel<D>, (long long)p.B * p.Hq * ceil_div(p.Nq, kT), smem, args_of(p), p.stream);
}

size_t delta_bytes(const WindowProblem &p) { return ((size_t)p.B * p.Hq * p.Nq * 4 + 255) & ~(size_t)255; }

// A share is at least a query tile; shares until there are two CTAs an SM, and until a tile
// of sinks has no more work a CTA than another tile.
Split split_of(const WindowProblem &p)
{
    Split sp;
    sp.tiles = ceil_div(p.Nk, kT);
    sp.sinks = ceil_div(p.sinks, kT);
    const long long group = p.Hq / p.Hk, rows = ceil_div(p.Nq, kT);
    const long long win = std::min<long long>(rows, (long long)(p.window + kT - 2) / kT + 1) * group;
    const long long ctas = (long long)p.B * p.Hk * sp.tiles, want = 2LL * tc::sm_count();
    sp.parts = (int)std::max<long long>(1, std::min(win, (want + ctas - 1) / ctas));
    const long long each = (win + sp.parts - 1) / sp.parts;
    // (many tiles of sinks: no more shares than fill the machine several times over)
    const long long cap = std::max<long long>(1, 4 * want / std::max<long long>(1, (long long)p.B * p.Hk * sp.sinks));
    sp.sink_parts = (int)std::min((rows * group + each - 1) / each, std::max<long long>(cap, sp.parts));
    sp.shared_tiles = sp.parts > 1 ? sp.tiles : sp.sink_parts > 1 ? sp.sinks : 0;
    sp.shared_units = sp.parts > 1 ? sp.units() : sp.shared_tiles * sp.sink_parts;
    return sp;
}

size_t part_floats(const WindowProblem &p, const Split &sp)
{
    return (size_t)p.B * p.Hk * sp.shared_units * 2 * kT * p.d;
}

template <int D>
la_status backward(const WindowProblem &p)
{
    const size_t tile = kT * stride<D>(), prob = kT * kPS;
    Args a = args_of(p);
    a.sp = split_of(p);
    a.part = reinterpret_cast<float *>(reinterpret_cast<char *>(p.delta) + delta_bytes(p));
    a.left = reinterpret_cast<int *>(a.part + part_floats(p, a.sp));
    const long long dkv = (long long)p.B * p.Hk * a.sp.units(), dq = (long long)p.B * p.Hq * ceil_div(p.Nq, kT);
    if (dkv > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    a.dkv_blocks = (unsigned)dkv;
    a.shared = p.B * p.Hk * a.sp.shared_tiles;  // no more than dkv
    const long long rows = (long long)p.B * p.Hq * p.Nq;
    la_status st = launch(window_delta_kernel<D>, (rows * (D / 4) + kThreads - 1) / kThreads, 0, a, p.stream);
    if (st != LA_OK) return st;
    return launch(window_backward_kernel<D>, dkv + dq, (4 * tile + 2 * prob) * sizeof(float), a, p.stream);
}

}  // namespace

la_status window_forward_simt(const WindowProblem &p)
{
    if (p.d == 32) return forward<32>(p);
    return p.d == 64 ? forward<64>(p) : forward<128>(p);
}

size_t window_backward_simt_scratch(const WindowProblem &p)
{
    const Split sp = split_of(p);
    return delta_bytes(p) + part_floats(p, sp) * sizeof(float) + (size_t)p.B * p.Hk * sp.shared_tiles * sizeof(int);
}

la_status window_backward_simt(const WindowProblem &p)
{
    if (p.d == 32) return backward<32>(p);
    return p.d == 64 ? backward<64>(p) : backward<128>(p);
}

}  // namespace la
