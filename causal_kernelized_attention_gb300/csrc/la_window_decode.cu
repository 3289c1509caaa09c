// Window attention for serving: the ring cache, its prefill and the decode step.
//
// A sequence keeps sinks + window slots per key head: token j is in slot j while j < sinks,
// else in slot sinks + (j - sinks) % window, where it replaces the token that has just left
// the window.  Softmax does not depend on the keys' order, so a decode step reads slots
// 0 .. min(pos + 1, sinks + window) - 1 as they lie; the new token's k and v come from the
// call's arguments and are written to their slot by the CTA whose share that slot is in (no
// other reads it).
//
// Bound by memory: the visible slots are read once, 2 d e bytes each.  The slots of one
// (entry, key head) are split over the warps of a cluster of CTAs; each warp runs its own
// softmax (running maximum, sum and output of its slots) and the partial results are
// joined once, through distributed shared memory, in a fixed order.
#include <math.h>

#include "la_tc_common.cuh"
#include "la_window.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    void *kc, *vc;
    const void *q, *k, *v;
    void *o;
    const int *pos;
    int Hq, Hk, window, sinks;
    float scale;
};

// The slots of one sequence at position pos >= 0.
struct Slots {
    int count, fresh;  // slots [0, count) are visible; `fresh` takes the new token
    __device__ __forceinline__ Slots(int pos, int window, int sinks)
    {
        count = (int)min((long long)pos + 1, (long long)sinks + window);
        fresh = pos < sinks ? pos : sinks + (pos - sinks) % window;
    }
};

// Joins the partial results of kParts warps in each of the cluster's S CTAs: per row of G heads
// m (the largest score before scaling by f, which turns it into log2 units) and l, then the
// unnormalised outputs, at the same place in every CTA's shared memory.  First every part's
// weight, exp2((m - top) f) / sum, then the weighted sum of the outputs, each CTA for its
// share of them; `wt` holds G x S kParts floats twice.
template <typename T, int D, int G, int kParts>
__device__ __forceinline__ void join(const float *m, const float *l, const float *acc, float *wt, int rows, float f, T *o,
                                     uint32_t S, uint32_t rank)
{
    const int P = (int)S * kParts;
    const uint32_t ma = smem_u32(m), la_ = smem_u32(l), aa = smem_u32(acc);
    float *wl = wt + G * kMaxCluster * kParts;
    for (int e = threadIdx.x; e < rows * P; e += blockDim.x) {
        const int r = e / P, i = e % P;
        const uint32_t at = 4 * (i % kParts * G + r), cta = i / kParts;
        wt[e] = ld_dsmem_f32(mapa_shared(ma + at, cta));
        wl[e] = ld_dsmem_f32(mapa_shared(la_ + at, cta));
    }
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
        float top = -INFINITY, sum = 0.f;
        for (int i = 0; i < P; ++i) top = fmaxf(top, wt[r * P + i]);
        for (int i = 0; i < P; ++i) {
            const float mi = wt[r * P + i], w = mi == -INFINITY ? 0.f : exp2f((mi - top) * f);  // -inf: no slots
            wt[r * P + i] = w;
            sum = fmaf(w, wl[r * P + i], sum);
        }
        for (int i = 0; i < P; ++i) wt[r * P + i] /= sum;
    }
    __syncthreads();
    for (int e = rank * blockDim.x + threadIdx.x; e < rows * (D / 4); e += S * blockDim.x) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < P; ++i) {
            const float4 y = ld_dsmem_f4(mapa_shared(aa + 4 * ((i % kParts * G + r) * D + c), i / kParts));
            const float w = wt[r * P + i];
            if (w != 0.f) {  // (a part without slots may hold anything)
                x.x = fmaf(w, y.x, x.x); x.y = fmaf(w, y.y, x.y); x.z = fmaf(w, y.z, x.z); x.w = fmaf(w, y.w, x.w);
            }
        }
        T *dst = o + (size_t)r * D + c;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4 *>(dst) = x;
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(tc::pack_bf16(x.x, x.y), tc::pack_bf16(x.z, x.w));
    }
}

template <typename T>
__device__ __forceinline__ void write_zeros(T *o, int n)
{
    for (int e = threadIdx.x; e < n; e += blockDim.x) o[e] = Elem<T>::from_f32(0.f);
}

// ---------------------------------------------------------------- fp32, CUDA cores
// A lane holds 8 features of a key (D / 8 lanes a key, 256 / D keys a warp at a time), so that
// a score costs log2(D / 8) shuffles for as many keys at once; G heads' queries in registers.
constexpr int kSimtWarps = 4;
constexpr int kSimtKeys = 2;  // per lane in flight: more cost occupancy (2: 562 us, 4: 758, 8: 1270 with 4 features a lane)

struct Row8 {
    float4 a, b;  // features c .. c + 3 and D / 2 + c .. + 3
};
template <int D>
__device__ __forceinline__ Row8 row8(const float *p)
{
    return Row8{*reinterpret_cast<const float4 *>(p), *reinterpret_cast<const float4 *>(p + D / 2)};
}
template <int D>
__device__ __forceinline__ void put8(float *p, const Row8 &r)
{
    *reinterpret_cast<float4 *>(p) = r.a;
    *reinterpret_cast<float4 *>(p + D / 2) = r.b;
}
__device__ __forceinline__ float dot8(const Row8 &x, const Row8 &y)
{
    const float s = fmaf(x.a.w, y.a.w, fmaf(x.a.z, y.a.z, fmaf(x.a.y, y.a.y, x.a.x * y.a.x)));
    return fmaf(x.b.w, y.b.w, fmaf(x.b.z, y.b.z, fmaf(x.b.y, y.b.y, fmaf(x.b.x, y.b.x, s))));
}
// r = r f + x w
__device__ __forceinline__ void scale_add(Row8 &r, float f, const Row8 &x, float w)
{
    r.a.x = fmaf(x.a.x, w, r.a.x * f); r.a.y = fmaf(x.a.y, w, r.a.y * f);
    r.a.z = fmaf(x.a.z, w, r.a.z * f); r.a.w = fmaf(x.a.w, w, r.a.w * f);
    r.b.x = fmaf(x.b.x, w, r.b.x * f); r.b.y = fmaf(x.b.y, w, r.b.y * f);
    r.b.z = fmaf(x.b.z, w, r.b.z * f); r.b.w = fmaf(x.b.w, w, r.b.w * f);
}

template <int D, int G>
__global__ void __launch_bounds__(kSimtWarps * 32) decode_f32_kernel(const Args a)
{
    constexpr int LK = D / 8, KW = 32 / LK, U = kSimtKeys;  // lanes a key, keys a warp
    __shared__ __align__(16) float sm_m[kSimtWarps * G], sm_l[kSimtWarps * G], sm_acc[kSimtWarps * G * D];
    __shared__ float sm_wt[2 * G * kMaxCluster * kSimtWarps];
    const uint32_t S = cluster_size(), rank = S > 1 ? cluster_ctarank() : 0;
    const int unit = (int)(blockIdx.x / S), b = unit / a.Hk, hk = unit % a.Hk, group = a.Hq / a.Hk;
    const int g0 = (int)blockIdx.y * G, rows = min(G, group - g0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LK, c = (lane % LK) * 4;
    float *o = static_cast<float *>(a.o) + ((size_t)b * a.Hq + hk * group + g0) * D;
    const int pos = __ldg(a.pos + b);
    if (pos < 0) {
        if (rank == 0) write_zeros(o, rows * D);
        return;
    }
    const Slots sl(pos, a.window, a.sinks);
    const size_t cache = (size_t)unit * ((size_t)a.sinks + a.window) * D;
    float *kc = static_cast<float *>(a.kc) + cache, *vc = static_cast<float *>(a.vc) + cache;
    const float *kn = static_cast<const float *>(a.k) + (size_t)unit * D, *vn = static_cast<const float *>(a.v) + (size_t)unit * D;
    const Row8 none{make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    Row8 q[G], acc[G];
    float m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        q[g] = none;
        if (g < rows) q[g] = row8<D>(static_cast<const float *>(a.q) + ((size_t)b * a.Hq + hk * group + g0 + g) * D + c);
        m[g] = -INFINITY;
        l[g] = 0.f;
        acc[g] = none;
    }
    const float f = a.scale * kLog2e;
    const int workers = (int)S * kSimtWarps, me = (int)rank * kSimtWarps + warp;
    for (long long j0 = (long long)me * KW * U; j0 < sl.count; j0 += (long long)workers * KW * U) {
        Row8 kx[U], vx[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long j = j0 + u * KW + sub;
            in[u] = j < sl.count;
            kx[u] = vx[u] = none;
            if (in[u]) {
                const bool fresh = j == sl.fresh;
                kx[u] = row8<D>((fresh ? kn : kc + j * D) + c);
                vx[u] = row8<D>((fresh ? vn : vc + j * D) + c);
                if (fresh && blockIdx.y == 0) {
                    put8<D>(kc + j * D + c, kx[u]);
                    put8<D>(vc + j * D + c, vx[u]);
                }
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float s[U], top = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] = dot8(q[g], kx[u]);
#pragma unroll
                for (int d = LK / 2; d > 0; d /= 2) s[u] += __shfl_xor_sync(0xffffffffu, s[u], d);
                if (!in[u]) s[u] = -INFINITY;
                top = fmaxf(top, s[u]);
            }
            const float safe = top == -INFINITY ? 0.f : top;
            float keep = exp2f((m[g] - safe) * f);
            m[g] = top;
            l[g] *= keep;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p = exp2f((s[u] - safe) * f);
                l[g] += p;
                scale_add(acc[g], keep, vx[u], p);
                keep = 1.f;
            }
        }
    }
    // join the warp's keys, then leave the warp's result for the cluster
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float top = m[g];
#pragma unroll
        for (int d = LK; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float wt = m[g] == -INFINITY ? 0.f : exp2f((m[g] - top) * f);
        float ls = l[g] * wt;
        float x[8] = {acc[g].a.x, acc[g].a.y, acc[g].a.z, acc[g].a.w, acc[g].b.x, acc[g].b.y, acc[g].b.z, acc[g].b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= wt;
#pragma unroll
        for (int d = LK; d < 32; d *= 2) {
            ls += __shfl_xor_sync(0xffffffffu, ls, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], d);
        }
        if (sub == 0)
            put8<D>(&sm_acc[(warp * G + g) * D + c],
                    Row8{make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])});
        if (lane == 0) {
            sm_m[warp * G + g] = top;
            sm_l[warp * G + g] = ls;
        }
    }
    if (S > 1)
        cluster_sync_all();
    else
        __syncthreads();
    join<float, D, G, kSimtWarps>(sm_m, sm_l, sm_acc, sm_wt, rows, f, o, S, rank);
    if (S > 1) cluster_sync_all();  // no CTA leaves while its shared memory is read
}

// ---------------------------------------------------------------- bf16
// Up to 16 heads of a group against 16 slots at a time on the warp-level matrix unit
// (m16n8k16): S = q K^T, O += P V.  Sixteen rows are far below a tcgen05 tile, and the
// step moves 2 d e bytes for 4 d g operations a slot, so the matrix rate does not matter;
// the matrix form matters because one instruction replaces the shuffles and conversions
// that a dot product per lane needs (at four heads they alone would take the whole issue
// rate).  Slots reach shared memory by 16-byte asynchronous copies, kStages blocks of 16
// slots per warp in flight.  A lane's 16 bytes of a key serve two matrix steps: the order
// of the features inside a product is free, so q and K are both read in the order the
// bytes lie in.  P enters as a high and a low bf16 part (two products), so the only
// rounding of the weights is at 2^-16.
constexpr int kMmaWarps = 2;
constexpr int kStages = 3;
constexpr int kRows = 16;  // heads of one pass

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in)
{
    const int bytes = in ? 16 : 0;  // the rest is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Byte offset of 16-byte chunk ch of row r in a block of 16 rows of D features: chunks are
// permuted so that the 8 lanes of one shared-memory phase meet 8 bank groups (keys are read
// by two rows x four chunks, values by four row pairs x two chunks).
template <int D, bool kValues>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch)
{
    const int x = D < 64 ? 0 : kValues ? ((r >> 1) & 3) * 2 : (r & 1) * 4;
    return (uint32_t)(r * (D * 2) + ((ch ^ x) << 4));
}

template <int D>
struct MmaSmem {
    static constexpr int kBlock = 16 * D * 2;  // bytes of 16 keys (or values)
    uint8_t ring[kMmaWarps][kStages][2 * kBlock];
    float m[kMmaWarps * kRows], l[kMmaWarps * kRows], wt[2 * kRows * kMaxCluster * kMmaWarps];
    // the warps' outputs [kMmaWarps][16][D] take the ring's place at the end
    static_assert(kStages * 2 * kBlock >= kRows * D * 4, "a warp's output fits its part of the ring");
};

template <int D>
__global__ void __launch_bounds__(kMmaWarps * 32) decode_bf16_kernel(const Args a)
{
    extern __shared__ __align__(128) uint8_t smem_raw[];
    MmaSmem<D> &sm = *reinterpret_cast<MmaSmem<D> *>(smem_raw);
    constexpr int kBlock = MmaSmem<D>::kBlock, kChunks = D / 8;
    constexpr int NU = D / 32;                // 32-feature groups of q and K
    constexpr int NW = D > 64 ? 2 : 1;        // 64-feature halves of V
    constexpr int NT = D > 32 ? 8 : 4;        // features a lane holds of each half
    const uint32_t S = cluster_size(), rank = S > 1 ? cluster_ctarank() : 0;
    const int unit = (int)(blockIdx.x / S), b = unit / a.Hk, hk = unit % a.Hk, group = a.Hq / a.Hk;
    const int g0 = (int)blockIdx.y * kRows, rows = min(kRows, group - g0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + ((size_t)b * a.Hq + hk * group + g0) * D;
    const int pos = __ldg(a.pos + b);
    if (pos < 0) {
        if (rank == 0) write_zeros(o, rows * D);
        return;
    }
    const Slots sl(pos, a.window, a.sinks);
    const size_t cache = (size_t)unit * ((size_t)a.sinks + a.window) * D;
    __nv_bfloat16 *kc = static_cast<__nv_bfloat16 *>(a.kc) + cache, *vc = static_cast<__nv_bfloat16 *>(a.vc) + cache;
    const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(a.k) + (size_t)unit * D;
    const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(a.v) + (size_t)unit * D;

    // 16-slot blocks of this warp: first, first + workers, ...
    const int blocks = (sl.count + 15) / 16, workers = (int)S * kMmaWarps;
    const int first = (int)rank * kMmaWarps + warp;
    const int mine = blocks > first ? (blocks - first + workers - 1) / workers : 0;
    const uint32_t ring = smem_u32(sm.ring[warp]);

    auto fetch = [&](int i) {
        if (i < mine) {
            const int j0 = (first + i * workers) * 16;
            const uint32_t dst = ring + (i % kStages) * 2 * kBlock;
#pragma unroll
            for (int u = 0; u < 16 * kChunks / 32; ++u) {
                const int row = (u * 32 + lane) / kChunks, ch = (u * 32 + lane) % kChunks, j = j0 + row;
                const bool in = j < sl.count, fresh = j == sl.fresh;
                const size_t at = (size_t)(in ? j : 0) * D + ch * 8;
                copy16(dst + chunk_at<D, false>(row, ch), fresh ? kn + ch * 8 : kc + at, in);
                copy16(dst + kBlock + chunk_at<D, true>(row, ch), fresh ? vn + ch * 8 : vc + at, in);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // q of heads r and r + 8 in the order of K's bytes
    uint32_t qa[NU][2][4];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
        const __nv_bfloat16 *qp =
            static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * a.Hq + hk * group + g0 + r) * D + u * 32 + c * 8;
        if (r < rows) x0 = *reinterpret_cast<const uint4 *>(qp);
        if (r + 8 < rows) x1 = *reinterpret_cast<const uint4 *>(qp + 8 * D);
        qa[u][0][0] = x0.x; qa[u][0][1] = x1.x; qa[u][0][2] = x0.y; qa[u][0][3] = x1.y;
        qa[u][1][0] = x0.z; qa[u][1][1] = x1.z; qa[u][1][2] = x0.w; qa[u][1][3] = x1.w;
    }
    float acc[NW][NT][4];
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[w][t][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const float f = a.scale * kLog2e;

    for (int i = 0; i < mine; ++i) {
        copy_wait<kStages - 2>();
        __syncwarp();  // every lane's copies of this block have landed; the block before is read
        fetch(i + kStages - 1);
        const uint8_t *kb = sm.ring[warp][i % kStages], *vb = kb + kBlock;
        const int j0 = (first + i * workers) * 16;
        float s[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const uint4 x = *reinterpret_cast<const uint4 *>(kb + chunk_at<D, false>(8 * t + r, 4 * u + c));
                mma16816(s[t], qa[u][0], x.x, x.y);
                mma16816(s[t], qa[u][1], x.z, x.w);
            }
        }
        float t0 = m0, t1 = m1;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool in = j0 + 8 * t + 2 * c + e < sl.count;
                s[t][e] = in ? s[t][e] : -INFINITY;
                s[t][2 + e] = in ? s[t][2 + e] : -INFINITY;
                t0 = fmaxf(t0, s[t][e]);
                t1 = fmaxf(t1, s[t][2 + e]);
            }
#pragma unroll
        for (int d = 1; d < 4; d *= 2) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
        }
        if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
            const float k0 = t0 == -INFINITY ? 1.f : exp2f((m0 - t0) * f), k1 = t1 == -INFINITY ? 1.f : exp2f((m1 - t1) * f);
            l0 *= k0;
            l1 *= k1;
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[w][t][0] *= k0; acc[w][t][1] *= k0;
                    acc[w][t][2] *= k1; acc[w][t][3] *= k1;
                }
            m0 = t0;
            m1 = t1;
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float z = h ? z1 : z0;
                const float p0 = exp2f((s[t][2 * h] - z) * f), p1 = exp2f((s[t][2 * h + 1] - z) * f);
                if (h) l1 += p0 + p1; else l0 += p0 + p1;
                const __nv_bfloat162 x = __floats2bfloat162_rn(p0, p1);
                hi[2 * t + h] = *reinterpret_cast<const uint32_t *>(&x);
                lo[2 * t + h] = tc::pack_bf16(p0 - __bfloat162float(x.x), p1 - __bfloat162float(x.y));
            }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            uint32_t x[4][NT / 2];  // values of slots 2c, 2c + 1, 2c + 8, 2c + 9: features 64 w + NT r ..
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 2 * c + (e & 1) + 8 * (e >> 1);
                if (NT == 8) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(vb + chunk_at<D, true>(row, 8 * w + r));
                    x[e][0] = y.x; x[e][1] = y.y; x[e][NT / 2 - 2] = y.z; x[e][NT / 2 - 1] = y.w;
                } else {
                    const uint2 y = *reinterpret_cast<const uint2 *>(vb + chunk_at<D, true>(row, r >> 1) + (r & 1) * 8);
                    x[e][0] = y.x; x[e][1] = y.y;
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t sel = (t & 1) ? 0x7632u : 0x5410u;
                const uint32_t b0 = __byte_perm(x[0][t / 2], x[1][t / 2], sel), b1 = __byte_perm(x[2][t / 2], x[3][t / 2], sel);
                mma16816(acc[w][t], hi, b0, b1);
                mma16816(acc[w][t], lo, b0, b1);
            }
        }
    }
    copy_wait<0>();
    // the new token into its slot: by the warp whose block holds it
    if (blockIdx.y == 0 && (sl.fresh / 16) % workers == first) {
        for (int e = lane; e < D; e += 32) {
            kc[(size_t)sl.fresh * D + e] = kn[e];
            vc[(size_t)sl.fresh * D + e] = vn[e];
        }
    }
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    __syncthreads();  // the rings are read: they become the warps' outputs
    float *out = reinterpret_cast<float *>(smem_raw) + warp * kRows * D;
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[(r + 8 * (e >> 1)) * D + 64 * w + (2 * c + (e & 1)) * NT + t] = acc[w][t][e];
    if (c == 0) {
        sm.m[warp * kRows + r] = m0;
        sm.m[warp * kRows + r + 8] = m1;
        sm.l[warp * kRows + r] = l0;
        sm.l[warp * kRows + r + 8] = l1;
    }
    if (S > 1)
        cluster_sync_all();
    else
        __syncthreads();
    join<__nv_bfloat16, D, kRows, kMmaWarps>(sm.m, sm.l, reinterpret_cast<const float *>(smem_raw), sm.wt, rows, f, o, S, rank);
    if (S > 1) cluster_sync_all();  // no CTA leaves while its shared memory is read
}

// CTAs per (entry, key head): one while there are at least two waves of them, else enough to
// fill the machine, each still with two blocks a warp.
int split(long long units, long long slots, int per_cta)
{
    int S = 1;
    while (S < kMaxCluster && units * S < 2LL * tc::sm_count() && slots > 2LL * per_cta * S) S *= 2;
    return S;
}

template <typename K>
la_status launch(K kern, const WindowDecodeProblem &p, int heads, int threads, size_t smem, int per_cta)
{
    const long long units = (long long)p.B * p.Hk;
    const int S = split(units, (long long)p.sinks + p.window, per_cta);
    if (units * S > 0x7fffffffLL || ceil_div(p.Hq / p.Hk, heads) > 65535) return LA_ERR_UNSUPPORTED;
    la_status st = smem ? ensure_smem((const void *)kern, (int)smem) : LA_OK;
    if (st != LA_OK) return st;
    Args a{p.kc, p.vc, p.q, p.k, p.v, p.o, p.pos, p.Hq, p.Hk, p.window, p.sinks, p.scale};
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(units * S), (unsigned)ceil_div(p.Hq / p.Hk, heads));
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = smem;
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

template <int D>
la_status decode(const WindowDecodeProblem &p)
{
    if (p.dtype == LA_BF16) return launch(decode_bf16_kernel<D>, p, kRows, kMmaWarps * 32, sizeof(MmaSmem<D>), kMmaWarps * 16);
    const int per_cta = kSimtWarps * (256 / D) * kSimtKeys, group = p.Hq / p.Hk;
    if (group == 1) return launch(decode_f32_kernel<D, 1>, p, 1, kSimtWarps * 32, 0, per_cta);
    if (group == 2) return launch(decode_f32_kernel<D, 2>, p, 2, kSimtWarps * 32, 0, per_cta);
    return launch(decode_f32_kernel<D, 4>, p, 4, kSimtWarps * 32, 0, per_cta);
}

// ---------------------------------------------------------------- prefill
// Copies the tokens that are still visible after the first n into their slots: one 16-byte
// chunk a thread, slots in order.
struct FillArgs {
    const uint4 *k, *v;
    uint4 *kc, *vc;
    const int *lens;
    int Hk, N, window, sinks, chunks;
    long long total;  // chunks of kc
};
__global__ void __launch_bounds__(256) fill_kernel(const FillArgs a)
{
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= a.total) return;
    const int ch = (int)(e % a.chunks);
    const long long row = e / a.chunks, slots = (long long)a.sinks + a.window;
    const long long unit = row / slots, slot = row % slots;
    const int n = window::valid(a.lens, (int)(unit / a.Hk), a.N);
    long long j = slot;
    if (slot >= a.sinks) {  // the last token of this slot
        const long long past = (long long)n - 1 - slot;
        if (past < 0) return;
        j = slot + past / a.window * a.window;
    }
    if (j >= n) return;
    const size_t src = ((size_t)unit * a.N + j) * a.chunks + ch;
    a.kc[e] = a.k[src];
    a.vc[e] = a.v[src];
}

}  // namespace

la_status window_decode(const WindowDecodeProblem &p)
{
    if (p.d == 32) return decode<32>(p);
    return p.d == 64 ? decode<64>(p) : decode<128>(p);
}

la_status window_cache(const void *k, const void *v, void *kc, void *vc, const int *lens, int B, int Hk, int N, int d,
                       int window, int sinks, la_dtype dtype, cudaStream_t stream)
{
    FillArgs a;
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.kc = static_cast<uint4 *>(kc);
    a.vc = static_cast<uint4 *>(vc);
    a.lens = lens;
    a.Hk = Hk;
    a.N = N;
    a.window = window;
    a.sinks = sinks;
    a.chunks = d * (dtype == LA_F32 ? 4 : 2) / 16;
    a.total = (long long)B * Hk * ((long long)sinks + window) * a.chunks;
    const long long ctas = (a.total + 255) / 256;
    if (ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    count_launches();
    fill_kernel<<<(unsigned)ctas, 256, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace la
