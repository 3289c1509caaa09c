// Group norm with an activation or a gate, channels last, and its gradients.
//
//   h = (x - m) r,  r = 1 / sqrt(var + eps),  z = h w + b,  y = act(z)  or  y = z act(gate)
//
// Two shapes of problem, both bound by memory: groups of one token's channels (per_token, the norm
// behind the heads of linear attention), where a few lanes hold a group in registers and every
// tensor is read once; and groups over all positions, where sums per channel come first.  Statistics
// are fp32 sums of differences (from the mean, or from the channel's first value).
#include <type_traits>

#include "la_common.cuh"
#include "la_internal.h"

namespace la {
namespace {

struct Params {
    const void *x, *gate, *dy;
    const float *w, *b, *mean, *rstd;
    void *y, *dx, *dgate;
    float *mean_out, *rstd_out;
    float *part;  // partial sums: [rows][2][C]
    int B, L, C, G, D;
    float eps;
    int heads_first, center, act;
    int splits, rows;  // over positions: splits of an entry, positions a split
};

// VEC elements of T at p as floats, and back.
template <typename T, int VEC> struct Pack {
    static __device__ __forceinline__ void get(const T *p, float (&v)[VEC])
    {
        static_assert(VEC == 1, "");
        v[0] = Elem<T>::to_f32(__ldg(p));
    }
    static __device__ __forceinline__ void put(T *p, const float (&v)[VEC]) { p[0] = Elem<T>::from_f32(v[0]); }
};
template <> struct Pack<float, 4> {
    static __device__ __forceinline__ void get(const float *p, float (&v)[4])
    {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    }
    static __device__ __forceinline__ void put(float *p, const float (&v)[4])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct Pack<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void get(const __nv_bfloat16 *p, float (&v)[8])
    {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// silu and its slope.  bf16 results take the fast exponential and division (2 ulp of fp32 each).
template <typename T> __device__ __forceinline__ float sigmoid(float z)
{
    return std::is_same<T, float>::value ? 1.f / (1.f + expf(-z)) : __fdividef(1.f, 1.f + __expf(-z));
}
template <typename T> __device__ __forceinline__ float act_of(float z, int act) { return act == LA_ACT_SILU ? z * sigmoid<T>(z) : z; }
template <typename T> __device__ __forceinline__ float act_slope(float z, int act, float *value)
{
    if (act != LA_ACT_SILU) {
        *value = z;
        return 1.f;
    }
    const float s = sigmoid<T>(z);
    *value = z * s;
    return s * fmaf(z, 1.f - s, 1.f);
}

// What one element passes back: dz = dL/dz, and dL/dgate.
template <typename T, bool kGate>
__device__ __forceinline__ float back(float h, float w, float b, float dy, float gate, int act, float *dgate)
{
    const float z = fmaf(h, w, b);
    float value;
    if (!kGate) return dy * act_slope<T>(z, act, &value);
    const float slope = act_slope<T>(gate, act, &value);
    *dgate = dy * z * slope;
    return dy * value;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// ---------------------------------------------------------------- a token's groups
// `lanes` lanes hold a group, VEC neighbouring channels at a time, NV times.  A slot of lanes keeps
// to one group of channels (slot % G), so weights, and the sums for their gradients, stay in
// registers, and walks over the tokens; the launch has a whole number of slots for each group.
template <typename T, int VEC, int NV, bool kGate, bool kBack>
__global__ void __launch_bounds__(256) norm_tokens(Params p, int lanes, long long slots)
{
    const int lane = threadIdx.x & (lanes - 1), per_block = 256 / lanes, local = threadIdx.x / lanes;
    const long long slot = (long long)blockIdx.x * per_block + local, tokens = (long long)p.B * p.L;
    const int g = (int)(slot % p.G);
    const float inv = 1.f / p.D;
    float w[NV][VEC], b[NV][VEC], dw[kBack ? NV : 1][VEC], db[kBack ? NV : 1][VEC];
    bool in[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = (lane + n * lanes) * VEC;
        in[n] = c < p.D;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[n][e] = in[n] ? (p.w ? __ldg(p.w + g * p.D + c + e) : 1.f) : 0.f;
            b[n][e] = in[n] && p.b ? __ldg(p.b + g * p.D + c + e) : 0.f;
            if (kBack) dw[n][e] = db[n][e] = 0.f;
        }
    }
    // every lane of a warp runs the same trips (the sums take all lanes): a slot past the last
    // token reads nothing and writes nothing
    const long long step = slots / p.G, first = slot / p.G, warp_first = ((long long)blockIdx.x * per_block + (threadIdx.x & ~31) / lanes) / p.G;
    for (long long t = first, wt = warp_first; wt < tokens; t += step, wt += step) {
        const bool live = t < tokens;
        const size_t flat = ((size_t)t * p.G + g) * p.D;
        const size_t xat = p.heads_first ? ((size_t)(t / p.L * p.G + g) * p.L + t % p.L) * p.D : flat;
        float x[NV][VEC], ga[kGate ? NV : 1][VEC], dy[kBack ? NV : 1][VEC];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = (lane + n * lanes) * VEC;
            const bool on = live && in[n];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                x[n][e] = 0.f;
                if (kGate) ga[n][e] = 0.f;
                if (kBack) dy[n][e] = 0.f;
            }
            if (on) {
                Pack<T, VEC>::get(static_cast<const T *>(p.x) + xat + c, x[n]);
                if (kGate) Pack<T, VEC>::get(static_cast<const T *>(p.gate) + flat + c, ga[n]);
                if (kBack) Pack<T, VEC>::get(static_cast<const T *>(p.dy) + flat + c, dy[n]);
            }
        }
        const size_t st = (size_t)t * p.G + g;
        if (!kBack) {
            float m = 0.f, v = 0.f;
            if (p.center) {
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) m += x[n][e];
                m = lanes_sum(m, lanes) * inv;
            }
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    x[n][e] -= m;
                    if (in[n]) v = fmaf(x[n][e], x[n][e], v);
                }
            const float r = 1.f / sqrtf(fmaf(lanes_sum(v, lanes), inv, p.eps));
            if (!live) continue;
            if (lane == 0) {
                if (p.mean_out && p.center) p.mean_out[st] = m;
                if (p.rstd_out) p.rstd_out[st] = r;
            }
#pragma unroll
            for (int n = 0; n < NV; ++n) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float z = fmaf(x[n][e] * r, w[n][e], b[n][e]);
                    x[n][e] = kGate ? z * act_of<T>(ga[n][e], p.act) : act_of<T>(z, p.act);
                }
                if (in[n]) Pack<T, VEC>::put(static_cast<T *>(p.y) + flat + (lane + n * lanes) * VEC, x[n]);
            }
        } else {
            const float m = live && p.center ? __ldg(p.mean + st) : 0.f, r = live ? __ldg(p.rstd + st) : 0.f;
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (x[n][e] - m) * r;
                    float dg = 0.f;
                    const float dz = back<T, kGate>(h, w[n][e], b[n][e], dy[n][e], kGate ? ga[n][e] : 0.f, p.act, &dg);
                    if (kGate) ga[n][e] = dg;
                    if (in[n] && live) {
                        dw[n][e] = fmaf(dz, h, dw[n][e]);
                        db[n][e] += dz;
                    }
                    const float dh = in[n] ? dz * w[n][e] : 0.f;
                    s1 += dh;
                    s2 = fmaf(dh, h, s2);
                    x[n][e] = h;
                    dy[n][e] = dh;
                }
            s1 = p.center ? lanes_sum(s1, lanes) * inv : 0.f;
            s2 = lanes_sum(s2, lanes) * inv;
            if (!live) continue;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[n][e] = r * (dy[n][e] - s1 - x[n][e] * s2);
                if (in[n]) {
                    Pack<T, VEC>::put(static_cast<T *>(p.dx) + xat + (lane + n * lanes) * VEC, x[n]);
                    if (kGate) Pack<T, VEC>::put(static_cast<T *>(p.dgate) + flat + (lane + n * lanes) * VEC, ga[n]);
                }
            }
        }
    }
    if (kBack && p.part) {
        // the block's sums: slots of one group are added in order, then written to the row of the partial sums that
        // the block (or, where a block holds fewer slots than there are groups, its run of slots) owns
        extern __shared__ float sums[];  // [slots][D]
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NV; ++n)
                if (in[n])
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        sums[local * p.D + (lane + n * lanes) * VEC + e] = which ? db[n][e] : dw[n][e];
            __syncthreads();
            const int own = min(per_block, p.G);
            const long long s0 = (long long)blockIdx.x * per_block;
            for (int i = threadIdx.x; i < own * p.D; i += 256) {
                const int sl = i / p.D, c = i % p.D;
                float v = 0.f;
                for (int k = sl; k < per_block; k += p.G) v += sums[k * p.D + c];
                const long long row = per_block >= p.G ? blockIdx.x : (s0 + sl) / p.G;
                p.part[((size_t)row * 2 + which) * p.C + (size_t)((s0 + sl) % p.G) * p.D + c] = v;
            }
        }
    }
}

// ---------------------------------------------------------------- groups over all positions
// Columns of VEC channels, `cols` of them to a block of 256 threads; the other threads of a column take
// further positions.  Sums per channel and split, joined in shared memory in a fixed order.
template <typename T, int VEC, bool kGate, bool kBack>
__global__ void __launch_bounds__(256) norm_sums(Params p, int cols)
{
    extern __shared__ float sums[];  // [2][threads of a column][cols * VEC]
    const int tx = threadIdx.x % cols, ty = threadIdx.x / cols, ny = 256 / cols;
    const int c = (blockIdx.z * cols + tx) * VEC, bi = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const bool on = ty < ny && c < p.C;
    float s1[VEC] = {}, s2[VEC] = {};
    if (on) {
        const T *x = static_cast<const T *>(p.x) + (size_t)bi * p.L * p.C + c;
        const T *dy = static_cast<const T *>(p.dy) + (kBack ? (size_t)bi * p.L * p.C + c : 0);
        const T *gate = static_cast<const T *>(p.gate) + (kGate ? (size_t)bi * p.L * p.C + c : 0);
        float shift[VEC], r[VEC], w[VEC], b[VEC];
        if (!kBack) {
            Pack<T, VEC>::get(x, shift);  // differences from the channel's first value (from 0 without centring)
            if (!p.center)
#pragma unroll
                for (int e = 0; e < VEC; ++e) shift[e] = 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const size_t st = (size_t)bi * p.G + (c + e) / p.D;
                shift[e] = p.center ? __ldg(p.mean + st) : 0.f;
                r[e] = __ldg(p.rstd + st);
                w[e] = p.w ? __ldg(p.w + c + e) : 1.f;
                b[e] = p.b ? __ldg(p.b + c + e) : 0.f;
            }
        }
        const int l1 = min(p.L, (split + 1) * p.rows);
#pragma unroll 4
        for (int l = split * p.rows + ty; l < l1; l += ny) {
            float v[VEC], d[VEC], ga[VEC];
            Pack<T, VEC>::get(x + (size_t)l * p.C, v);
            if (kBack) Pack<T, VEC>::get(dy + (size_t)l * p.C, d);
            if (kGate) Pack<T, VEC>::get(gate + (size_t)l * p.C, ga);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (kBack) {
                    const float h = (v[e] - shift[e]) * r[e];
                    float dg;
                    const float dz = back<T, kGate>(h, w[e], b[e], d[e], kGate ? ga[e] : 0.f, p.act, &dg);
                    s1[e] = fmaf(dz, h, s1[e]);
                    s2[e] += dz;
                } else {
                    const float t = v[e] - shift[e];
                    s1[e] += t;
                    s2[e] = fmaf(t, t, s2[e]);
                }
            }
        }
    }
    const int width = cols * VEC;
    if (ty < ny)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sums[ty * width + tx * VEC + e] = s1[e];
            sums[(ny + ty) * width + tx * VEC + e] = s2[e];
        }
    __syncthreads();
    float *out = p.part + ((size_t)bi * p.splits + split) * 2 * p.C;
    for (int i = threadIdx.x; i < 2 * width; i += 256) {
        const int which = i / width, j = i % width, ch = blockIdx.z * width + j;
        float v = 0.f;
        for (int k = 0; k < ny; ++k) v += sums[(which * ny + k) * width + j];
        if (ch < p.C) out[(size_t)which * p.C + ch] = v;
    }
}

__device__ __forceinline__ float block_sum(float v, float *tmp)
{
    v = lanes_sum(v, 32);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    return (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
}

// A group's statistics from its channels' sums: the mean of the channels' means, and their
// squared deviations about it.
template <typename T>
__global__ void __launch_bounds__(128) norm_statistics(Params p)
{
    __shared__ float tmp[4];
    const int bi = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const float *part = p.part + (size_t)bi * p.splits * 2 * p.C;
    const T *x = static_cast<const T *>(p.x) + (size_t)bi * p.L * p.C;
    auto channel = [&](int c, float *mean, float *m2) {
        float s1 = 0.f, s2 = 0.f;
        for (int s = 0; s < p.splits; ++s) {
            s1 += part[(size_t)s * 2 * p.C + c];
            s2 += part[((size_t)s * 2 + 1) * p.C + c];
        }
        if (!p.center) {
            *mean = 0.f, *m2 = s2;
            return;
        }
        const float d = s1 / p.L;
        *mean = Elem<T>::to_f32(x[c]) + d;
        *m2 = fmaxf(0.f, fmaf(-s1, d, s2));
    };
    const float inv = 1.f / p.D;
    float a = 0.f, mean0 = 0.f, sq0 = 0.f;  // the thread's first channel is kept: most groups have no more
    for (int c = threadIdx.x; c < p.D; c += 128) {
        float mc, m2;
        channel(g * p.D + c, &mc, &m2);
        if (c == threadIdx.x) mean0 = mc, sq0 = m2;
        a += mc;
    }
    const float m = block_sum(a, tmp) * inv;
    float v = 0.f;
    for (int c = threadIdx.x; c < p.D; c += 128) {
        float mc = mean0, m2 = sq0;
        if (c != threadIdx.x) channel(g * p.D + c, &mc, &m2);
        const float d = p.center ? mc - m : 0.f;
        v += fmaf(d * d, (float)p.L, m2);
    }
    v = block_sum(v, tmp) * inv / p.L;
    if (threadIdx.x == 0) {
        if (p.center) p.mean_out[blockIdx.x] = m;
        p.rstd_out[blockIdx.x] = 1.f / sqrtf(v + p.eps);
    }
}

// The two means of a group that its dx takes off: of dh = dz w (into mean_out) and of dh h (rstd_out).
__global__ void __launch_bounds__(128) norm_group_means(Params p)
{
    __shared__ float tmp[4];
    const int bi = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const float *part = p.part + (size_t)bi * p.splits * 2 * p.C;
    float a = 0.f, v = 0.f;
    for (int i = threadIdx.x; i < p.D * p.splits; i += 128) {
        const int c = g * p.D + i % p.D;
        const float *at = part + (size_t)(i / p.D) * 2 * p.C + c, w = p.w ? p.w[c] : 1.f;
        v = fmaf(w, at[0], v);
        a = fmaf(w, at[p.C], a);
    }
    const float inv = 1.f / p.D / p.L;
    a = block_sum(a, tmp);
    v = block_sum(v, tmp);
    if (threadIdx.x == 0) {
        p.mean_out[blockIdx.x] = p.center ? a * inv : 0.f;
        p.rstd_out[blockIdx.x] = v * inv;
    }
}

// y, or dx and dgate, of all positions.
template <typename T, int VEC, bool kGate, bool kBack>
__global__ void __launch_bounds__(256) norm_apply(Params p, int cols)
{
    const int tx = threadIdx.x % cols, ty = threadIdx.x / cols, ny = 256 / cols;
    const int c = (blockIdx.z * cols + tx) * VEC, bi = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    if (ty >= ny || c >= p.C) return;
    float m[VEC], r[VEC], w[VEC], b[VEC], a1[VEC], a2[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const size_t st = (size_t)bi * p.G + (c + e) / p.D;
        m[e] = p.center ? p.mean[st] : 0.f;
        r[e] = p.rstd[st];
        w[e] = p.w ? __ldg(p.w + c + e) : 1.f;
        b[e] = p.b ? __ldg(p.b + c + e) : 0.f;
        if (kBack) a1[e] = p.mean_out[st], a2[e] = p.rstd_out[st];
    }
    const size_t base = (size_t)bi * p.L * p.C + c;
    const int l1 = min(p.L, (split + 1) * p.rows);
#pragma unroll 4
    for (int l = split * p.rows + ty; l < l1; l += ny) {
        const size_t at = base + (size_t)l * p.C;
        float v[VEC], d[VEC], ga[VEC];
        Pack<T, VEC>::get(static_cast<const T *>(p.x) + at, v);
        if (kGate) Pack<T, VEC>::get(static_cast<const T *>(p.gate) + at, ga);
        if (kBack) Pack<T, VEC>::get(static_cast<const T *>(p.dy) + at, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float h = (v[e] - m[e]) * r[e];
            if (kBack) {
                float dg = 0.f;
                const float dz = back<T, kGate>(h, w[e], b[e], d[e], kGate ? ga[e] : 0.f, p.act, &dg);
                v[e] = r[e] * (fmaf(dz, w[e], -a1[e]) - h * a2[e]);
                ga[e] = dg;
            } else {
                const float z = fmaf(h, w[e], b[e]);
                v[e] = kGate ? z * act_of<T>(ga[e], p.act) : act_of<T>(z, p.act);
            }
        }
        Pack<T, VEC>::put(static_cast<T *>(kBack ? p.dx : p.y) + at, v);
        if (kBack && kGate) Pack<T, VEC>::put(static_cast<T *>(p.dgate) + at, ga);
    }
}

// dw and db: the sum of all rows of the partial sums, 32 channels a block, in a fixed order.
__global__ void __launch_bounds__(1024) norm_weight_grads(const float *part, float *dw, float *db, long long rows, int C)
{
    __shared__ float tmp[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
    float *out = which ? db : dw;
    if (!out) return;
    float v = 0.f;
    if (c < C)
#pragma unroll 8
        for (long long r = threadIdx.y; r < rows; r += 32) v += part[((size_t)r * 2 + which) * C + c];
    tmp[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = lanes_sum(tmp[threadIdx.x][threadIdx.y], 32);
    const int cy = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cy < C) out[cy] = v;
}

// ---------------------------------------------------------------- launches
constexpr int kSMs = 152;

Params params_of(const NormProblem &p)
{
    Params q{};
    q.x = p.x, q.gate = p.gate, q.dy = p.dy, q.w = p.w, q.b = p.b, q.mean = p.mean, q.rstd = p.rstd;
    q.y = p.y, q.dx = p.dx, q.dgate = p.dgate, q.mean_out = p.mean_out, q.rstd_out = p.rstd_out;
    q.B = p.B, q.L = p.L, q.C = p.C, q.G = p.spec.groups, q.D = p.C / p.spec.groups;
    q.eps = p.spec.eps, q.heads_first = p.spec.heads_first, q.center = p.spec.center, q.act = p.spec.act;
    return q;
}

// Lanes and registers of a token's group: the widest vectors that divide it.
struct TokenShape {
    int vec, nv, lanes;
    long long blocks, slots, part_rows;
};
TokenShape token_shape(const NormProblem &p)
{
    TokenShape s;
    const int G = p.spec.groups, D = p.C / G, full = p.dtype == LA_F32 ? 4 : 8;
    s.vec = D % full == 0 ? full : 1;
    const int n = D / s.vec;  // vectors of a group
    s.nv = 1;
    while (s.nv * 32 < n) s.nv *= s.vec == 1 ? 4 : 2;
    s.lanes = 1;
    while (s.lanes * s.nv < n) s.lanes *= 2;
    const int per_block = 256 / s.lanes;
    const long long tokens = (long long)p.B * p.L, all = tokens * G;
    // whole slots for each group: blocks come in multiples of G / gcd(G, slots of a block)
    int a = G, b = per_block;
    while (b) {
        const int t = a % b;
        a = b;
        b = t;
    }
    const long long unit = G / a;
    const long long need = (all + per_block - 1) / per_block, most = (long long)kSMs * (p.backward ? 4 : 8);
    s.blocks = (need < most ? need : most);
    s.blocks = (s.blocks + unit - 1) / unit * unit;
    s.slots = s.blocks * per_block;
    s.part_rows = per_block >= G ? s.blocks : s.slots / G;
    return s;
}

struct MapShape {
    int vec, cols, zs, splits, rows;
};
MapShape map_shape(const NormProblem &p)
{
    MapShape s;
    const int full = p.dtype == LA_F32 ? 4 : 8;
    s.vec = p.C % full == 0 ? full : 1;
    const int n = p.C / s.vec;
    s.zs = ceil_div(n, 256);
    s.cols = ceil_div(n, s.zs);
    const int ny = 256 / s.cols;
    const long long blocks = (long long)p.B * s.zs;
    int want = (int)((kSMs * 6 + blocks - 1) / blocks);
    const int most = ceil_div(p.L, ny * 4);
    want = want < most ? want : most;
    if (want < 1) want = 1;
    s.rows = ceil_div(p.L, want);
    s.splits = ceil_div(p.L, s.rows);
    return s;
}

bool by_token(const NormProblem &p) { return p.spec.per_token && p.C / p.spec.groups <= kNormTokenChannels; }

// An entry's groups of one token wider than the token kernel's registers: entries of one position.
NormProblem as_map(const NormProblem &p)
{
    NormProblem q = p;
    if (p.spec.per_token) q.B = p.B * p.L, q.L = 1;
    return q;
}

template <typename T, bool kGate, bool kBack> la_status launch_tokens(const NormProblem &p, Params q)
{
    const TokenShape s = token_shape(p);
    const int smem = kBack && q.part ? 256 / s.lanes * q.D * 4 : 0;  // at most 16 KB
    constexpr int kFull = std::is_same<T, float>::value ? 4 : 8;
    auto go = [&](auto kernel) {
        count_launches();
        kernel<<<(unsigned)s.blocks, 256, smem, p.stream>>>(q, s.lanes, s.slots);
        return cuda_status(cudaGetLastError());
    };
    if (s.vec == 1) {
        if (s.nv == 1) return go(&norm_tokens<T, 1, 1, kGate, kBack>);
        if (s.nv == 4) return go(&norm_tokens<T, 1, 4, kGate, kBack>);
        return go(&norm_tokens<T, 1, 16, kGate, kBack>);
    }
    if (s.nv == 1) return go(&norm_tokens<T, kFull, 1, kGate, kBack>);
    if (s.nv == 2) return go(&norm_tokens<T, kFull, 2, kGate, kBack>);
    return go(&norm_tokens<T, kFull, 4, kGate, kBack>);
}

template <typename T, bool kGate, bool kBack> la_status launch_map(const NormProblem &p, Params q)
{
    const MapShape s = map_shape(p);
    constexpr int kFull = std::is_same<T, float>::value ? 4 : 8;
    q.splits = s.splits, q.rows = s.rows;
    const dim3 grid((unsigned)s.splits * p.B, 1, (unsigned)s.zs);
    const int smem = 2 * (256 / s.cols) * s.cols * s.vec * 4;
    auto sums = s.vec == 1 ? &norm_sums<T, 1, kGate && kBack, kBack> : &norm_sums<T, kFull, kGate && kBack, kBack>;
    auto apply = s.vec == 1 ? &norm_apply<T, 1, kGate, kBack> : &norm_apply<T, kFull, kGate, kBack>;
    count_launches(3);
    sums<<<grid, 256, smem, p.stream>>>(q, s.cols);
    if (kBack)
        norm_group_means<<<(unsigned)(p.B * q.G), 128, 0, p.stream>>>(q);
    else
        norm_statistics<T><<<(unsigned)(p.B * q.G), 128, 0, p.stream>>>(q);
    if (!kBack) q.mean = q.mean_out, q.rstd = q.rstd_out;
    apply<<<grid, 256, 0, p.stream>>>(q, s.cols);
    return cuda_status(cudaGetLastError());
}

template <bool kBack> la_status launch(const NormProblem &p, const Params &q)
{
    auto go = [&](auto t, auto gate) {
        using T = decltype(t);
        return by_token(p) ? launch_tokens<T, decltype(gate)::value, kBack>(p, q)
                           : launch_map<T, decltype(gate)::value, kBack>(p, q);
    };
    auto typed = [&](auto t) { return p.gate ? go(t, std::true_type()) : go(t, std::false_type()); };
    return p.dtype == LA_F32 ? typed(0.f) : typed(__nv_bfloat16());
}

}  // namespace

// Scratch: partial sums, then two values a group.
size_t norm_scratch(const NormProblem &p)
{
    const bool grads = p.backward && (p.dw || p.db);
    if (by_token(p)) return grads ? (size_t)token_shape(p).part_rows * 2 * p.C * 4 : 0;
    const NormProblem q = as_map(p);
    return ((size_t)q.B * map_shape(q).splits * 2 * p.C + 2 * (size_t)q.B * p.spec.groups) * 4;
}

la_status group_norm(const NormProblem &given)
{
    const bool tokens = by_token(given), grads = given.backward && (given.dw || given.db);
    const NormProblem p = tokens ? given : as_map(given);
    Params q = params_of(p);
    long long rows = 0;
    if (tokens) {
        q.part = grads ? p.scratch : nullptr;
        if (grads) rows = token_shape(p).part_rows;
    } else {
        q.part = p.scratch;
        rows = (long long)p.B * map_shape(p).splits;
        float *means = p.scratch + rows * 2 * p.C;
        if (p.backward || !q.mean_out) q.mean_out = means;
        if (p.backward || !q.rstd_out) q.rstd_out = means + (size_t)p.B * q.G;
    }
    la_status st = p.backward ? launch<true>(p, q) : launch<false>(p, q);
    if (st != LA_OK || !grads) return st;
    count_launches();
    norm_weight_grads<<<dim3((unsigned)ceil_div(p.C, 32), 2), dim3(32, 32), 0, p.stream>>>(q.part, p.dw, p.db, rows, p.C);
    return cuda_status(cudaGetLastError());
}

}  // namespace la
