// Group norm with an activation or a gate, channels last, and its gradients.
//
//   h = (x - m) r,  r = 1 / sqrt(var + eps),  z = h w + b,  y = act(z)  or  y = z act(gate)
//
// Two shapes of problem, both bound by memory: groups of one token's channels (per_token, the norm
// behind the heads of linear attention), where a few lanes hold a group in registers and every
// tensor is read once; and groups over all positions, where sums per channel come first.  Statistics
// are fp32: a token's are sums of differences from the mean; over positions each thread keeps the mean of a channel and the
// squares about it, and these are joined as such, so that no value counts for more than it is worth.
#include <type_traits>

#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

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
    int heads_first, center;
    int splits, rows, zs;  // over positions: splits of an entry, positions a split, blocks across the channels
};

// VEC elements of T as they lie in memory (loaded ahead of their use), as floats, and back.
template <typename T, int VEC> struct Pack {
    typedef T Raw;
    static __device__ __forceinline__ Raw none() { return Elem<T>::from_f32(0.f); }
    static __device__ __forceinline__ Raw load(const T *p) { return __ldcs(p); }
    static __device__ __forceinline__ Raw keep(const T *p) { return __ldg(p); }
    static __device__ __forceinline__ void open(Raw r, float (&v)[VEC])
    {
        static_assert(VEC == 1, "");
        v[0] = Elem<T>::to_f32(r);
    }
    static __device__ __forceinline__ float at(Raw r, int) { return Elem<T>::to_f32(r); }
    static __device__ __forceinline__ void put(T *p, const float (&v)[VEC]) { __stcs(p, Elem<T>::from_f32(v[0])); }
};
template <> struct Pack<float, 4> {
    typedef float4 Raw;
    static __device__ __forceinline__ Raw none() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ Raw load(const float *p) { return __ldcs(reinterpret_cast<const float4 *>(p)); }
    static __device__ __forceinline__ Raw keep(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
    static __device__ __forceinline__ void open(const Raw &a, float (&v)[4]) { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w; }
    static __device__ __forceinline__ float at(const Raw &a, int e) { return e == 0 ? a.x : e == 1 ? a.y : e == 2 ? a.z : a.w; }
    static __device__ __forceinline__ void put(float *p, const float (&v)[4])
    {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <> struct Pack<__nv_bfloat16, 8> {
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw none() { return make_uint4(0u, 0u, 0u, 0u); }
    static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
    static __device__ __forceinline__ Raw keep(const __nv_bfloat16 *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }
    static __device__ __forceinline__ void open(const Raw &a, float (&v)[8])
    {
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ float at(const Raw &a, int e)
    {
        const uint32_t u = e < 2 ? a.x : e < 4 ? a.y : e < 6 ? a.z : a.w;
        return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(u[0], u[1], u[2], u[3]));
    }
};

// silu and its slope (kAct; otherwise the identity).  bf16 results take the hardware's exponential and reciprocal
// (within 2^-21 together; a sigmoid that underflows is 0).
template <typename T> __device__ __forceinline__ float sigmoid(float z)
{
    if (std::is_same<T, float>::value) return 1.f / (1.f + expf(-z));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <typename T, bool kAct> __device__ __forceinline__ float act_of(float z) { return kAct ? z * sigmoid<T>(z) : z; }
template <typename T, bool kAct> __device__ __forceinline__ float act_slope(float z, float *value)
{
    if (!kAct) {
        *value = z;
        return 1.f;
    }
    const float s = sigmoid<T>(z);
    *value = z * s;
    return s * fmaf(z, 1.f - s, 1.f);
}

// What one element passes back: dz = dL/dz, and dL/dgate.
template <typename T, bool kGate, bool kAct>
__device__ __forceinline__ float back(float h, float w, float b, float dy, float gate, float *dgate)
{
    const float z = fmaf(h, w, b);
    float value;
    if (!kGate) return dy * act_slope<T, kAct>(z, &value);
    const float slope = act_slope<T, kAct>(gate, &value);
    *dgate = dy * z * slope;
    return dy * value;
}

// 1 / n of a count, within 2^-23 (it weighs corrections that are themselves of that accuracy).
__device__ __forceinline__ float inverse(float n)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(n));
    return r;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
#pragma unroll
    for (int d = 1; d < 32; d *= 2)
        if (d < lanes) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// ---------------------------------------------------------------- a token's groups
// `lanes` lanes hold a group, VEC neighbouring channels at a time, NV times.  A slot of lanes keeps
// to one group of channels (slot % G), so weights, and the sums for their gradients, stay in
// registers, and walks over the tokens; the launch has a whole number of slots for each group.  The loads of the
// next tokens are under way meanwhile: each thread copies its vectors asynchronously into a ring of its own in
// shared memory, kRing tokens deep (held in registers, one token ahead, they were too few to keep HBM busy: 47 us
// against 41 for 16384 tokens of 16 x 128 gated channels in bf16, 37 with today's grid: 5.4 TB/s; backward 64 us, 5.2
// TB/s); channels by ones are loaded one token ahead.  What bounds them then is instructions: an issue slot is used in 3 of 4
// cycles, by the exponentials, conversions and the sums over lanes.
constexpr int kRing = 4;
__device__ __forceinline__ void copy_async(void *dst, const void *src, bool on)  // 16 bytes, or zeros
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async4(void *dst, const void *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}
template <int NV, bool kGate, bool kBack> struct RingStage {
    uint4 x[NV][256], gate[kGate ? NV : 1][kGate ? 256 : 1], dy[kBack ? NV : 1][kBack ? 256 : 1];
    float mean[kBack ? 256 : 4], rstd[kBack ? 256 : 4];
};
template <typename T, int VEC, int NV, bool kGate, bool kBack, bool kAct>
__global__ void __launch_bounds__(256, VEC * NV > 8 ? 1 : kBack || VEC * NV > 4 ? 2 : 3) norm_tokens(Params p, int lanes, long long slots)
{
    typedef Pack<T, VEC> Pk;
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int lane = threadIdx.x & (lanes - 1), per_block = 256 / lanes, local = threadIdx.x / lanes;
    const long long slot = (long long)blockIdx.x * per_block + local;
    const int tokens = p.B * p.L, g = (int)(slot % p.G);
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
    // every lane of a warp runs the same trips (the sums take all lanes): a slot past the last token reads and
    // writes nothing.  Token t is position l of entry bi.
    const int step = (int)(slots / p.G), step_b = step / p.L, step_l = step % p.L;
    int t = (int)(slot / p.G), wt = (int)(((long long)blockIdx.x * per_block + (threadIdx.x & ~31) / lanes) / p.G);
    int l = t % p.L;
    // token t's group: its place among all groups, where it starts in gate and y, and in x; and what a step adds
    size_t next_st = (size_t)t * p.G + g, next_flat = next_st * p.D;
    size_t next_x = p.heads_first ? (((size_t)(t / p.L) * p.G + g) * p.L + l) * p.D : next_flat;
    const size_t st_step = (size_t)step * p.G, flat_step = st_step * p.D;
    const size_t x_step = p.heads_first ? ((size_t)step_b * p.G * p.L + step_l) * p.D : flat_step;
    const size_t x_wrap = p.heads_first ? (size_t)(p.G - 1) * p.L * p.D : 0;  // to the next entry
    typename Pk::Raw rx[NV], rg[kGate ? NV : 1], rd[kBack ? NV : 1];
    float rm = 0.f, rr = 0.f;
    extern __shared__ __align__(16) uint8_t shared[];
    RingStage<NV, kGate, kBack> *ring = reinterpret_cast<RingStage<NV, kGate, kBack> *>(shared);
    int ahead = t;  // the token whose loads come next
    auto load = [&](int stage) {
        const bool live = ahead < tokens;
        if constexpr (VEC > 1) {
            RingStage<NV, kGate, kBack> &r = ring[stage];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c = (lane + n * lanes) * VEC;
                const bool on = live && in[n];
                const size_t at = on ? next_flat + c : 0;
                copy_async(&r.x[n][threadIdx.x], static_cast<const T *>(p.x) + (on ? next_x + c : 0), on);
                if (kGate) copy_async(&r.gate[n][threadIdx.x], static_cast<const T *>(p.gate) + at, on);
                if (kBack) copy_async(&r.dy[n][threadIdx.x], static_cast<const T *>(p.dy) + at, on);
            }
            if (kBack) {
                if (p.center) copy_async4(&r.mean[threadIdx.x], p.mean + (live ? next_st : 0), live);
                copy_async4(&r.rstd[threadIdx.x], p.rstd + (live ? next_st : 0), live);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c = (lane + n * lanes) * VEC;
                const bool on = live && in[n];
                rx[n] = on ? Pk::load(static_cast<const T *>(p.x) + next_x + c) : Pk::none();
                if (kGate) rg[n] = on ? Pk::load(static_cast<const T *>(p.gate) + next_flat + c) : Pk::none();
                if (kBack) rd[n] = on ? Pk::load(static_cast<const T *>(p.dy) + next_flat + c) : Pk::none();
            }
            if (kBack && live) {
                rm = p.center ? __ldg(p.mean + next_st) : 0.f;
                rr = __ldg(p.rstd + next_st);
            }
        }
        ahead = tokens - ahead > step ? ahead + step : tokens;
        next_st += st_step, next_flat += flat_step, next_x += x_step;
        l += step_l;
        if (l >= p.L) l -= p.L, next_x += x_wrap;
    };
    size_t st = next_st, flat = next_flat, xat = next_x;  // of token t
    int l_now = l, stage = 0;
    for (int i = 0; i < (VEC > 1 ? kRing - 1 : 1); ++i) load(i);
    for (; wt < tokens; t = tokens - t > step ? t + step : tokens, wt = tokens - wt > step ? wt + step : tokens, st += st_step,
                        flat += flat_step, xat += x_step, l_now += step_l, xat += l_now >= p.L ? x_wrap : 0,
                        l_now -= l_now >= p.L ? p.L : 0) {
        const bool live = t < tokens;
        float x[NV][VEC], ga[kGate ? NV : 1][VEC], dy[kBack ? NV : 1][VEC], m_in = rm, r_in = rr;
        if constexpr (VEC > 1) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            const RingStage<NV, kGate, kBack> &r = ring[stage];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                Pk::open(*reinterpret_cast<const typename Pk::Raw *>(&r.x[n][threadIdx.x]), x[n]);
                if (kGate) Pk::open(*reinterpret_cast<const typename Pk::Raw *>(&r.gate[n][threadIdx.x]), ga[n]);
                if (kBack) Pk::open(*reinterpret_cast<const typename Pk::Raw *>(&r.dy[n][threadIdx.x]), dy[n]);
            }
            if (kBack) m_in = p.center ? r.mean[threadIdx.x] : 0.f, r_in = r.rstd[threadIdx.x];
            load((stage + kRing - 1) % kRing);
            stage = (stage + 1) % kRing;
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                Pk::open(rx[n], x[n]);
                if (kGate) Pk::open(rg[n], ga[n]);
                if (kBack) Pk::open(rd[n], dy[n]);
            }
            load(0);
        }
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
                    x[n][e] = in[n] ? x[n][e] - m : 0.f;
                    v = fmaf(x[n][e], x[n][e], v);
                }
            const float r = rsqrtf(fmaf(lanes_sum(v, lanes), inv, p.eps));
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
                    x[n][e] = kGate ? z * act_of<T, kAct>(ga[n][e]) : act_of<T, kAct>(z);
                }
                if (in[n]) Pk::put(static_cast<T *>(p.y) + flat + (lane + n * lanes) * VEC, x[n]);
            }
        } else {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (x[n][e] - m_in) * r_in;
                    float dg = 0.f;
                    const float dz = back<T, kGate, kAct>(h, w[n][e], b[n][e], dy[n][e], kGate ? ga[n][e] : 0.f, &dg);
                    if (kGate) ga[n][e] = dg;
                    // dy is 0 past the channels and the tokens, so dz is (w is 0 there too)
                    dw[n][e] = fmaf(dz, h, dw[n][e]);
                    db[n][e] += dz;
                    const float dh = dz * w[n][e];
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
                for (int e = 0; e < VEC; ++e) x[n][e] = r_in * (dy[n][e] - s1 - x[n][e] * s2);
                if (in[n]) {
                    Pk::put(static_cast<T *>(p.dx) + xat + (lane + n * lanes) * VEC, x[n]);
                    if (kGate) Pk::put(static_cast<T *>(p.dgate) + flat + (lane + n * lanes) * VEC, ga[n]);
                }
            }
        }
    }
    if (kBack && p.part) {
        // the block's sums: slots of one group are added in order, then written to the row of the partial sums that
        // the block (or, where a block holds fewer slots than there are groups, its run of slots) owns
        float *sums = reinterpret_cast<float *>(shared);  // [slots][D], over the ring
        asm volatile("cp.async.wait_group 0;" ::: "memory");
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
// f(e, group of channel c + e) for e < VEC, groups of D channels.
template <int VEC, typename F> __device__ __forceinline__ void for_groups(int c, int D, F f)
{
    int g = c / D, r = c - g * D;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        f(e, g);
        if (++r == D) r = 0, ++g;
    }
}

// Blocks that the registers let an SM hold; a launch is one round of them (16 x 1024 positions of 32 x 40 channels, backward: 60
// us with rounds and a third, and a thread a column of 160, 43 so; 16 x 4096 of 32 x 16 forward 42 -> 38, gated 58 -> 44).
constexpr int sums_per_sm(bool back) { return back ? 2 : 4; }
constexpr int apply_per_sm(bool gate, bool back) { return back ? 2 : gate ? 3 : 4; }

// The mean m of the rows so far of a thread's channels, and the sum q of the squares about it (without centring about 0).
// With the sum s of K new rows' differences from m, n rows with them: m' = m + s / n, and q' = q + (their squares) - s^2 / n.
// Differences are from the rows before, so neither a large mean nor an outlier, first or later, cancels: one shift for a whole
// group, its first value, lost 2^-24 (mean - shift)^2 of the variance.
template <typename T, int VEC> struct Moments {
    typedef Pack<T, VEC> Pk;
    float m[VEC] = {}, q[VEC] = {};
    int n = 0;
    template <int K> __device__ __forceinline__ void add(const typename Pk::Raw *r, bool center)
    {
        if (center && n == 0) Pk::open(r[0], m);
        n += K;
        const float part = inverse((float)n);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < K; ++u) {
                const float d = Pk::at(r[u], e) - m[e];
                s += d;
                q[e] = fmaf(d, d, q[e]);
            }
            if (center) {
                const float t = s * part;
                m[e] += t;
                q[e] = fmaf(-s, t, q[e]);
            }
        }
    }
};
// The moments of one channel over `ny` threads, `step` floats apart, whose means stand at `m` and squares at `q`; thread k
// has n / ny rows, one more if k < n % ny.
__device__ __forceinline__ void join_moments(const float *m, const float *q, int step, int ny, int n, float &mean, float &squares)
{
    const int base = n / ny, more = n % ny;
    const float ref = m[0];
    float s = 0.f, v = 0.f;
#pragma unroll 4
    for (int k = 0; k < ny; ++k) s = fmaf((float)(base + (k < more)), m[k * step] - ref, s);
    mean = n > 0 ? fmaf(s, inverse((float)n), ref) : 0.f;
#pragma unroll 4
    for (int k = 0; k < ny; ++k) {
        const float d = m[k * step] - mean;
        v += fmaf((float)(base + (k < more)) * d, d, q[k * step]);
    }
    squares = v;
}

// Columns of VEC channels, `cols` of them to a block of 256 threads; the other threads of a column take
// further positions.  Moments (forward) or sums (backward) per channel and split, joined in shared memory in a fixed order.
template <typename T, int VEC, bool kGate, bool kBack, bool kAct>
__global__ void __launch_bounds__(256, sums_per_sm(kBack)) norm_sums(Params p, int cols)
{
    typedef Pack<T, VEC> Pk;
    extern __shared__ float sums[];  // [2][threads of a column][cols * VEC]
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int tx = threadIdx.x % cols, ty = threadIdx.x / cols, ny = 256 / cols;
    const int z = blockIdx.x % p.zs, c = (z * cols + tx) * VEC, bi = blockIdx.x / p.zs / p.splits, split = blockIdx.x / p.zs % p.splits;
    const bool on = ty < ny && c < p.C;
    float s1[VEC] = {}, s2[VEC] = {};
    Moments<T, VEC> so_far;
    if (on) {
        const T *x = static_cast<const T *>(p.x) + (size_t)bi * p.L * p.C + c;
        const T *dy = static_cast<const T *>(p.dy) + (kBack ? (size_t)bi * p.L * p.C + c : 0);
        const T *gate = static_cast<const T *>(p.gate) + (kGate ? (size_t)bi * p.L * p.C + c : 0);
        constexpr int kAhead = kBack ? (kGate ? 2 : 3) : 4;  // rows whose loads are under way while as many are summed
        const int l1 = min(p.L, (split + 1) * p.rows);
        typename Pk::Raw rx[kAhead], rd[kBack ? kAhead : 1], rg[kGate ? kAhead : 1];
        auto load = [&](int l) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (l + u * ny >= l1) break;
                const size_t at = (size_t)(l + u * ny) * p.C;
                rx[u] = Pk::keep(x + at);
                if (kBack) rd[u] = Pk::keep(dy + at);
                if (kGate) rg[u] = Pk::keep(gate + at);
            }
        };
        int l = split * p.rows + ty;
        load(l);
        float m[VEC], r[VEC], w[VEC], b[VEC];
        if (kBack)
            for_groups<VEC>(c, p.D, [&](int e, int g) {
                const size_t st = (size_t)bi * p.G + g;
                m[e] = p.center ? __ldg(p.mean + st) : 0.f;
                r[e] = __ldg(p.rstd + st);
                w[e] = p.w ? __ldg(p.w + c + e) : 1.f;
                b[e] = p.b ? __ldg(p.b + c + e) : 0.f;
            });
        while (l < l1) {
            typename Pk::Raw cx[kAhead], cd[kBack ? kAhead : 1], cg[kGate ? kAhead : 1];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                cx[u] = rx[u];
                if (kBack) cd[u] = rd[u];
                if (kGate) cg[u] = rg[u];
            }
            const int l0 = l;
            l += kAhead * ny;
            load(l);
            if constexpr (!kBack) {
                if (l0 + (kAhead - 1) * ny < l1) {
                    so_far.template add<kAhead>(cx, p.center);
                } else {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        if (l0 + u * ny < l1) so_far.template add<1>(cx + u, p.center);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (l0 + u * ny >= l1) break;
                    float v[VEC], d[VEC], ga[VEC];
                    Pk::open(cx[u], v);
                    Pk::open(cd[u], d);
                    if (kGate) Pk::open(cg[u], ga);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float h = (v[e] - m[e]) * r[e];
                        float dg;
                        const float dz = back<T, kGate, kAct>(h, w[e], b[e], d[e], kGate ? ga[e] : 0.f, &dg);
                        s1[e] = fmaf(dz, h, s1[e]);
                        s2[e] += dz;
                    }
                }
            }
        }
    }
    const int width = cols * VEC;
    if (ty < ny)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sums[ty * width + tx * VEC + e] = kBack ? s1[e] : so_far.m[e];
            sums[(ny + ty) * width + tx * VEC + e] = kBack ? s2[e] : so_far.q[e];
        }
    __syncthreads();
    float *out = p.part + ((size_t)bi * p.splits + split) * 2 * p.C;
    if constexpr (!kBack) {
        const int n = min(p.L, (split + 1) * p.rows) - split * p.rows;
        for (int i = threadIdx.x; i < width && z * width + i < p.C; i += 256) {
            float mean, squares;
            join_moments(sums + i, sums + ny * width + i, width, ny, n, mean, squares);
            out[z * width + i] = mean;
            out[p.C + z * width + i] = squares;
        }
    } else {
        for (int i = threadIdx.x; i < 2 * width; i += 256) {
            const int which = i / width, j = i % width, ch = z * width + j;
            float v = 0.f;
            for (int k = 0; k < ny; ++k) v += sums[(which * ny + k) * width + j];
            if (ch < p.C) out[(size_t)which * p.C + ch] = v;
        }
    }
}

constexpr int kFinish = 512;  // threads of the blocks that finish sums

__device__ __forceinline__ float block_sum(float v, float *tmp)
{
    v = lanes_sum(v, 32);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = tmp[threadIdx.x & (kFinish / 32 - 1)];
    return lanes_sum(v, kFinish / 32);
}

// The two sums of a group, over its channels and the splits of its entry: of value 0 and value 1 of the
// partial sums, with the channels' weights.
__device__ __forceinline__ void group_sums(const Params &p, int bg, float *tmp, float &s0, float &s1)
{
    const int bi = bg / p.G, g = bg % p.G, n = p.D * p.splits;
    const float *part = p.part + (size_t)bi * p.splits * 2 * p.C + g * p.D;
    s0 = s1 = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kFinish) {
        const int split = i / p.D, c = i - split * p.D;
        const float *at = part + (size_t)split * 2 * p.C + c, w = p.w ? __ldg(p.w + g * p.D + c) : 1.f;
        s0 = fmaf(w, at[0], s0);
        s1 = fmaf(w, at[p.C], s1);
    }
    s0 = block_sum(s0, tmp);
    s1 = block_sum(s1, tmp);
}

// Forward: mean and rstd of each group, from the moments of its channels' splits.
__global__ void __launch_bounds__(kFinish) norm_statistics(Params p)
{
    __shared__ float tmp[kFinish / 32];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int bi = blockIdx.x / p.G, g = blockIdx.x % p.G, n = p.D * p.splits;
    const float *part = p.part + (size_t)bi * p.splits * 2 * p.C + g * p.D, inv = 1.f / p.D / p.L;
    float rows = 0.f, m = 0.f, q = 0.f;  // of the thread's share: channels' splits, four at a time
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * kFinish) {
        float r[4], mean[4], sq[4], s = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kFinish, split = i / p.D, c = i - split * p.D;
            const float *at = part + (size_t)split * 2 * p.C + c;
            r[u] = i < n ? (float)(min(p.L, (split + 1) * p.rows) - split * p.rows) : 0.f;
            mean[u] = i < n ? at[0] : 0.f;
            sq[u] = i < n ? at[p.C] : 0.f;
        }
        if (i0 == (int)threadIdx.x) m = mean[0];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float d = i0 + u * kFinish < n ? mean[u] - m : 0.f;
            s = fmaf(r[u], d, s);
            rows += r[u];
            q += fmaf(r[u] * d, d, sq[u]);
        }
        const float t = s * inverse(rows);
        q = fmaf(-s, t, q);
        m += t;
    }
    __shared__ float first;
    if (threadIdx.x == 0) first = m;
    __syncthreads();
    const float mean = fmaf(block_sum(rows * (m - first), tmp), inv, first);
    const float v = block_sum(fmaf(rows * (m - mean), m - mean, q), tmp) * inv;
    if (threadIdx.x == 0) {
        if (p.center) p.mean_out[blockIdx.x] = mean;
        p.rstd_out[blockIdx.x] = rsqrtf(v + p.eps);
    }
}

// dw or db: the sum of all rows of the partial sums, in a fixed order; 32 channels, a warp to every 16th row.
__device__ __forceinline__ void weight_grads(const float *part, float *out, long long rows, int C, int block, int which, float (*tmp)[33])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = block * 32 + lane;
    float v = 0.f;
    if (c < C)
#pragma unroll 8
        for (long long r = warp; r < rows; r += kFinish / 32) v += part[((size_t)r * 2 + which) * C + c];
    tmp[warp][lane] = v;
    __syncthreads();
    v = lanes_sum(tmp[lane & (kFinish / 32 - 1)][threadIdx.x >> 4], kFinish / 32);
    const int cy = block * 32 + (threadIdx.x >> 4);
    if ((threadIdx.x & 15) == 0 && cy < C) out[cy] = v;
}

// Backward: the two means of a group that its dx takes off, of dh = dz w (into mean_out) and of dh h (rstd_out);
// blocks past the groups find dw, those past them db.
__global__ void __launch_bounds__(kFinish) norm_group_means(Params p, float *dw, float *db)
{
    __shared__ float tmp[kFinish / 32][33];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int groups = p.B * p.G, block = (int)blockIdx.x - groups, per = (p.C + 31) / 32;
    if (block >= 0) {
        const int which = block >= per;
        if (which ? db != nullptr : dw != nullptr)
            weight_grads(p.part, which ? db : dw, (long long)p.B * p.splits, p.C, block - which * per, which, tmp);
        return;
    }
    float dhh, dh;
    group_sums(p, blockIdx.x, tmp[0], dhh, dh);
    if (threadIdx.x == 0) {
        const float inv = 1.f / p.D / p.L;
        p.mean_out[blockIdx.x] = p.center ? dh * inv : 0.f;
        p.rstd_out[blockIdx.x] = dhh * inv;
    }
}

__global__ void __launch_bounds__(kFinish) norm_weight_grads(const float *part, float *dw, float *db, long long rows, int C)
{
    __shared__ float tmp[kFinish / 32][33];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int per = (C + 31) / 32, which = (int)blockIdx.x >= per;
    float *out = which ? db : dw;
    if (out) weight_grads(part, out, rows, C, blockIdx.x - which * per, which, tmp);
}

// y, or dx and dgate, of all positions.
template <typename T, int VEC, bool kGate, bool kBack, bool kAct>
__global__ void __launch_bounds__(256, apply_per_sm(kGate, kBack)) norm_apply(Params p, int cols)
{
    typedef Pack<T, VEC> Pk;
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int tx = threadIdx.x % cols, ty = threadIdx.x / cols, ny = 256 / cols;
    const int z = blockIdx.x % p.zs, c = (z * cols + tx) * VEC, bi = blockIdx.x / p.zs / p.splits, split = blockIdx.x / p.zs % p.splits;
    if (ty >= ny || c >= p.C) return;
    constexpr int kAhead = kBack && kGate ? 1 : 2;  // rows whose loads are under way while as many are computed
    const size_t base = (size_t)bi * p.L * p.C + c;
    const int l1 = min(p.L, (split + 1) * p.rows);
    typename Pk::Raw rx[kAhead], rd[kBack ? kAhead : 1], rg[kGate ? kAhead : 1];
    auto load = [&](int l) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (l + u * ny >= l1) break;
            const size_t at = base + (size_t)(l + u * ny) * p.C;
            rx[u] = Pk::load(static_cast<const T *>(p.x) + at);
            if (kGate) rg[u] = Pk::load(static_cast<const T *>(p.gate) + at);
            if (kBack) rd[u] = Pk::load(static_cast<const T *>(p.dy) + at);
        }
    };
    int l = split * p.rows + ty;
    load(l);
    float m[VEC], r[VEC], w[VEC], b[VEC], a1[VEC], a2[VEC];
    for_groups<VEC>(c, p.D, [&](int e, int g) {
        const size_t st = (size_t)bi * p.G + g;
        m[e] = p.center ? p.mean[st] : 0.f;
        r[e] = p.rstd[st];
        w[e] = p.w ? __ldg(p.w + c + e) : 1.f;
        b[e] = p.b ? __ldg(p.b + c + e) : 0.f;
        if (kBack) a1[e] = p.mean_out[st], a2[e] = p.rstd_out[st];
    });
    while (l < l1) {
        typename Pk::Raw cx[kAhead], cd[kBack ? kAhead : 1], cg[kGate ? kAhead : 1];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            cx[u] = rx[u];
            if (kBack) cd[u] = rd[u];
            if (kGate) cg[u] = rg[u];
        }
        const int l0 = l;
        l += kAhead * ny;
        load(l);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (l0 + u * ny >= l1) break;
            const size_t at = base + (size_t)(l0 + u * ny) * p.C;
            float v[VEC], d[VEC], ga[VEC];
            Pk::open(cx[u], v);
            if (kGate) Pk::open(cg[u], ga);
            if (kBack) Pk::open(cd[u], d);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float h = (v[e] - m[e]) * r[e];
                if (kBack) {
                    float dg = 0.f;
                    const float dz = back<T, kGate, kAct>(h, w[e], b[e], d[e], kGate ? ga[e] : 0.f, &dg);
                    v[e] = r[e] * (fmaf(dz, w[e], -a1[e]) - h * a2[e]);
                    ga[e] = dg;
                } else {
                    const float z = fmaf(h, w[e], b[e]);
                    v[e] = kGate ? z * act_of<T, kAct>(ga[e]) : act_of<T, kAct>(z);
                }
            }
            Pk::put(static_cast<T *>(kBack ? p.dx : p.y) + at, v);
            if (kBack && kGate) Pk::put(static_cast<T *>(p.dgate) + at, ga);
        }
    }
}

// ---------------------------------------------------------------- groups that fit on chip
// An entry's slab of neighbouring groups (rows of 128 bytes or more where there are as many channels) is held in the shared
// memory of one cluster, its positions split over the CTAs: one launch, every tensor read once.  A thread keeps
// to a column of VEC channels, so that what it copies in (asynchronously) only it reads; the sums of a group go over threads,
// then over the CTAs of the cluster, in a fixed order.
constexpr int kFusedThreads = 256, kFusedMost = 8 /* CTAs of a cluster */, kFusedGroups = 64 /* of a slab */;
constexpr int kFusedSmem = 200 << 10, kFusedShare = 72 << 10;  // of a CTA: at most, and if the cluster can be that large (two share an SM, three up to 70 KB)
struct Slab {
    int groups, slabs, rows, cols;  // groups of a slab, slabs of an entry, positions a CTA, columns
};

template <typename T, int VEC, bool kGate, bool kBack, bool kAct>
__global__ void __launch_bounds__(kFusedThreads, kBack ? 1 : 4 /* 80 registers would leave room for three */) norm_fused(Params p, Slab q)
{
    typedef Pack<T, VEC> Pk;
    typedef typename Pk::Raw Raw;
    extern __shared__ __align__(16) uint8_t shared[];
    __shared__ float mine[2][kFusedGroups], all[kFusedMost][2][kFusedGroups], done[2][kFusedGroups];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int rank = (int)sm100::cluster_ctarank(), size = (int)sm100::cluster_size();
    const int entry = blockIdx.x / size / q.slabs, slab = blockIdx.x / size % q.slabs;
    const int g0 = slab * q.groups, groups = min(q.groups, p.G - g0), width = groups * p.D;
    const int tx = threadIdx.x % q.cols, ty = threadIdx.x / q.cols, ny = kFusedThreads / q.cols, c = tx * VEC;
    const bool on = ty < ny && c < width;
    const int l0 = rank * q.rows, rows = max(0, min(q.rows, p.L - l0));
    const size_t base = ((size_t)entry * p.L + l0) * p.C + (size_t)g0 * p.D + c;
    const T *x = static_cast<const T *>(p.x) + base, *dy = static_cast<const T *>(p.dy) + (kBack ? base : 0);
    const T *gate = static_cast<const T *>(p.gate) + (kGate ? base : 0);
    constexpr bool kKeepGate = kGate && kBack;
    Raw *sx = reinterpret_cast<Raw *>(shared), *sd = sx + (kBack ? (size_t)q.rows * q.cols : 0), *sg = sd + (kKeepGate ? (size_t)q.rows * q.cols : 0);
    float *sums = reinterpret_cast<float *>(shared + ((reinterpret_cast<uint8_t *>(sg + (size_t)q.rows * q.cols) - shared + 15) & ~15));  // [2][ny][cols * VEC]
    if (size > 1) sm100::cluster_sync_all();  // every CTA's shared memory may be written from here on
    auto copy = [&](Raw *dst, const T *src) {
        if constexpr (sizeof(Raw) == 16)
            copy_async(dst, src, true);
        else if constexpr (sizeof(Raw) == 4)
            copy_async4(dst, src, true);
        else
            *dst = __ldg(src);
    };
    constexpr int kWaits = 4;  // the first quarter of the rows is summed while the others are on their way
    const int mine_rows = on && rows > ty ? (rows - ty + ny - 1) / ny : 0, quarter = (mine_rows + kWaits - 1) / kWaits;
    for (int w = 0; w < kWaits; ++w) {
        for (int i = w * quarter; i < min(mine_rows, (w + 1) * quarter); ++i) {
            const int l = ty + i * ny, at = l * q.cols + tx;
            copy(sx + at, x + (size_t)l * p.C);
            if (kBack) copy(sd + at, dy + (size_t)l * p.C);
            if (kKeepGate) copy(sg + at, gate + (size_t)l * p.C);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float m_in[VEC], r[VEC], wv[VEC], b[VEC], s1[VEC] = {}, s2[VEC] = {};
    Moments<T, VEC> so_far;
    if (on)
        for_groups<VEC>(c, p.D, [&](int e, int g) {
            const size_t st = (size_t)entry * p.G + g0 + g;
            if (c + e >= width) {
                m_in[e] = 0.f, r[e] = 0.f, wv[e] = 0.f, b[e] = 0.f;
                return;
            }
            if (kBack) m_in[e] = p.center ? __ldg(p.mean + st) : 0.f, r[e] = __ldg(p.rstd + st);
            wv[e] = p.w ? __ldg(p.w + g0 * p.D + c + e) : 1.f;
            b[e] = p.b ? __ldg(p.b + g0 * p.D + c + e) : 0.f;
        });
    auto sum_rows = [&](int w) {
        int i = w * quarter;
        const int end = min(mine_rows, (w + 1) * quarter), at0 = ty * q.cols + tx, step = ny * q.cols;
        if constexpr (!kBack) {
            constexpr int kRows = 4;
            for (; i + kRows <= end; i += kRows) {
                Raw v[kRows];
#pragma unroll
                for (int u = 0; u < kRows; ++u) v[u] = sx[at0 + (i + u) * step];
                so_far.template add<kRows>(v, p.center);
            }
            if (i + 2 <= end) {
                const Raw v[2] = {sx[at0 + i * step], sx[at0 + (i + 1) * step]};
                so_far.template add<2>(v, p.center);
                i += 2;
            }
            if (i < end) so_far.template add<1>(sx + at0 + i * step, p.center);
        } else {
            for (; i < end; ++i) {
                const int at = at0 + i * step;
                float v[VEC], d[VEC], ga[VEC];
                Pk::open(sx[at], v);
                Pk::open(sd[at], d);
                if (kKeepGate) Pk::open(sg[at], ga);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (v[e] - m_in[e]) * r[e];
                    float dg;
                    const float dz = back<T, kGate, kAct>(h, wv[e], b[e], d[e], kGate ? ga[e] : 0.f, &dg);
                    s1[e] = fmaf(dz, h, s1[e]);
                    s2[e] += dz;
                }
            }
        }
    };
    asm volatile("cp.async.wait_group 3;" ::: "memory");
    sum_rows(0);
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    sum_rows(1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    sum_rows(2);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    sum_rows(3);
    const int wide = q.cols * VEC;
    if (ty < ny)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sums[ty * wide + c + e] = kBack ? s1[e] : so_far.m[e];
            sums[(ny + ty) * wide + c + e] = kBack ? s2[e] : so_far.q[e];
        }
    __syncthreads();
    if constexpr (!kBack) {
        for (int i = threadIdx.x; i < width; i += kFusedThreads) {  // the channels' moments, over row 0 of each
            float mean, squares;
            join_moments(sums + i, sums + ny * wide + i, wide, ny, rows, mean, squares);
            sums[i] = mean;
            sums[ny * wide + i] = squares;
        }
        __syncthreads();
        for (int g = threadIdx.x >> 5; g < groups; g += kFusedThreads / 32) {  // a warp to a group's
            const float *m = sums + g * p.D, *sq = m + ny * wide;
            float s = 0.f, v = 0.f;
            for (int k = threadIdx.x & 31; k < p.D; k += 32) s += m[k] - m[0];
            const float mean = fmaf(lanes_sum(s, 32), 1.f / p.D, m[0]);
            for (int k = threadIdx.x & 31; k < p.D; k += 32) v += fmaf((float)rows * (m[k] - mean), m[k] - mean, sq[k]);
            v = lanes_sum(v, 32);
            if ((threadIdx.x & 31) == 0) mine[0][g] = mean, mine[1][g] = v;
        }
    } else {
        for (int i = threadIdx.x; i < 2 * width; i += kFusedThreads) {  // the channels' sums, over row 0 of each
            float *at = sums + (i < width ? 0 : ny * wide - width) + i;
            float v = at[0];
            for (int k = 1; k < ny; ++k) v += at[k * wide];
            at[0] = v;
            if (p.part) p.part[((size_t)(entry * size + rank) * 2 + (i >= width)) * p.C + (size_t)g0 * p.D + (i < width ? i : i - width)] = v;
        }
        __syncthreads();
        for (int i = threadIdx.x >> 5; i < 2 * groups; i += kFusedThreads / 32) {  // a warp to a group's sum
            const int which = i >= groups, g = i - which * groups;
            float v = 0.f;
            for (int k = threadIdx.x & 31; k < p.D; k += 32) {
                const float one = sums[which * ny * wide + g * p.D + k];
                v += p.w ? one * __ldg(p.w + (size_t)(g0 + g) * p.D + k) : one;
            }
            v = lanes_sum(v, 32);
            if ((threadIdx.x & 31) == 0) mine[which][g] = v;
        }
    }
    __syncthreads();
    if (size > 1) {
        for (int i = threadIdx.x; i < size * 2 * groups; i += kFusedThreads) {  // to every CTA of the cluster
            const int to = i / (2 * groups), which = i % (2 * groups) / groups, g = i % groups;
            const uint32_t at = sm100::mapa_shared(sm100::smem_u32(&all[rank][which][g]), (uint32_t)to);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(mine[which][g]) : "memory");
        }
        sm100::cluster_sync_all();
    }
    for (int i = threadIdx.x; i < groups; i += kFusedThreads) {
        const float inv = 1.f / p.D / p.L;
        const size_t st = (size_t)entry * p.G + g0 + i;
        auto one = [&](int k, int which) { return size > 1 ? all[k][which][i] : mine[which][i]; };
        if (kBack) {  // the means of dh h and of dh
            float a0 = 0.f, a1 = 0.f;
            for (int k = 0; k < size; ++k) a0 += one(k, 0), a1 += one(k, 1);
            done[0][i] = a0 * inv;
            done[1][i] = p.center ? a1 * inv : 0.f;
        } else {
            const float inv_l = 1.f / p.L;
            auto share = [&](int k) { return (float)max(0, min(q.rows, p.L - k * q.rows)) * inv_l; };  // of the positions
            float mk[kFusedMost], d = 0.f, v = 0.f;
#pragma unroll
            for (int k = 0; k < kFusedMost; ++k) {
                mk[k] = k < size ? one(k, 0) : 0.f;
                v += k < size ? one(k, 1) * inv : 0.f;
                d = k < size ? fmaf(share(k), mk[k] - mk[0], d) : d;
            }
            const float m = mk[0] + d;
#pragma unroll
            for (int k = 0; k < kFusedMost; ++k) v = k < size ? fmaf(share(k) * (mk[k] - m), mk[k] - m, v) : v;
            const float rs = rsqrtf(v + p.eps);
            done[0][i] = m, done[1][i] = rs;
            if (rank == 0) {
                if (p.center && p.mean_out) p.mean_out[st] = m;
                if (p.rstd_out) p.rstd_out[st] = rs;
            }
        }
    }
    __syncthreads();
    if (!on) return;
    float a0[VEC], a1[VEC];
    for_groups<VEC>(c, p.D, [&](int e, int g) { a0[e] = done[0][min(g, groups - 1)], a1[e] = done[1][min(g, groups - 1)]; });
#pragma unroll 2
    for (int i = 0; i < mine_rows; ++i) {
        const int l = ty + i * ny, at = l * q.cols + tx;
        float v[VEC], d[VEC], ga[VEC];
        if (kGate && !kBack) Pk::open(Pk::load(gate + (size_t)l * p.C), ga);
        Pk::open(sx[at], v);
        if (kBack) Pk::open(sd[at], d);
        if (kKeepGate) Pk::open(sg[at], ga);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (kBack) {
                const float h = (v[e] - m_in[e]) * r[e];
                float dg = 0.f;
                const float dz = back<T, kGate, kAct>(h, wv[e], b[e], d[e], kGate ? ga[e] : 0.f, &dg);
                v[e] = r[e] * (fmaf(dz, wv[e], -a1[e]) - h * a0[e]);
                ga[e] = dg;
            } else {
                const float z = fmaf((v[e] - a0[e]) * a1[e], wv[e], b[e]);
                v[e] = kGate ? z * act_of<T, kAct>(ga[e]) : act_of<T, kAct>(z);
            }
        }
        Pk::put(static_cast<T *>(kBack ? p.dx : p.y) + base + (size_t)l * p.C, v);
        if (kKeepGate) Pk::put(static_cast<T *>(p.dgate) + base + (size_t)l * p.C, ga);
    }
}

// ---------------------------------------------------------------- launches
Params params_of(const NormProblem &p)
{
    Params q{};
    q.x = p.x, q.gate = p.gate, q.dy = p.dy, q.w = p.w, q.b = p.b, q.mean = p.mean, q.rstd = p.rstd;
    q.y = p.y, q.dx = p.dx, q.dgate = p.dgate, q.mean_out = p.mean_out, q.rstd_out = p.rstd_out;
    q.B = p.B, q.L = p.L, q.C = p.C, q.G = p.spec.groups, q.D = p.C / p.spec.groups;
    q.eps = p.spec.eps, q.heads_first = p.spec.heads_first, q.center = p.spec.center;
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
    // About one round of resident blocks, each walking over many tokens: more blocks only repeat the start (weights, first
    // loads) and, backward, add rows of partial sums (16384 tokens of 16 x 128 gated channels in bf16, forward 36 us at 3
    // blocks an SM, 37 at 6, 39 at 8; backward 65 at 2, 74 at 3 and 4; channels by ones, 30 of them, backward 62 / 51 / 52).
    const int per_sm = s.vec > 1 ? (p.backward ? 2 : 3) : (p.backward ? 3 : 6);
    const long long need = (all + per_block - 1) / per_block, most = (long long)tc::sm_count() * per_sm;
    s.blocks = (need < most ? need : most);
    s.blocks = (s.blocks + unit - 1) / unit * unit;
    s.slots = s.blocks * per_block;
    s.part_rows = per_block >= G ? s.blocks : s.slots / G;
    return s;
}

struct MapShape {
    int vec, cols, zs, splits, rows;
};
MapShape map_shape(const NormProblem &p, int per_sm)
{
    MapShape s;
    const int full = p.dtype == LA_F32 ? 4 : 8;
    s.vec = p.C % full == 0 ? full : 1;
    const int n = p.C / s.vec;
    // the fewest runs of columns that leave no more than a tenth of the threads idle (160 columns: two of 80, three threads
    // a column), or else the one that leaves fewest
    int best = 0;
    for (int zs = ceil_div(n, 256); zs <= 8 * ceil_div(n, 256) && best * 10 < 256 * 9; ++zs) {
        if (best && (long long)p.B * zs > 1 << 24) break;  // (a grid's size)
        const int cols = ceil_div(n, zs), busy = 256 / cols * n / zs;
        if (busy > best && (zs == ceil_div(n, 256) || cols >= 8)) best = busy, s.zs = zs, s.cols = cols;
    }
    const int ny = 256 / s.cols;
    const long long blocks = (long long)p.B * s.zs;
    int want = (int)(tc::sm_count() * per_sm / blocks);
    const int most = ceil_div(p.L, ny * 6);
    want = want < most ? want : most;
    if (want < 1) want = 1;
    s.rows = ceil_div(p.L, want);
    s.splits = ceil_div(p.L, s.rows);
    return s;
}

// The slab and cluster of norm_fused; size 0 where the groups do not fit, or what would be held is so large that three
// launches of many small blocks do better (device times in bf16, one launch against three: forward 2.1 M elements 8.2 / 12.0 us,
// 8.4 M 15.9 / 18.7, 10.5 M 19.9 / 20.7 and gated 28.6 / 22.2; backward 2.1 M 12.4 / 15.1, 5.2 M 22.2 / 18.6, gated 31.5 / 19.7:
// a CTA that holds its part of a group loads it, sums it and stores it one after another, with few of its kind beside it).
struct FusedShape {
    int vec, size, smem;
    Slab slab;
};
FusedShape fused_shape(const NormProblem &p)
{
    FusedShape f{};
    const int G = p.spec.groups, D = p.C / G, e = p.dtype == LA_F32 ? 4 : 2, full = 16 / e;
    const int tensors = 1 + (p.backward ? 1 + (p.gate != nullptr) : 0);
    int groups = 1;
    while (groups < G && groups < kFusedGroups && groups * D * e < 128) ++groups;
    while (groups < G && groups < kFusedGroups && groups * D % full != 0) ++groups;  // whole vectors
    const int width = groups * D;
    if ((long long)p.B * p.L * p.C * e * tensors > 16ll << 20) return f;
    f.vec = p.C % full == 0 && width % full == 0 ? full : 1;
    f.slab.groups = groups, f.slab.slabs = ceil_div(G, groups), f.slab.cols = width / f.vec;
    if (f.slab.cols > kFusedThreads) return f;
    const int ny = kFusedThreads / f.slab.cols, raw = f.vec * e, sums = 2 * ny * width * 4;
    const long long slabs = (long long)p.B * f.slab.slabs;
    for (int size = 1; size <= kFusedMost; size *= 2) {
        const int rows = ceil_div(p.L, size);
        const long long smem = (long long)rows * f.slab.cols * raw * tensors + 16 + sums;
        if (smem > (size < kFusedMost ? kFusedShare : kFusedSmem)) continue;
        // as many CTAs as there are SMs, if a CTA's rows still occupy its threads
        if (slabs * size * 2 <= tc::sm_count() && size < kFusedMost && rows >= 8 * ny) continue;
        f.size = size, f.slab.rows = rows, f.smem = (int)smem;
        return f;
    }
    return f;
}

bool by_token(const NormProblem &p) { return p.spec.per_token && p.C / p.spec.groups <= kNormTokenChannels; }

// An entry's groups of one token wider than the token kernel's registers: entries of one position.
NormProblem as_map(const NormProblem &p)
{
    NormProblem q = p;
    if (p.spec.per_token) q.B = p.B * p.L, q.L = 1;
    return q;
}

template <typename T, bool kGate, bool kBack, bool kAct> la_status launch_tokens(const NormProblem &p, Params q)
{
    const TokenShape s = token_shape(p);
    const int sums = kBack && q.part ? 256 / s.lanes * q.D * 4 : 0;  // at most 16 KB
    auto ring = [](auto nv) { return (int)(kRing * sizeof(RingStage<decltype(nv)::value, kGate, kBack>)); };
    const int copies = s.vec == 1 ? 0 : s.nv == 1 ? ring(std::integral_constant<int, 1>()) : s.nv == 2 ? ring(std::integral_constant<int, 2>()) : ring(std::integral_constant<int, 4>());
    const int smem = sums > copies ? sums : copies;
    constexpr int kFull = std::is_same<T, float>::value ? 4 : 8;
    auto go = [&](auto kernel) {
        const la_status st = smem > 48 << 10 ? ensure_smem(reinterpret_cast<const void *>(kernel), smem) : LA_OK;
        if (st != LA_OK) return st;
        count_launches();
        return tc::launch_dependent(kernel, (unsigned)s.blocks, 256, smem, p.stream, q, s.lanes, s.slots);
    };
    if (s.vec == 1) {
        if (s.nv == 1) return go(&norm_tokens<T, 1, 1, kGate, kBack, kAct>);
        if (s.nv == 4) return go(&norm_tokens<T, 1, 4, kGate, kBack, kAct>);
        return go(&norm_tokens<T, 1, 16, kGate, kBack, kAct>);
    }
    if (s.nv == 1) return go(&norm_tokens<T, kFull, 1, kGate, kBack, kAct>);
    if constexpr (kFull == 4)
        if (s.nv == 4) return go(&norm_tokens<T, kFull, 4, kGate, kBack, kAct>);
    return go(&norm_tokens<T, kFull, 2, kGate, kBack, kAct>);
}

template <typename T, int VEC, bool kGate, bool kBack, bool kAct>
la_status launch_fused(const NormProblem &p, const Params &q, const FusedShape &f)
{
    auto kernel = &norm_fused<T, VEC, kGate, kBack, kAct>;
    const la_status st = ensure_smem(reinterpret_cast<const void *>(kernel), kFusedSmem);
    if (st != LA_OK) return st;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(p.B * f.slab.slabs * f.size));
    lc.blockDim = dim3(kFusedThreads);
    lc.dynamicSmemBytes = (size_t)f.smem;
    lc.stream = p.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)f.size, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = tc::dependent_launch_allowed(p.stream) ? 2 : 1;
    count_launches();
    return cuda_status(cudaLaunchKernelEx(&lc, kernel, q, f.slab));
}

template <typename T, bool kGate, bool kBack, bool kAct> la_status launch_map(const NormProblem &p, Params q)
{
    const FusedShape f = fused_shape(p);
    if (f.size > 0) {
        constexpr int kWide = std::is_same<T, float>::value ? 4 : 8;
        return f.vec == 1 ? launch_fused<T, 1, kGate, kBack, kAct>(p, q, f) : launch_fused<T, kWide, kGate, kBack, kAct>(p, q, f);
    }
    const MapShape s = map_shape(p, sums_per_sm(kBack)), a = map_shape(p, apply_per_sm(kGate, kBack));
    constexpr int kFull = std::is_same<T, float>::value ? 4 : 8;
    q.splits = s.splits, q.rows = s.rows, q.zs = s.zs;
    const int smem = 2 * (256 / s.cols) * s.cols * s.vec * 4;
    auto sums = s.vec == 1 ? &norm_sums<T, 1, kGate && kBack, kBack, kBack && kAct> : &norm_sums<T, kFull, kGate && kBack, kBack, kBack && kAct>;
    auto apply = s.vec == 1 ? &norm_apply<T, 1, kGate, kBack, kAct> : &norm_apply<T, kFull, kGate, kBack, kAct>;
    const unsigned grid = (unsigned)(s.splits * s.zs) * p.B, groups = (unsigned)(p.B * q.G);
    count_launches(3);
    la_status st = tc::launch_dependent(sums, grid, 256, smem, p.stream, q, s.cols);
    if (st != LA_OK) return st;
    if (kBack)
        st = tc::launch_dependent(&norm_group_means, groups + (p.dw || p.db ? 2u * ceil_div(p.C, 32) : 0u), kFinish, 0, p.stream, q, p.dw, p.db);
    else
        st = tc::launch_dependent(&norm_statistics, groups, kFinish, 0, p.stream, q);
    if (st != LA_OK) return st;
    if (!kBack) q.mean = q.mean_out, q.rstd = q.rstd_out;
    q.splits = a.splits, q.rows = a.rows;
    return tc::launch_dependent(apply, (unsigned)(a.splits * a.zs) * p.B, 256, 0, p.stream, q, s.cols);
}

template <bool kBack> la_status launch(const NormProblem &p, const Params &q)
{
    auto go = [&](auto t, auto gate, auto act) {
        using T = decltype(t);
        return by_token(p) ? launch_tokens<T, decltype(gate)::value, kBack, decltype(act)::value>(p, q)
                           : launch_map<T, decltype(gate)::value, kBack, decltype(act)::value>(p, q);
    };
    auto acted = [&](auto t, auto gate) {
        return p.spec.act == LA_ACT_SILU ? go(t, gate, std::true_type()) : go(t, gate, std::false_type());
    };
    auto typed = [&](auto t) { return p.gate ? acted(t, std::true_type()) : acted(t, std::false_type()); };
    return p.dtype == LA_F32 ? typed(0.f) : typed(__nv_bfloat16());
}

}  // namespace

// Scratch: partial sums, then (groups that do not fit on chip) two values a group.
size_t norm_scratch(const NormProblem &p)
{
    const bool grads = p.backward && (p.dw || p.db);
    if (by_token(p)) return grads ? (size_t)token_shape(p).part_rows * 2 * p.C * 4 : 0;
    const NormProblem q = as_map(p);
    const FusedShape f = fused_shape(q);
    if (f.size > 0) return grads ? (size_t)q.B * f.size * 2 * p.C * 4 : 0;
    return ((size_t)q.B * map_shape(q, sums_per_sm(q.backward)).splits * 2 * p.C + 2 * (size_t)q.B * p.spec.groups) * 4;
}

la_status group_norm(const NormProblem &given)
{
    const bool tokens = by_token(given), grads = given.backward && (given.dw || given.db);
    const NormProblem p = tokens ? given : as_map(given);
    const int fused = tokens ? 0 : fused_shape(p).size;
    Params q = params_of(p);
    q.part = grads || !(tokens || fused) ? p.scratch : nullptr;
    if (!tokens && !fused) {
        float *means = p.scratch + (size_t)p.B * map_shape(p, sums_per_sm(p.backward)).splits * 2 * p.C;
        if (p.backward || !q.mean_out) q.mean_out = means;
        if (p.backward || !q.rstd_out) q.rstd_out = means + (size_t)p.B * q.G;
    }
    la_status st = p.backward ? launch<true>(p, q) : launch<false>(p, q);
    if (st != LA_OK || !grads || !(tokens || fused)) return st;
    count_launches();
    return tc::launch_dependent(&norm_weight_grads, 2u * ceil_div(p.C, 32), kFinish, 0, p.stream, (const float *)q.part, p.dw, p.db,
                                tokens ? token_shape(p).part_rows : (long long)p.B * fused, p.C);
}

}  // namespace la
