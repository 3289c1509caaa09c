// The preparing kernel and the scan of the tensor-core gated delta rule (bf16; d_k and d_v of 32 as 64): forward
// (la_tc_delta.cu), and for the backward pass forward without o and in reverse (la_tc_delta_bwd.cu).
//
// The scan is a chain, chunk by chunk.  It is laid out so that a CTA owns a (b, h) and every product has
// the value features as its 128 rows: E^T and what S^T gains appear in TMEM with one thread (of each half of the columns) to a feature,
// the state itself in those threads' registers,
// so that each step's result becomes the left operand of the next (tcgen05.ld, scale, split, tcgen05.st)
// without passing through shared memory or another thread.  What the state feeds is held to fp32's
// neighbourhood: T, W, S and U are multiplied as two bf16 parts (within 2^-17; the product of two low parts is
// left out), K, Q, V and dO are exact.  So is what ends in o, whose two terms, the state's answer and that of the chunk's own
// writes, nearly cancel where a key is overwritten (with E, P and S in one part there, o of near-parallel keys was off by
// 1.6%, four times its own rounding).
#pragma once

#include "la_tc_delta.cuh"

namespace la {

static __device__ unsigned g_delta_status = 0;  // one for each translation unit
static std::atomic<bool> g_launched{false};

namespace delta {
namespace {

// ---------------------------------------------------------------- preparing kernel
// A CTA a (b, h, chunk): [Q; K] K^T in one product of 128 rows (TMEM lanes 0-63: Q K^T, 64-127: K K^T); N in
// shared memory, inverted in place by blocks; T back as an operand for W.  Four warps, or eight (kBack): the
// second four invert diag(beta) N, and what follows is shared out.
constexpr int kRowStride = kChunk + 4;
typedef float Square[kChunk][kRowStride];

template <int DK, bool kBack> struct PrepSmem {
    union alignas(1024) {
        uint8_t qk[DK / 64][2 * kSq];             // per 64 columns: 64 rows of Q, 64 of K
        uint8_t w[2][DK / 64][kSq];               // then W (or W2)
    };
    uint8_t extra[DK == 64 ? kSq : 1024];         // where Q leaves room for one part of T alone
    uint8_t p[kBack ? 2 : 1][kBack ? 2 * kSq : 1024];  // P, as 128 rows of which the second half is not used
    Square a[kBack ? 2 : 1];
    Scalars s;
    long long G[kChunk];
    uint64_t full, done;
    uint32_t tmem_base;
    int abort;
};

// (I + A)^-1 in place, A strictly lower triangular: 16-wide diagonal blocks by substitution (a thread a column),
// then the blocks below them, T10 = -T11 (A10 T00), for 16 and for 32.  128 threads t, barrier `bar`.
__device__ __forceinline__ void invert(Square &a, int t, int bar)
{
    {
        const int b = (t >> 4) & 3, c = t & 15;
        float x[16];
        if (t < 64) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s[4] = {i == c ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 r = *reinterpret_cast<const float4 *>(&a[16 * b + i][16 * b + j]);
                    s[0] = fmaf(-r.x, x[j], s[0]);
                    if (j + 1 < i) s[1] = fmaf(-r.y, x[j + 1], s[1]);
                    if (j + 2 < i) s[2] = fmaf(-r.z, x[j + 2], s[2]);
                    if (j + 3 < i) s[3] = fmaf(-r.w, x[j + 3], s[3]);
                }
                x[i] = (s[0] + s[1]) + (s[2] + s[3]);
            }
        }
        named_bar_sync(bar, 128);
        if (t < 64)
#pragma unroll
            for (int i = 0; i < 16; ++i) a[16 * b + i][16 * b + c] = x[i];
        named_bar_sync(bar, 128);
    }
    {
        const int o = 32 * (t >> 6), r = (t & 63) >> 2, c = 4 * (t & 3);
#pragma unroll
        for (int step = 0; step < 2; ++step) {  // A10 T00, then -T11 of that
            const float *l = step ? &a[o + 16 + r][o + 16] : &a[o + 16 + r][o];
            const int k0 = step ? o + 16 : o;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float w = l[k];
                const float4 z = *reinterpret_cast<const float4 *>(&a[k0 + k][o + c]);
                y.x = fmaf(w, z.x, y.x), y.y = fmaf(w, z.y, y.y), y.z = fmaf(w, z.z, y.z), y.w = fmaf(w, z.w, y.w);
            }
            if (step) y = make_float4(-y.x, -y.y, -y.z, -y.w);
            named_bar_sync(bar, 128);
            *reinterpret_cast<float4 *>(&a[o + 16 + r][o + c]) = y;
            named_bar_sync(bar, 128);
        }
    }
    {   // a warp takes 8 columns of A10 T00, whose rows k before them are 0, then 8 rows of T11, 0 behind them
        const int w = t >> 5, l = t & 31;
        auto product = [&](int r, int c, int k0, int from, int to, float4 (&y)[2]) {
            y[0] = y[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k = from; k < to; k += 4) {
                float4 z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = *reinterpret_cast<const float4 *>(&a[k0 + k + e][c]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 q = *reinterpret_cast<const float4 *>(&a[32 + r + u][k0 + k]);
                    const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[u].x = fmaf(f[e], z[e].x, y[u].x), y[u].y = fmaf(f[e], z[e].y, y[u].y);
                        y[u].z = fmaf(f[e], z[e].z, y[u].z), y[u].w = fmaf(f[e], z[e].w, y[u].w);
                    }
                }
            }
        };
        float4 y[2];
        int r = 2 * (l >> 1), c = 8 * w + 4 * (l & 1);
        product(r, c, 0, 8 * w, 32, y);
        named_bar_sync(bar, 128);
        *reinterpret_cast<float4 *>(&a[32 + r][c]) = y[0];
        *reinterpret_cast<float4 *>(&a[33 + r][c]) = y[1];
        named_bar_sync(bar, 128);
        r = 8 * w + 2 * (l >> 3), c = 4 * (l & 7);
        product(r, c, 32, 0, 8 * w + 8, y);
        named_bar_sync(bar, 128);
        *reinterpret_cast<float4 *>(&a[32 + r][c]) = make_float4(-y[0].x, -y[0].y, -y[0].z, -y[0].w);
        *reinterpret_cast<float4 *>(&a[33 + r][c]) = make_float4(-y[1].x, -y[1].y, -y[1].z, -y[1].w);
        named_bar_sync(bar, 128);
    }
}

// Eight values to both parts of a swizzled row: 16 bytes each.
__device__ __forceinline__ void split8(const float (&x)[8], uint4 &hi, uint4 &lo)
{
    split2(x[0], x[1], hi.x, lo.x);
    split2(x[2], x[3], hi.y, lo.y);
    split2(x[4], x[5], hi.z, lo.z);
    split2(x[6], x[7], hi.w, lo.w);
}

// Columns x0 .. x1 of a row (token i: its TMEM lane) to both parts of an image [token][d_k] in shared memory.
template <int DK> __device__ __forceinline__ void put_row(uint32_t taddr, uint8_t (*w)[DK / 64][kSq], int i, int x0, int x1)
{
#pragma unroll 1
    for (int x = x0; x < x1; x += 32) {
        uint32_t a[32];
        tmem_ld32(taddr + x, a);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = __uint_as_float(a[e + u]);
            uint4 hi, lo;
            split8(v, hi, lo);
            const uint32_t at = sw128_offset(i, (x + e) & 63);
            *reinterpret_cast<uint4 *>(w[0][x >> 6] + at) = hi;
            *reinterpret_cast<uint4 *>(w[1][x >> 6] + at) = lo;
        }
    }
}

// (g, beta) of the chunk's token tid; tokens past the sequence leave the state as it is.
__device__ __forceinline__ float2 load_gates(const Params &p, int bh, int chunk, int tid)
{
    const int t = chunk * kChunk + tid;
    if (tid >= kChunk || t >= p.N) return make_float2(0.f, 0.f);
    const size_t at = (size_t)bh * p.N + t;
    return make_float2(__ldg(p.g + at), __ldg(p.beta + at));
}

// One chunk by kBack ? 256 : 128 threads `tid`, whose barrier is sync(); barriers of sm initialised, `ok` unless it aborted.
// `gates`: load_gates of the thread.  `turn`: how many chunks the threads have prepared before (the parity of sm.full).  `bar`: a barrier for 128 of them
// (kBack: and the next one, for the others).  `stay` leaves the last store to the caller, committed by an elected
// thread of warp 0, and the other stores visible to the device.
template <int DK, bool kBack, typename Sync>
__device__ __forceinline__ void prepare_chunk(PrepSmem<DK, kBack> &sm, const CUtensorMap &map_q, const CUtensorMap &map_k, const Params &p,
                                              uint8_t *image, float2 gates, int bh, int chunk, int tid, int warp, uint32_t tmem, uint32_t turn,
                                              bool sound, int bar, bool stay, Sync sync)
{
    typedef Layout<DK> Lay;
    constexpr int kNT = kBack ? 256 : 128;
    const int lane = tid & 31, t0 = chunk * kChunk, bhk = bh / p.H * p.Hk + bh % p.H / (p.H / p.Hk);
    if (warp == 0 && sound && elect_one()) {
        mbar_arrive_expect_tx(&sm.full, DK / 64 * 2 * kSq);
        for (int x = 0; x < DK / 64; ++x) {
            tma_load_3d(sm.qk[x], &map_q, &sm.full, 64 * x, t0, bhk);
            tma_load_3d(sm.qk[x] + kSq, &map_k, &sm.full, 64 * x, t0, bhk);
        }
    }
    __syncwarp();
    // The running sum of the gates, in units of 2^-40 as 64-bit integers (doubles cost a thousand cycles here, and floats
    // would lose what differences of large sums need).  A gate below -200 closes as well as -inf.
    long long G = 0;
    if (tid < 64) {
        G = __float2ll_rn(fminf(fmaxf(gates.x, -200.f), 65536.f) * 0x1p40f);
        if (gates.x != gates.x) gates.y = gates.x;  // a NaN gate makes what the token writes NaN
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long x = __shfl_up_sync(0xffffffffu, G, d);
            if (lane >= d) G += x;
        }
        sm.G[tid] = G;
    }
    sync();
    if (tid < 64) {
        const long long half = sm.G[31], end = sm.G[63] + half;
        if (tid >= 32) G += half;
        // as two floats, times log2(e) (its head and tail)
        auto scaled = [](long long v, float &lo) {
            const float h = __ll2float_rn(v) * 0x1p-40f, l = __ll2float_rn(v - __float2ll_rn(h * 0x1p40f)) * 0x1p-40f;
            constexpr double kLog2e = 1.4426950408889634074;
            constexpr float head = (float)kLog2e, tail = (float)(kLog2e - (double)head);
            const float hi = h * head;
            lo = fmaf(h, head, -hi) + fmaf(h, tail, l * head);
            return hi;
        };
        float lo, lo_end;
        const float hi = scaled(G, lo), rest = scaled(end - G, lo_end);
        const float first = exp2f(hi) * exp2f(lo), last = exp2f(rest) * exp2f(lo_end);
        constexpr float kLeast = -kClosed * 1.4426950408889634f;  // (kClosed in powers of two)
        const bool closed = rest < kLeast;
        const float open = closed ? exp2f(-kLeast) : exp2f(-rest) * exp2f(-lo_end);
        Scalars &s = sm.s;
        s.hi[tid] = hi;
        s.lo[tid] = lo;
        s.first[tid] = first;
        s.last[tid] = last;
        s.beta[tid] = gates.y;
        s.back[tid] = -gates.y * first;
        s.write[tid] = gates.y * (!kBack && closed ? exp2f(kLeast) : last);
        s.open[tid] = open;
    }
    uint8_t *tp[2] = {sm.qk[0], DK == 64 ? sm.extra : sm.qk[DK / 64 - 1]};  // over Q, once its product is done: P', then T's parts
    bool ok = sound;
    if (warp == 0) {
        ok = ok && wait_bar_warp(&g_delta_status, &sm.abort, &sm.full, turn & 1u);
        if (ok) {
            tc_fence_after();
            if (elect_one()) {
                constexpr uint32_t id = idesc_bf16_f32(128, kChunk, false, false);
                const uint32_t a = smem_u32(sm.qk[0]);
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_ss(tmem, rows_k(a, kk, 2 * kSq), rows_k(a + kSq, kk, 2 * kSq), id, kk > 0);
                mma_commit(&sm.done);
            }
        }
        __syncwarp();
    }
    sync();
    ok = sound && wait_bar_warp(&g_delta_status, &sm.abort, &sm.done, 0);
    tc_fence_after();
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    if (ok) {
        for (int i = tid; i < (int)sizeof(Scalars) / 16; i += kNT) reinterpret_cast<uint4 *>(image)[i] = reinterpret_cast<uint4 *>(&sm.s)[i];
        const int row = 32 * (warp & 3) + lane, i = row & 63;
        const uint64_t hi = pair(sm.s.hi[i], sm.s.hi[i]), lo = pair(sm.s.lo[i], sm.s.lo[i]);
        const float bi = sm.s.beta[i];
#pragma unroll 1
        for (int j0 = kBack ? 32 * (warp >> 2) : 0; j0 < kChunk; j0 += kBack ? kChunk : 32) {
            float d[32];
            if (j0 > 0 && (warp & 1) == 0) {  // above the diagonal
#pragma unroll
                for (int e = 0; e < 32; ++e) d[e] = 0.f;
            } else {
                uint32_t s[32];
                tmem_ld32(tl + j0, s);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const uint64_t w = decay2(hi, lo, *reinterpret_cast<const float2 *>(&sm.s.hi[j0 + e]), *reinterpret_cast<const float2 *>(&sm.s.lo[j0 + e]));
                    unpair(mul2(w, pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1]))), d[e], d[e + 1]);
                }
                if (j0 == 32 * (warp & 1)) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e > lane) d[e] = 0.f;
                }
            }
            if (row < 64) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float x[8] = {d[8 * c], d[8 * c + 1], d[8 * c + 2], d[8 * c + 3], d[8 * c + 4], d[8 * c + 5], d[8 * c + 6], d[8 * c + 7]};
                    uint4 h, l;
                    const uint32_t at = sw128_offset(i, j0 + 8 * c);
                    if (kBack) {
                        split8(x, h, l);
                        *reinterpret_cast<uint4 *>(sm.p[0] + at) = h;
                        *reinterpret_cast<uint4 *>(sm.p[kBack ? 1 : 0] + at) = l;
                    } else {
                        const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(sm.s.open + j0 + 8 * c);
                        split2(mul2(b[0].x, pair(x[0], x[1])), h.x, l.x);
                        split2(mul2(b[0].y, pair(x[2], x[3])), h.y, l.y);
                        split2(mul2(b[1].x, pair(x[4], x[5])), h.z, l.z);
                        split2(mul2(b[1].y, pair(x[6], x[7])), h.w, l.w);
                        *reinterpret_cast<uint4 *>(tp[0] + at) = h;
                        *reinterpret_cast<uint4 *>(tp[1] + at) = l;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const int j = j0 + e;
                    const float4 b = *reinterpret_cast<const float4 *>(&sm.s.beta[j]);
                    const float4 n = make_float4(j == i ? 0.f : d[e], j + 1 == i ? 0.f : d[e + 1], j + 2 == i ? 0.f : d[e + 2], j + 3 == i ? 0.f : d[e + 3]);
                    *reinterpret_cast<float4 *>(&sm.a[0][i][j]) = make_float4(n.x * b.x, n.y * b.y, n.z * b.z, n.w * b.w);
                    if (kBack) *reinterpret_cast<float4 *>(&sm.a[kBack ? 1 : 0][i][j]) = make_float4(bi * n.x, bi * n.y, bi * n.z, bi * n.w);
                }
            }
        }
    }
    if (!kBack) fence_proxy_async_smem();
    tc_fence_before();
    sync();
    if (!kBack && warp == 0) {  // P', while T is found
        if (ok && elect_one()) {
            bulk_store(image + Lay::p, tp[0], kSq);
            bulk_store(image + Lay::p + kSq, tp[1], kSq);
            tma_store_commit();
        }
        __syncwarp();
    }
    if (!kBack || warp < 4)
        invert(sm.a[0], tid & 127, bar);
    else
        invert(sm.a[kBack ? 1 : 0], tid & 127, bar + 1);
    if (!kBack && warp == 0) {
        if (elect_one()) tma_store_wait_read_all();
        __syncwarp();
    }
    sync();
    // T to global memory, and -T exp(G) over the rows of Q
    for (int u = tid; u < kChunk * 8; u += kNT) {
        const int i = u >> 3, c = 8 * (u & 7);
        const uint32_t at = sw128_offset(i, c);
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) *reinterpret_cast<float4 *>(&x[e]) = *reinterpret_cast<const float4 *>(&sm.a[0][i][c + e]);
        uint4 h, l;
        split8(x, h, l);
        *reinterpret_cast<uint4 *>(image + Lay::t + at) = h;
        *reinterpret_cast<uint4 *>(image + Lay::t + kSq + at) = l;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] * -sm.s.first[c + e];
        split8(y, h, l);
        *reinterpret_cast<uint4 *>(tp[0] + at) = h;
        *reinterpret_cast<uint4 *>(tp[1] + at) = l;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    sync();
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;
    // W = -T exp(G) K: rows 0-63 of 128 (the rest of the left operand is whatever follows it)
    constexpr uint32_t id_w = idesc_bf16_f32(128, DK, false, true), id_w2 = idesc_bf16_f32(128, DK, true, true);
    constexpr uint32_t tW = 0, tZ = 128, tW2 = 128;
    const uint32_t ka = smem_u32(sm.qk[0]) + kSq, th = smem_u32(tp[0]), tlo = smem_u32(tp[1]);
    if (warp == 0) {
        tc_fence_after();
        if (ok && elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(tmem + tW, rows_k(part ? tlo : th, kk), cols_mn(ka, kk, 2 * kSq), id_w, part + kk > 0);
            mma_commit(&sm.done);
        }
        __syncwarp();
    }
    ok = ok && wait_bar_warp(&g_delta_status, &sm.abort, &sm.done, 1);
    tc_fence_after();
    if (kBack) {
        // T2 over T exp(G) as an operand: Z = scale P T2; then scaled, W2 = (exp(G_C - G) T2)^T K
        constexpr uint32_t id_z = idesc_bf16_f32(128, kChunk, false, true);
        for (int pass = 0; pass < 2; ++pass) {
            if (ok)
                for (int u = tid; u < kChunk * 8; u += kNT) {
                    const int i = u >> 3, c = 8 * (u & 7);
                    const uint32_t at = sw128_offset(i, c);
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) *reinterpret_cast<float4 *>(&x[e]) = *reinterpret_cast<const float4 *>(&sm.a[kBack ? 1 : 0][i][c + e]);
                    const float f = pass ? sm.s.last[i] : 1.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= f;
                    uint4 h, l;
                    split8(x, h, l);
                    *reinterpret_cast<uint4 *>(tp[0] + at) = h;
                    *reinterpret_cast<uint4 *>(tp[1] + at) = l;
                }
            fence_proxy_async_smem();
            tc_fence_before();
            sync();
            if (warp == 0) {
                tc_fence_after();
                if (ok && elect_one()) {
                    const uint32_t ph = smem_u32(sm.p[0]), pl = smem_u32(sm.p[kBack ? 1 : 0]);
                    if (pass == 0) {
#pragma unroll
                        for (int part = 0; part < 3; ++part)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ss(tmem + tZ, rows_k(part == 1 ? pl : ph, kk), cols_mn(part == 2 ? tlo : th, kk), id_z, part + kk > 0);
                    } else {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ss(tmem + tW2, cols_mn(part ? tlo : th, kk, 0), cols_mn(ka, kk, 2 * kSq), id_w2, part + kk > 0);
                    }
                    mma_commit(&sm.done);
                }
                __syncwarp();
            }
            ok = ok && wait_bar_warp(&g_delta_status, &sm.abort, &sm.done, pass);
            tc_fence_after();
            if (pass == 0 && ok && row < 64) {
                uint32_t a[32];
                tmem_ld32(tl + tZ + 32 * half, a);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = p.scale * __uint_as_float(a[8 * c + e]);
                    uint4 h, l;
                    split8(x, h, l);
                    const uint32_t at = sw128_offset(row, 32 * half + 8 * c);
                    *reinterpret_cast<uint4 *>(sm.p[0] + at) = h;
                    *reinterpret_cast<uint4 *>(sm.p[kBack ? 1 : 0] + at) = l;
                }
            }
        }
    }
    for (int which = 0; which < (kBack ? 2 : 1); ++which) {
        if (ok && row < 64) put_row<DK>(tl + (which ? tW2 : tW), sm.w, row, half * (DK / 2), kBack ? (half + 1) * (DK / 2) : DK);
        fence_proxy_async_smem();
        tc_fence_before();
        if (stay) __threadfence();
        sync();
        if (warp == 0) {
            if (ok && elect_one()) {
                if (kBack && which == 0) {
                    bulk_store(image + Lay::z, sm.p[0], kSq);
                    bulk_store(image + Lay::z + kSq, sm.p[kBack ? 1 : 0], kSq);
                }
                bulk_store(image + (which ? Lay::w2 : Lay::w), sm.w, Lay::w_bytes);
                tma_store_commit();
                if ((kBack && which == 0) || stay)
                    tma_store_wait_read_all();
                else
                    tma_store_wait_all();
            }
            __syncwarp();
        }
        if (kBack && which == 0) sync();
    }
}

constexpr uint32_t prep_columns(int DK, bool back) { return back ? 256 : DK; }  // of TMEM: scores, then W over them; Z, then W2 over it

// The barriers and the sound state of one set of preparing threads.
template <int DK, bool kBack> __device__ __forceinline__ void prepare_start(PrepSmem<DK, kBack> &sm)
{
    mbar_init(&sm.full, 1);
    mbar_init(&sm.done, 1);
    sm.abort = (smem_u32(&sm) & 1023u) == 0 ? 0 : 1;
    if (sm.abort) atomicOr(&g_delta_status, kStatusTimeout);
}

template <int DK, bool kBack>
__global__ void __launch_bounds__(kBack ? 256 : 128)
delta_prepare(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k, const Params p, uint8_t *images)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    typedef PrepSmem<DK, kBack> Sm;
    typedef Layout<DK> Lay;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int tid = threadIdx.x, warp = uniform_warp(), chunks = (p.N + kChunk - 1) / kChunk;
    if (tid == 0) {
        prepare_start(sm);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, prep_columns(DK, kBack));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    const int bh = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    uint8_t *image = images + (size_t)blockIdx.x * (kBack ? Lay::backward_bytes : Lay::forward_bytes);
    prepare_chunk<DK, kBack>(sm, map_q, map_k, p, image, load_gates(p, bh, chunk, tid), bh, chunk, tid, warp, tmem, 0,
                             !aborted(&sm.abort), 1, false, [] { __syncthreads(); });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, prep_columns(DK, kBack));
}

// Waits (with the limit of every wait) until another CTA of the launch has published a chunk's image.
__device__ __forceinline__ bool wait_flag(const unsigned *flag, int *abort_flag, uint64_t limit_ns)
{
    const uint64_t t0 = globaltimer_ns();
    bool there;
    while (!(there = __all_sync(0xffffffffu, ld_acquire_gpu(flag) != 0))) {
        if (__any_sync(0xffffffffu, aborted(abort_flag))) return false;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) {
            *(volatile int *)abort_flag = 1;
            atomicOr(&g_delta_status, kStatusTimeout);
            return false;
        }
        __nanosleep(100);
    }
    fence_proxy_async_global();
    return there;
}

// ---------------------------------------------------------------- scan
// kForward: o and the last state.  kSave: instead of o the state before each chunk, as MMA operand images [d_v rows of
// 64 d_k columns] of its two parts, and E as images [64 tokens of 64 d_v columns].  kReverse: the same of R and dX, chunks
// in descending order, dO in the place of V.
enum Mode { kForward, kSave, kReverse };
// Warps 0-15: the chain (warp w: value features 32 (w % 4) .. + 31, quarter w / 4 of the columns: with halves, 8 warps,
// a scan of 256 chunks took 470 us against 459);
// warps 16-19: o, or E's images and dO as an operand; warp 20: products; warp 21: copies.
constexpr int kParts = 4, kChainWarps = 4 * kParts, kOutWarp = kChainWarps, kMmaWarp = kOutWarp + 4, kCopyWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kCopyWarp + 1);

constexpr uint32_t state_bytes(int DK, int DV) { return 2u * DK * DV * 2; }  // both parts of a state's image
constexpr uint32_t rows_bytes(int DV) { return 2u * kChunk * DV * 2; }       // both parts of a chunk's rows

template <int DK, int DV, int kMode> struct ScanSmem {
    // K (and in reverse Q) are needed late in a chunk: one stage where shared memory is short
    static constexpr int kKeyStages = kMode == kForward ? 2 : 1;
    static constexpr bool kOutOverW = kMode != kForward && DK >= DV;  // E's rows are staged where W was
    // o is staged where its products have room for two chunks (d 64 without a stage: 67.8 us of a call against 64); with room for
    // one, the next chunk's wait for its reading, which stores without a stage end sooner (d 128 x 64, 16381 tokens of one head:
    // 556 us with a stage, 504 without), and at d_v 128 there is none
    static constexpr bool kStageO = kMode == kForward && DK == 64;
    static constexpr uint32_t kMats = 2 * kSq + Layout<DK>::w_bytes;
    // forward, d_k 64: the products of o have room for two chunks, so that the chain does not wait for the warps of o
    static constexpr int kOuts = kMode == kForward && DK == 64 ? 2 : 1, kScalarRing = kOuts + 2;
    uint8_t v[2][DV / 64][kSq];
    uint8_t mats[2][kMats];  // T or Z, W or W2
    uint8_t k[kKeyStages][DK / 64][kSq];
    uint8_t q[kMode == kSave ? 1 : kKeyStages][kMode == kSave ? 1 : DK / 64][kSq];  // (kSave: not used)
    union {  // P is used by one mode, a state kept by the others
        uint8_t p[kMode == kForward ? 2 : 1][kMode == kForward ? 2 * kSq : 16];
        uint8_t state[kMode == kForward ? 16 : state_bytes(DK, DV)];
    };
    uint8_t rows[kStageO ? rows_bytes(DV) / 2 : kMode == kForward || kOutOverW ? 16 : rows_bytes(DV)];  // of o, or of E
    float scalars[kScalarRing][3][kChunk];  // beta, write, first; in reverse write, first, back
    uint64_t full[2];                       // a stage's V and matrices are there (and scalars, but for kForward)
    uint64_t keys_full[2], rows_read[2];    // its K, Q, P (and scalars) are; the warps of E's rows are done with it
    uint64_t s_ready, u_ready, d_ready;     // left operands are in TMEM (512, 512, 128 arrivals)
    // products are there (one barrier a stage where a waiter may come a chunk late); the warps of o have read theirs
    uint64_t e_full[2], s_full, o_full[2], o_read[2];
    uint64_t stored;                        // the state's image has been read by its store
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
// TMEM columns: what S^T gains in a chunk; S^T's bf16 parts; E^T of two chunks (forward: later U'^T's parts);
// forward: (Q S)^T and (P' U')^T; otherwise U^T's parts and dO^T's
template <int DK> struct Columns {
    static constexpr uint32_t S = 0, parts = DK, e = 2 * DK, qs = e + 128, pu = qs + 64;
};

template <int DK, int DV, int kMode>
__device__ __forceinline__ void scan_body(const CUtensorMap &map_q, const CUtensorMap &map_k, const CUtensorMap &map_v,
                                          const CUtensorMap &map_o, const Params &p, const float *first_state, float *last_state,
                                          const uint8_t *images, const unsigned *ready, uint8_t *states, uint8_t *rows, int bh,
                                          uint8_t *smem_raw)
{
    typedef ScanSmem<DK, DV, kMode> Sm;
    typedef Columns<DK> Col;
    typedef Layout<DK> Lay;
    constexpr bool kKeep = kMode != kForward;
    constexpr uint32_t kStride = kKeep ? Lay::backward_bytes : Lay::forward_bytes;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const int bhk = bh / p.H * p.Hk + bh % p.H / (p.H / p.Hk), chunks = (p.N + kChunk - 1) / kChunk;
    if (tid == 0) {
        uint64_t *one[] = {&sm.full[0], &sm.full[1], &sm.keys_full[0], &sm.keys_full[1], &sm.rows_read[0], &sm.rows_read[1],
                           &sm.e_full[0], &sm.e_full[1], &sm.s_full, &sm.o_full[0], &sm.o_full[1], &sm.stored, &sm.drain};
        for (uint64_t *b : one) mbar_init(b, 1);
        mbar_init(&sm.s_ready, 32 * kChainWarps);
        mbar_init(&sm.u_ready, 32 * kChainWarps);
        mbar_init(&sm.d_ready, 128);
        mbar_init(&sm.o_read[0], 128);
        mbar_init(&sm.o_read[1], 128);
        sm.abort = (smem_u32(smem_raw) & 1023u) == 0 ? 0 : 1;
        if (sm.abort) atomicOr(&g_delta_status, kStatusTimeout);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    int *abort_flag = &sm.abort;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_bar_warp(&g_delta_status, abort_flag, bar, parity); };
    auto chunk_of = [&](int c) { return kMode == kReverse ? chunks - 1 - c : c; };
    bool ok = !aborted(abort_flag);

    if (warp == kCopyWarp) {
        fence_proxy_async_global();  // the images were written by plain stores
        constexpr uint32_t kKeyBytes = (kMode == kSave ? 1 : 2) * (DK / 64) * kSq + (kKeep ? 0 : 2 * kSq + kScanScalars);
        int c = 0;
        for (; ok && c < chunks; ++c) {
            const int st = c & 1, x = chunk_of(c);
            const uint8_t *img = images + ((size_t)bh * chunks + x) * kStride;
            // V and the matrices of chunk c - 2 end with its E; where states are kept, the warps of E's rows tell when they have
            // read them, too, and (rows staged over W) when the rows' store has
            if (c >= 2 && !(ok = wait(kKeep ? &sm.rows_read[st] : &sm.e_full[st], (uint32_t)((c >> 1) - 1) & 1u))) break;
            if (ready && !(ok = wait_flag(ready + (size_t)bh * chunks + x, abort_flag, p.wait_ns))) break;
            if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.full[st], DV / 64 * kSq + Sm::kMats + (kKeep ? kScanScalars : 0));
                if (kKeep) bulk_load(sm.scalars[c % Sm::kScalarRing], img + (kMode == kReverse ? kChunk * 4 : 0), kScanScalars, &sm.full[st]);
                bulk_load(sm.mats[st], img + (kMode == kReverse ? Lay::z : Lay::t), Sm::kMats, &sm.full[st]);
                for (int b = 0; b < DV / 64; ++b) tma_load_3d(sm.v[st][b], &map_v, &sm.full[st], 64 * b, x * kChunk, bh);
            }
            __syncwarp();
            // K, Q and P end with the chunk's last product
            const int ks = kKeep ? 0 : st, back = kKeep ? 1 : 2;
            if (c >= back && !(ok = wait(kKeep ? &sm.s_full : &sm.o_full[st], (uint32_t)(kKeep ? c - 1 : (c >> 1) - 1) & 1u))) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.keys_full[ks], kKeyBytes);
                for (int b = 0; b < DK / 64; ++b) {
                    if (kMode != kSave) tma_load_3d(sm.q[ks][b], &map_q, &sm.keys_full[ks], 64 * b, x * kChunk, bhk);
                    tma_load_3d(sm.k[ks][b], &map_k, &sm.keys_full[ks], 64 * b, x * kChunk, bhk);
                }
                if (!kKeep) bulk_load(sm.p[st], img + Lay::p, 2 * kSq, &sm.keys_full[ks]);
                if (!kKeep) bulk_load(sm.scalars[c % Sm::kScalarRing], img, kScanScalars, &sm.keys_full[ks]);
            }
            __syncwarp();
        }
        if (c < chunks && c > 0) let_copies_land();
    } else if (warp == kMmaWarp) {
        // The loop's control and operands stay in uniform registers (an MMA issued from elsewhere costs more to issue
        // than to run): waits return nothing here, and an abort is seen at the head of the next chunk.
        constexpr uint32_t id = idesc_bf16_f32(128, kChunk, false, false), id_s = idesc_bf16_f32(128, DK, false, true);
        constexpr uint32_t kBox = kSq >> 4;  // descriptors count 16 bytes
        const uint64_t dv = cols_mn(smem_u32(sm.v[0][0]), 0, DV == 128 ? kSq : 0);
        const uint64_t dt = kMode == kReverse ? cols_mn(smem_u32(sm.mats[0]), 0) : rows_k(smem_u32(sm.mats[0]), 0);
        const uint64_t dw = rows_k(smem_u32(sm.mats[0]) + 2 * kSq, 0), dp = rows_k(smem_u32(sm.p[0]), 0);
        const uint64_t dk = cols_mn(smem_u32(sm.k[0][0]), 0), dq = rows_k(smem_u32(sm.q[0][0]), 0), dqm = cols_mn(smem_u32(sm.q[0][0]), 0);
        auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(&g_delta_status, abort_flag, bar, parity); };
        // E^T = V^T T^T (in reverse dO^T Z), ahead of the state's part.  T and Z are lower triangular: step kk of 16
        // tokens reaches the columns from 16 kk on (in reverse those up to 16 kk + 15, so the last step comes first).
        auto from_values = [&](int c) {
            const uint32_t st = (uint32_t)c & 1u;
            wait(&sm.full[st], (uint32_t)(c >> 1) & 1u);
            tc_fence_after();
            if (elect_one()) {
                const uint64_t a = dv + st * (DV / 64 * kBox), b = dt + st * (Sm::kMats >> 4);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int kk = kMode == kReverse ? 3 - u : u;
                        if (kMode == kReverse)
                            mma_ss(tmem + Col::e + 64 * st, a + kk * (2048 >> 4), b + part * kBox + kk * (2048 >> 4),
                                   idesc_bf16_f32(128, 16 * (kk + 1), true, true), part + u > 0);
                        else
                            mma_ss(tmem + Col::e + 64 * st + 16 * kk, a + kk * (2048 >> 4), b + part * kBox + kk * 2 + kk * (2048 >> 4),
                                   idesc_bf16_f32(128, kChunk - 16 * kk, true, false), part + u > 0);
                    }
            }
            __syncwarp();
        };
        if (chunks > 0 && !__any_sync(0xffffffffu, aborted(abort_flag))) from_values(0);
        for (int c = 0; c < chunks; ++c) {
            if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
            const uint32_t st = (uint32_t)c & 1u, ph = st;
            const uint32_t tE = tmem + Col::e + 64 * st, tU = kKeep ? tmem + Col::qs : tE;
            wait(&sm.s_ready, ph);
            tc_fence_after();
            if (elect_one()) {  // E^T += S^T W^T: high high, low high, high low
                const uint64_t b = dw + st * (Sm::kMats >> 4);
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_ts(tE, tmem + Col::parts + (part == 1) * (DK / 2) + kk * 8,
                               b + (part == 2) * (DK / 64) * kBox + (kk >> 2) * kBox + (kk & 3) * 2, id, 1);
                mma_commit(&sm.e_full[st]);
            }
            __syncwarp();
            // what the warps of o (or of E's rows) read of the chunk before, or of the one before that
            if (c >= Sm::kOuts) wait(&sm.o_read[(c - Sm::kOuts) & 1], (uint32_t)((c - Sm::kOuts) >> 1) & 1u);
            const uint32_t tQ = tmem + Col::qs + (Sm::kOuts == 2 ? 128 * st : 0);
            if (kKeep)
                wait(&sm.keys_full[0], ph);
            else
                wait(&sm.keys_full[st], (uint32_t)(c >> 1) & 1u);
            if (!kKeep) {
                tc_fence_after();
                if (elect_one()) {  // (Q S)^T, both parts
                    const uint64_t b = dq + st * (DK / 64 * kBox);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < DK / 16; ++kk)
                            mma_ts(tQ, tmem + Col::parts + part * (DK / 2) + kk * 8, b + (kk >> 2) * kBox + (kk & 3) * 2, id, part + kk > 0);
                }
                __syncwarp();
            }
            if (kMode == kReverse) wait(&sm.d_ready, ph);
            wait(&sm.u_ready, ph);
            tc_fence_after();
            if (elect_one()) {  // what the state gains, U^T K (in reverse also dO^T Q), both parts; (P' U')^T
                const uint64_t b = dk + (kKeep ? 0 : st * (DK / 64 * kBox));
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_ts(tmem + Col::S, tU + kk * 16 + part * 8, b + kk * (2048 >> 4), id_s, part + kk > 0);
                        if (kMode == kReverse)
                            mma_ts(tmem + Col::S, tmem + Col::pu + part * 32 + kk * 8, dqm + kk * (2048 >> 4), id_s, 1);
                    }
                mma_commit(&sm.s_full);
                if (!kKeep) {
                    // high high, low high, high low (P' lower triangular); the low parts take 3 of 68 us (32 heads of 2048, d 64),
                    // and behind the next errors' product, where the chain leaves the tensor cores idle, 5
                    const uint64_t bp = dp + st * (2 * kBox);
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts(tQ + 64 + 16 * kk, tU + kk * 16 + (part == 1) * 8, bp + (part == 2) * kBox + kk * 2 + kk * (2048 >> 4),
                                   idesc_bf16_f32(128, kChunk - 16 * kk, false, false), part + kk > 0);
                    mma_commit(&sm.o_full[st]);
                }
            }
            __syncwarp();
            // (the next E^T goes over operands that P' U' of the chunk before has read)
            if (!kKeep && c > 0) wait(&sm.o_full[st ^ 1], (uint32_t)((c - 1) >> 1) & 1u);
            if (c + 1 < chunks) from_values(c + 1);
        }
        if (elect_one()) {
            mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
            drain(&sm.drain, 0);
        }
        __syncwarp();
    } else if (warp < kChainWarps) {
        constexpr int kKeys = DK / kParts, kTokens = kChunk / kParts;  // columns of S, of E, a thread
        const int part = warp >> 2, f = 32 * (warp & 3) + lane;        // value feature
        const bool live = 32 * (warp & 3) < DV;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tS = tl + Col::S + part * kKeys, tP = tl + Col::parts + part * (kKeys / 2);
        // (widths of 32 fill half of the tiles: their copies read zeros past the rows' ends)
        const bool mine = f < p.dv;
        const size_t state = (size_t)bh * p.dk * p.dv + (size_t)part * kKeys * p.dv + f;
        float s[kKeys];  // the state: key features part kKeys ..
#pragma unroll
        for (int e = 0; e < kKeys; ++e)
            s[e] = first_state && mine && part * kKeys + e < p.dk ? first_state[state + (size_t)e * p.dv] : 0.f;
        for (int c = 0; ok && c < chunks; ++c) {
            const int st = c & 1;
            const uint32_t ph = (uint32_t)c & 1u;
            if (kKeep && c > 0 && !(ok = wait(&sm.stored, ph ^ 1u))) break;
#pragma unroll
            for (int x = 0; x < kKeys; x += 16) {  // two parts: to TMEM and to the image that is kept
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) split2(s[x + 2 * e], s[x + 2 * e + 1], hi[e], lo[e]);
                tmem_st8(tP + x / 2, hi);
                tmem_st8(tP + DK / 2 + x / 2, lo);
                if (kKeep && live) {
                    const int k0 = part * kKeys + x;
                    uint8_t *at = sm.state + (k0 >> 6) * (DV * 128);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t off = sw128_offset(f, (k0 & 63) + 8 * e);
                        *reinterpret_cast<uint4 *>(at + off) = make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
                        *reinterpret_cast<uint4 *>(at + state_bytes(DK, DV) / 2 + off) = make_uint4(lo[4 * e], lo[4 * e + 1], lo[4 * e + 2], lo[4 * e + 3]);
                    }
                }
            }
            if (kKeep) fence_proxy_async_smem();
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.s_ready);
            if (!(ok = wait(kKeep ? &sm.full[st] : &sm.keys_full[st], (uint32_t)(c >> 1) & 1u))) break;
            const float (*scalars)[kChunk] = sm.scalars[c % Sm::kScalarRing];
            const float whole = scalars[kMode == kReverse ? 1 : 2][kChunk - 1];
            if (!(ok = wait(&sm.e_full[st], (uint32_t)(c >> 1) & 1u))) break;
            tc_fence_after();
            const uint32_t tE = tl + Col::e + 64 * st + kTokens * part;
            uint32_t a[16];
            static_assert(kTokens == 16, "");
            tmem_ld16(tE, a);
            tmem_ld_wait();
            {
                const float *mul = scalars[kMode == kReverse ? 2 : 1] + kTokens * part;
                const uint32_t tU = kKeep ? tl + Col::qs + kTokens * part : tE;
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(mul + e);
                    split2(mul2(pair(w.x, w.y), pair(__uint_as_float(a[e]), __uint_as_float(a[e + 1]))), hi[e / 2], lo[e / 2]);
                    split2(mul2(pair(w.z, w.w), pair(__uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]))), hi[e / 2 + 1], lo[e / 2 + 1]);
                }
                tmem_st8(tU, hi);
                tmem_st8(tU + 8, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.u_ready);
            if (!(ok = wait(&sm.s_full, ph))) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < kKeys; x += 16) {
                tmem_ld16(tS + x, a);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    unpair(fma2(pair(whole, whole), pair(s[x + e], s[x + e + 1]), pair(__uint_as_float(a[e]), __uint_as_float(a[e + 1]))),
                           s[x + e], s[x + e + 1]);
            }
        }
        if (ok && last_state && mine)
#pragma unroll
            for (int e = 0; e < kKeys; ++e)
                if (part * kKeys + e < p.dk) last_state[state + (size_t)e * p.dv] = s[e];
    } else if (warp < kMmaWarp) {
        const int f = 32 * (warp & 3) + lane;
        const bool live = 32 * (warp & 3) < DV;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        uint32_t at[8];  // (row e, feature f) of a tile of 64-column boxes
#pragma unroll
        for (int e = 0; e < 8; ++e) at[e] = ((f & 127) >> 6) * kSq + sw128_offset(e, f & 63);
        for (int c = 0; ok && c < chunks; ++c) {
            const int st = c & 1, x = chunk_of(c);
            const uint32_t ph = (uint32_t)c & 1u;
            uint8_t *out = Sm::kOutOverW ? sm.mats[st] + 2 * kSq : sm.rows;
            if (kMode == kReverse) {  // scale exp(G) dO as a left operand, once the last state product has read it
                if (!(ok = wait(&sm.full[st], (uint32_t)(c >> 1) & 1u))) break;
                if (c > 0 && !(ok = wait(&sm.s_full, ph ^ 1u))) break;
                tc_fence_after();
                const uint8_t *v = sm.v[st][0];
#pragma unroll
                for (int y = 0; y < kChunk; y += 16) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const uint8_t *r = v + (y + e) / 8 * 1024;
                        const float d0 = live ? bf16_at(r + at[e & 7]) : 0.f, d1 = live ? bf16_at(r + at[(e + 1) & 7]) : 0.f;
                        const float2 w = *reinterpret_cast<const float2 *>(&sm.scalars[c % Sm::kScalarRing][1][y + e]);
                        split2(p.scale * w.x * d0, p.scale * w.y * d1, hi[e / 2], lo[e / 2]);
                    }
                    tmem_st8(tl + Col::pu + y / 2, hi);
                    tmem_st8(tl + Col::pu + 32 + y / 2, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sm.d_ready);
            }
            if (kKeep) {  // the state before the chunk, once its image is written
                if (!(ok = wait(&sm.s_ready, ph))) break;
                if (warp == kOutWarp && lane == 0) {
                    bulk_store(states + ((size_t)bh * chunks + x) * state_bytes(DK, DV), sm.state, state_bytes(DK, DV));
                    tma_store_commit();
                    tma_store_wait_read_all();
                    mbar_arrive(&sm.stored);
                }
                __syncwarp();
                if (!(ok = wait(&sm.e_full[st], (uint32_t)(c >> 1) & 1u))) break;
                tc_fence_after();
                if (!Sm::kOutOverW && c > 0) named_bar_sync(1, 128);  // (the store above waited for the last rows' too)
                if (live)
#pragma unroll
                    for (int y = 0; y < kChunk; y += 16) {
                        uint32_t a[16];
                        tmem_ld16(tl + Col::e + 64 * st + y, a);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            uint32_t hi, lo;
                            split2(__uint_as_float(a[e]), __uint_as_float(a[e + 1]), hi, lo);
                            uint8_t *to = out + (y + e) / 8 * 1024;
                            *reinterpret_cast<uint16_t *>(to + at[e & 7]) = (uint16_t)hi;
                            *reinterpret_cast<uint16_t *>(to + at[(e + 1) & 7]) = (uint16_t)(hi >> 16);
                            *reinterpret_cast<uint16_t *>(to + rows_bytes(DV) / 2 + at[e & 7]) = (uint16_t)lo;
                            *reinterpret_cast<uint16_t *>(to + rows_bytes(DV) / 2 + at[(e + 1) & 7]) = (uint16_t)(lo >> 16);
                        }
                    }
                tc_fence_before();
                fence_proxy_async_smem();
                mbar_arrive(&sm.o_read[st]);
                named_bar_sync(1, 128);
                if (warp == kOutWarp && lane == 0) {
                    bulk_store(rows + ((size_t)bh * chunks + x) * rows_bytes(DV), out, rows_bytes(DV));
                    tma_store_commit();
                    if (Sm::kOutOverW) tma_store_wait_read_all();
                    mbar_arrive(&sm.rows_read[st]);
                }
                __syncwarp();
            } else {
                if (!(ok = wait(&sm.o_full[st], (uint32_t)(c >> 1) & 1u))) break;
                tc_fence_after();
                if (Sm::kStageO && c > 0) {  // the last store has read the tile
                    if (warp == kOutWarp && lane == 0) tma_store_wait_read_all();
                    __syncwarp();
                    named_bar_sync(1, 128);
                }
                const float *first = sm.scalars[c % Sm::kScalarRing][2];
                const int t0 = x * kChunk;
                // (without a stage: a warp writes 32 neighbouring features of a row, whole sectors)
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + ((size_t)bh * p.N + t0) * p.dv + f;
                if (Sm::kStageO ? live : f < p.dv)
#pragma unroll
                    for (int y = 0; y < kChunk; y += 16) {
                        uint32_t a[16], b[16];
                        const uint32_t tQ = tl + Col::qs + (Sm::kOuts == 2 ? 128 * st : 0);
                        tmem_ld16(tQ + y, a);
                        tmem_ld16(tQ + 64 + y, b);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 w = *reinterpret_cast<const float2 *>(first + y + e);
                            float o0, o1;
                            unpair(mul2(pair(p.scale, p.scale), fma2(pair(w.x, w.y), pair(__uint_as_float(a[e]), __uint_as_float(a[e + 1])),
                                                                     pair(__uint_as_float(b[e]), __uint_as_float(b[e + 1])))), o0, o1);
                            if constexpr (Sm::kStageO) {
                                const uint32_t both = pack_bf16(o0, o1);
                                uint8_t *to = out + (y + e) / 8 * 1024;
                                *reinterpret_cast<uint16_t *>(to + at[e & 7]) = (uint16_t)both;
                                *reinterpret_cast<uint16_t *>(to + at[(e + 1) & 7]) = (uint16_t)(both >> 16);
                            } else {
                                if (t0 + y + e < p.N) o[(size_t)(y + e) * p.dv] = __float2bfloat16_rn(o0);
                                if (t0 + y + e + 1 < p.N) o[(size_t)(y + e + 1) * p.dv] = __float2bfloat16_rn(o1);
                            }
                        }
                    }
                tc_fence_before();
                if constexpr (Sm::kStageO) {
                    fence_proxy_async_smem();
                    mbar_arrive(&sm.o_read[st]);
                    named_bar_sync(1, 128);
                    if (warp == kOutWarp && lane == 0) {
                        for (int b = 0; b < DV / 64; ++b) tma_store_3d(&map_o, out + b * kSq, 64 * b, t0, bh);
                        tma_store_commit();
                    }
                    __syncwarp();
                } else {
                    mbar_arrive(&sm.o_read[st]);
                }
            }
        }
        if (warp == kOutWarp && lane == 0) tma_store_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Prepares the chunks' images, for the forward pass or (kBack) for the backward.
template <int DK, bool kBack>
la_status prepare(const DeltaProblem &p, const Params &prm, uint8_t *images, CUtensorMap *mq, CUtensorMap *mk)
{
    typedef PrepSmem<DK, kBack> Sm;
    la_status st = make_map(mq, p.q, p.B * p.Hk, p.N, p.dk, kChunk);
    if (st == LA_OK) st = make_map(mk, p.k, p.B * p.Hk, p.N, p.dk, kChunk);
    if (st == LA_OK) st = ensure_smem((const void *)delta_prepare<DK, kBack>, (int)sizeof(Sm));
    if (st != LA_OK) return st;
    g_launched = true;
    count_launches();
    return launch_dependent(delta_prepare<DK, kBack>, (unsigned)(p.B * p.H * ceil_div(p.N, kChunk)), kBack ? 256 : 128, (int)sizeof(Sm),
                            p.stream, *mq, *mk, prm, images);
}

}  // namespace
}  // namespace delta
}  // namespace la
