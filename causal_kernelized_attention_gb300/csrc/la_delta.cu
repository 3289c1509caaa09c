// Gated delta rule on the CUDA cores: for fp32 the scan, its reverse and the gradients of a chunk; and the
// decode step.
//
//   D_t = a_t S_{t-1},  e_t = v_t - D_t^T k_t,  S_t = D_t + k_t (b_t e_t)^T,  o_t = scale S_t^T q_t
//
// with a_t = exp(g_t).  Columns of S (one per value feature) do not meet, so a scan's blocks take
// 8 or 32 columns each and hold them in registers.  Token by token a scan waits: a dot product over d_k, two
// shuffles and the update follow one another (345 cycles a token at d_k 32, whatever the machine has free).  So
// eight tokens are taken together: with G the running sum of g from their first on and D_ij = exp(G_i - G_j),
//   e_i = v_i - exp(G_i) S^T k_i - sum_{j<i} D_ij (k_i.k_j) u_j,   u = b e,
//   o_i = scale (exp(G_i) S^T q_i + sum_{j<=i} D_ij (q_i.k_j) u_j),   S' = exp(G_8) S + sum_j exp(G_8 - G_j) k_j u_j^T,
// where the 16 dot products with S are independent and the small matrices are found once for all columns.
#include "la_common.cuh"
#include "la_delta.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace delta {
namespace {

constexpr int kTile = 16;   // tokens staged in shared memory at a time
constexpr int kB = 8;       // tokens taken together
constexpr int kStepCols = 32;  // columns of S a block of the decode step
// Rows of S a lane holds in a scan of CB columns a block; d_k / rows lanes share a column.
constexpr int rows_of(int CB) { return CB == 8 ? 4 : 8; }
template <int DK, int CB> constexpr int scan_threads() { return CB * DK / rows_of(CB); }
constexpr int kMakers = 128;  // threads that load and prepare the tiles
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

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void named_bar(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
template <int n> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

// The rows of one tile: keys, queries (four floats further apart than they are long: the pairs' dot products read
// eight rows at once), a slice of CB values (forward: v, reverse: dO), gates.
template <int DK, int CB> struct alignas(16) Stage {
    float k[kTile][DK + 4], q[kTile][DK + 4], v[kTile][CB];
    float g[kTile], beta[kTile];
};
// What a tile's groups of 8 tokens need: D_ij (k_i.k_j) below the diagonal, D_ij (q_i.k_j) up to it (and their
// transposes, which the reverse reads).
struct alignas(16) Group {
    float N[kB][kB], P[kB][kB], first[kB], last[kB], whole[4];
};
// Three tiles are under way: one scanned, the next one's groups made by the last four warps, a third loaded.
template <int DK, int CB> struct ScanSmem {
    Stage<DK, CB> stage[3];
    Group groups[2][2];
};

// Rows t0 .. of one tile, by the kMakers threads; rows past the sequence are zeros (which leave S as it is).
template <int DK, int CB>
__device__ __forceinline__ void load_stage(Stage<DK, CB> &s, const float *k, const float *q, const float *v, const float *g,
                                           const float *beta, int t0, int n, int dv, int tid)
{
    const int rows = min(kTile, n - t0);
    auto copy = [&](float *dst, const float *src, bool on) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                     "r"(on ? 16 : 0));
    };
    for (int i = tid; i < kTile * (DK / 4); i += kMakers) {
        const int r = i / (DK / 4), c = i % (DK / 4) * 4;
        const size_t at = r < rows ? (size_t)(t0 + r) * DK + c : 0;
        copy(&s.k[r][c], k + at, r < rows);
        copy(&s.q[r][c], q + at, r < rows);
    }
    if (tid < kTile * CB / 4) {
        const int r = tid / (CB / 4), c = tid % (CB / 4) * 4;
        copy(&s.v[r][c], v + (r < rows ? (size_t)(t0 + r) * dv + c : 0), r < rows);
    }
    if (tid < 2 * kTile) {
        const int t = tid & (kTile - 1);
        const float *src = (tid < kTile ? g : beta) + (t < rows ? t0 + t : 0);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(tid < kTile ? &s.g[t] : &s.beta[t])),
                     "l"(src), "r"(t < rows ? 4 : 0));
    }
}

__device__ __forceinline__ void row8(const float *p, float (&v)[kB])
{
    const float4 a = Vec4<float>::get(p), b = Vec4<float>::get(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// The tile's two groups, by the kMakers threads, 64 to a group and each with one product of rows: thread (x, y) has
// q_x.k_y for y <= x, else k_y.k_x.  The sums of at most 8 gates are taken as they are, without differences.
template <int DK, int CB, bool kTransposed>
__device__ __forceinline__ void make_groups(const Stage<DK, CB> &s, Group (&out)[2], int tid)
{
    const int x = tid >> 3 & 7, y = tid & 7, r0 = tid >> 6 << 3, i = x > y ? x : y, j = x > y ? y : x;
    Group &o = out[tid >> 6];
    float g[kB];
    row8(s.g + r0, g);
    const ulonglong2 *a = reinterpret_cast<const ulonglong2 *>(y <= x ? s.q[r0 + i] : s.k[r0 + i]);
    const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(s.k[r0 + j]);
    uint64_t s0 = 0, s1 = 0;
#pragma unroll 8
    for (int c = 0; c < DK / 4; ++c) {
        const ulonglong2 u = a[c], w = b[c];
        s0 = fma2(u.x, w.x, s0);
        s1 = fma2(u.y, w.y, s1);
    }
    float d = 0.f, up = 0.f, down = 0.f, e, f;  // G_i - G_j, G_i, G_8 - G_i
#pragma unroll
    for (int t = 0; t < kB; ++t) {
        d += t > j && t <= i ? g[t] : 0.f;
        up += t <= i ? g[t] : 0.f;
        down += t > i ? g[t] : 0.f;
    }
    unpair(add2(s0, s1), e, f);
    const float product = expf(d) * (e + f);
    if (y <= x) {
        (kTransposed ? o.P[j][i] : o.P[i][j]) = product;
        if (i != j) (kTransposed ? o.P[i][j] : o.P[j][i]) = 0.f;
    } else {
        (kTransposed ? o.N[j][i] : o.N[i][j]) = product;
    }
    if (i == j) {
        const float all = expf(up);
        o.first[i] = all;
        o.last[i] = expf(down);
        if (i == kB - 1) o.whole[0] = all;
    }
}

// R rows of a column to a lane, DK / R lanes to a column: lane `part` holds rows 4 part .. + 3 of each R / 4-th of
// them, so that a warp's reads of a key are consecutive.  The lane's share of x^T S:
template <int DK, int R> __device__ __forceinline__ float dot_rows(const float *x, const uint64_t (&S)[R / 2], int part)
{
    uint64_t sum = 0;
#pragma unroll
    for (int r = 0; r < R / 2; r += 2) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(x + r / 2 * (4 * DK / R) + 4 * part);
        sum = r ? fma2(a.x, S[r], sum) : mul2(a.x, S[r]);
        sum = fma2(a.y, S[r + 1], sum);
    }
    float u, v;
    unpair(sum, u, v);
    return u + v;
}
template <int DK, int R> __device__ __forceinline__ void add_row(uint64_t (&S)[R / 2], const float *x, float w, int part)
{
    const uint64_t ww = pair(w, w);
#pragma unroll
    for (int r = 0; r < R / 2; r += 2) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(x + r / 2 * (4 * DK / R) + 4 * part);
        S[r] = fma2(a.x, ww, S[r]);
        S[r + 1] = fma2(a.y, ww, S[r + 1]);
    }
}
// Sums of 8 values over the L lanes of a column: lane p gets that of value p % 8, and with four lanes that of p + 4.
template <int L> __device__ __forceinline__ void lane_sums(const float (&v)[kB], int part, float (&out)[L == 4 ? 2 : 1])
{
    float a[4], b[2];
    auto swap = [](float keep, float give, int d) { return keep + __shfl_xor_sync(0xffffffffu, give, d); };
    const bool b0 = part & 1, b1 = part & 2, b2 = part & 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = swap(b0 ? v[2 * e + 1] : v[2 * e], b0 ? v[2 * e] : v[2 * e + 1], 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) b[e] = swap(b1 ? a[2 * e + 1] : a[2 * e], b1 ? a[2 * e] : a[2 * e + 1], 2);
    if constexpr (L == 4) {
        out[0] = b[0], out[1] = b[1];
    } else {
        out[0] = swap(b2 ? b[1] : b[0], b2 ? b[0] : b[1], 4);
        if (L >= 16) out[0] += __shfl_xor_sync(0xffffffffu, out[0], 8);
        if (L == 32) out[0] += __shfl_xor_sync(0xffffffffu, out[0], 16);
    }
}
// All 8 sums in every lane of the column.
template <int L> __device__ __forceinline__ void all_sums(float (&v)[kB], int part)
{
    float own[L == 4 ? 2 : 1];
    lane_sums<L>(v, part, own);
#pragma unroll
    for (int j = 0; j < kB; ++j) v[j] = __shfl_sync(0xffffffffu, own[L == 4 ? j >> 2 : 0], L == 4 ? j & 3 : j, L);
}
template <int DK, int R> __device__ __forceinline__ void state_out(float *at, const uint64_t (&S)[R / 2], int part, int dv)
{
#pragma unroll
    for (int r = 0; r < R; r += 2) {
        float x, y;
        unpair(S[r / 2], x, y);
        float *to = at + (size_t)(r / 4 * (4 * DK / R) + part * 4 + r % 4) * dv;
        to[0] = x, to[dv] = y;
    }
}
template <int DK, int R> __device__ __forceinline__ void state_in(const float *at, uint64_t (&S)[R / 2], int part, int dv)
{
#pragma unroll
    for (int r = 0; r < R; r += 2) {
        const float *from = at + (size_t)(r / 4 * (4 * DK / R) + part * 4 + r % 4) * dv;
        S[r / 2] = at ? pair(from[0], from[dv]) : 0;
    }
}
// The tiles of one slice in order (kDown: from the last): one(stage, groups, tile) by all but the last four warps
// on a tile that is there.
template <int DK, int CB, bool kDown, typename F>
__device__ __forceinline__ void over_tiles(ScanSmem<DK, CB> &sm, const float *k, const float *q, const float *v, const float *g,
                                           const float *beta, int n, int dv, F one)
{
    const int tiles = (n + kTile - 1) / kTile, tid = (int)threadIdx.x - scan_threads<DK, CB>();
    const bool maker = tid >= 0;
    auto tile = [&](int i) { return kDown ? tiles - 1 - i : i; };
    auto load = [&](int i) {
        if (i < tiles) load_stage<DK, CB>(sm.stage[i % 3], k, q, v, g, beta, tile(i) * kTile, n, dv, tid);
        copies_commit();
    };
    if (maker) {
        load(0);
        load(1);
        copies_wait<1>();
        named_bar(1, kMakers);  // tile 0 of all the makers
        if (tiles > 0) make_groups<DK, CB, kDown>(sm.stage[0], sm.groups[0], tid);
    }
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        if (maker) {
            load(i + 2);
            copies_wait<1>();
            named_bar(1, kMakers);
            if (i + 1 < tiles) make_groups<DK, CB, kDown>(sm.stage[(i + 1) % 3], sm.groups[(i + 1) & 1], tid);
        } else {
            one(sm.stage[i % 3], sm.groups[i & 1], tile(i));
        }
        __syncthreads();
    }
}

// kSave: instead of o, the errors e_t and the state before each chunk of kC tokens.
template <int DK, int CB, bool kSave>
__device__ __forceinline__ void scan(ScanSmem<DK, CB> &sm, const Params &p, int block, float *errors, float *before)
{
    const int slices = p.dv / CB, bh = block / slices, c0 = block % slices * CB;
    constexpr int R = rows_of(CB), L = DK / R;  // rows of a lane, lanes of a column
    const int part = threadIdx.x % L, col = threadIdx.x / L % CB;
    const bool scanner = threadIdx.x < CB * L;
    const int b = bh / p.H, bhk = b * p.Hk + bh % p.H / (p.H / p.Hk);
    const float *k = static_cast<const float *>(p.k) + (size_t)bhk * p.N * DK, *q = static_cast<const float *>(p.q) + (size_t)bhk * p.N * DK;
    const float *v = static_cast<const float *>(p.v) + (size_t)bh * p.N * p.dv + c0;
    const size_t at = (size_t)bh * DK * p.dv + c0 + col;
    const int chunks = (p.N + kC - 1) / kC;
    uint64_t S[R / 2];
    state_in<DK, R>(p.S0 && scanner ? p.S0 + at : nullptr, S, part, p.dv);
    over_tiles<DK, CB, false>(sm, k, q, v, p.g + (size_t)bh * p.N, p.beta + (size_t)bh * p.N, p.N, p.dv,
                              [&](const Stage<DK, CB> &s, const Group (&groups)[2], int tile) {
        const int t0 = tile * kTile;
        if (kSave && t0 % kC == 0)
            state_out<DK, R>(before + ((size_t)bh * chunks + t0 / kC) * DK * p.dv + c0 + col, S, part, p.dv);
#pragma unroll  // the second group's dot products fill the waits of the first one's outputs (68 us -> 55 at 3 x 5 heads of 32 x 64, 1021 tokens)
        for (int h = 0; h < kTile / kB; ++h) {
            const Group &m = groups[h];
            const int r0 = kB * h;
            float u[kB], d[kB], first[kB], beta[kB];
#pragma unroll
            for (int j = 0; j < kB; ++j) u[j] = dot_rows<DK, R>(s.k[r0 + j], S, part);
            if (!kSave)
#pragma unroll
                for (int j = 0; j < kB; ++j) d[j] = dot_rows<DK, R>(s.q[r0 + j], S, part);
            row8(m.first, first);
            row8(s.beta + r0, beta);
            constexpr int kOwn = L == 4 ? 2 : 1;  // tokens whose results the lane writes: part % 8, and with four lanes part + 4
            float e[kOwn] = {};
            all_sums<L>(u, part);
#pragma unroll
            for (int j = 0; j < kB; ++j) u[j] = fmaf(-first[j], u[j], s.v[r0 + j][col]);
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                float n[kB], x = u[j];
                row8(m.N[j], n);
#pragma unroll
                for (int c = 0; c < j; ++c) x = fmaf(-n[c], u[c], x);
                if (kSave && (j & (L == 4 ? 3 : 7)) == (part & 7)) e[L == 4 ? j >> 2 : 0] = x;
                u[j] = beta[j] * x;
            }
            if (!kSave) {
                lane_sums<L>(d, part, e);
#pragma unroll
                for (int y = 0; y < kOwn; ++y) {
                    const int t = (part & 7) + 4 * y;
                    float w[kB];
                    row8(m.P[t], w);
                    e[y] *= m.first[t];
#pragma unroll
                    for (int c = 0; c < kB; ++c) e[y] = fmaf(w[c], u[c], e[y]);
                    e[y] *= p.scale;
                }
            }
#pragma unroll
            for (int y = 0; y < kOwn; ++y) {
                const int t = t0 + r0 + (part & 7) + 4 * y;
                if (part < 8 && t < p.N) (kSave ? errors : static_cast<float *>(p.o))[((size_t)bh * p.N + t) * p.dv + c0 + col] = e[y];
            }
            float last[kB];
            row8(m.last, last);
            const float whole = m.whole[0];
#pragma unroll
            for (int r = 0; r < R / 2; ++r) S[r] = mul2(S[r], pair(whole, whole));
#pragma unroll
            for (int j = 0; j < kB; ++j) add_row<DK, R>(S, s.k[r0 + j], last[j] * u[j], part);
        }
    });
    if (!kSave && p.SN && scanner) state_out<DK, R>(p.SN + at, S, part, p.dv);
}

// The reverse scan of R = dL/dS, 8 tokens together from the last on:
//   dX_j = exp(G_8 - G_j) R^T k_j + sum_{i>=j} D_ij (q_i.k_j) scale dO_i - sum_{i>j} D_ij (k_i.k_j) b_i dX_i,   dv = b dX,
//   R' = exp(G_8) R + sum_i exp(G_i) (q_i scale dO_i^T - k_i dv_i^T).
// Writes dv, dX, R behind each chunk (before the chunk's own dO) and dS0.
template <int DK, int CB>
__device__ __forceinline__ void reverse_scan(ScanSmem<DK, CB> &sm, const Params &p, int block, float *dX, float *after)
{
    const int slices = p.dv / CB, bh = block / slices, c0 = block % slices * CB;
    constexpr int R = rows_of(CB), L = DK / R;  // rows of a lane, lanes of a column
    const int part = threadIdx.x % L, col = threadIdx.x / L % CB;
    const bool scanner = threadIdx.x < CB * L;
    const int b = bh / p.H, bhk = b * p.Hk + bh % p.H / (p.H / p.Hk);
    const float *k = static_cast<const float *>(p.k) + (size_t)bhk * p.N * DK, *q = static_cast<const float *>(p.q) + (size_t)bhk * p.N * DK;
    const float *dout = static_cast<const float *>(p.dout) + (size_t)bh * p.N * p.dv + c0;
    const size_t at = (size_t)bh * DK * p.dv + c0 + col;
    const int tiles = (p.N + kTile - 1) / kTile, chunks = (p.N + kC - 1) / kC;
    uint64_t S[R / 2];  // dL/dS
    state_in<DK, R>(p.dSN && scanner ? p.dSN + at : nullptr, S, part, p.dv);
    over_tiles<DK, CB, true>(sm, k, q, dout, p.g + (size_t)bh * p.N, p.beta + (size_t)bh * p.N, p.N, p.dv,
                             [&](const Stage<DK, CB> &s, const Group (&groups)[2], int tile) {
        const int t0 = tile * kTile;
        if (tile == tiles - 1 || (t0 + kTile) % kC == 0)
            state_out<DK, R>(after + ((size_t)bh * chunks + t0 / kC) * DK * p.dv + c0 + col, S, part, p.dv);
#pragma unroll
        for (int h = kTile / kB - 1; h >= 0; --h) {
            const Group &m = groups[h];
            const int r0 = kB * h;
            float x[kB], o[kB], w[kB], beta[kB];
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                x[j] = dot_rows<DK, R>(s.k[r0 + j], S, part);
                o[j] = p.scale * s.v[r0 + j][col];
            }
            row8(m.last, w);
            row8(s.beta + r0, beta);
            all_sums<L>(x, part);
#pragma unroll
            for (int j = 0; j < kB; ++j) x[j] *= w[j];
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                row8(m.P[j], w);
#pragma unroll
                for (int c = j; c < kB; ++c) x[j] = fmaf(w[c], o[c], x[j]);
            }
            constexpr int kOwn = L == 4 ? 2 : 1;
            float dx[kOwn] = {}, y[kB];  // dX of the lane's own tokens; y = dv
#pragma unroll
            for (int j = kB - 1; j >= 0; --j) {
                row8(m.N[j], w);
#pragma unroll
                for (int c = kB - 1; c > j; --c) x[j] = fmaf(-w[c], y[c], x[j]);
                if ((j & (L == 4 ? 3 : 7)) == (part & 7)) dx[L == 4 ? j >> 2 : 0] = x[j];
                y[j] = beta[j] * x[j];
            }
#pragma unroll
            for (int u = 0; u < kOwn; ++u) {
                const int t = t0 + r0 + (part & 7) + 4 * u;
                const size_t row = ((size_t)bh * p.N + t) * p.dv + c0 + col;
                if (part < 8 && t < p.N) {
                    dX[row] = dx[u];
                    static_cast<float *>(p.dv_out)[row] = s.beta[t - t0] * dx[u];
                }
            }
            row8(m.first, w);
            const float whole = m.whole[0];
#pragma unroll
            for (int r = 0; r < R / 2; ++r) S[r] = mul2(S[r], pair(whole, whole));
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                add_row<DK, R>(S, s.q[r0 + j], w[j] * o[j], part);
                add_row<DK, R>(S, s.k[r0 + j], -w[j] * y[j], part);
            }
        }
    });
    if (p.dS0 && scanner) state_out<DK, R>(p.dS0 + at, S, part, p.dv);
}

template <int DK, int CB> __global__ void __launch_bounds__(scan_threads<DK, CB>() + kMakers) delta_scan(Params p)
{
    extern __shared__ float4 smem_raw[];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    scan<DK, CB, false>(*reinterpret_cast<ScanSmem<DK, CB> *>(smem_raw), p, blockIdx.x, nullptr, nullptr);
}
// Both scans of the backward pass, which do not meet: the first half of the blocks goes forward, the second in reverse.
template <int DK, int CB>
__global__ void __launch_bounds__(scan_threads<DK, CB>() + kMakers)
delta_scans(Params p, float *errors, float *before, float *dX, float *after)
{
    extern __shared__ float4 smem_raw[];
    ScanSmem<DK, CB> &sm = *reinterpret_cast<ScanSmem<DK, CB> *>(smem_raw);
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half)
        scan<DK, CB, true>(sm, p, blockIdx.x, errors, before);
    else
        reverse_scan<DK, CB>(sm, p, blockIdx.x - half, dX, after);
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

template <int DK, int DV>
__global__ void __launch_bounds__(256) delta_local(Params p, const float *errors, const float *dX, const float *before,
                                                   const float *after)
{
    extern __shared__ float4 smem_raw[];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    LocalSmem<DK, DV> &s = *reinterpret_cast<LocalSmem<DK, DV> *>(smem_raw);
    constexpr int kKG = DK / 4, kI = DK / 32;  // threads along d_k; rows a thread
    const int chunks = (p.N + kC - 1) / kC, bhk = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int group = p.H / p.Hk, t0 = chunk * kC, rows = min(kC, p.N - t0), tid = threadIdx.x;
    const int kg = tid % kKG, i0 = tid / kKG * kI;
    for (int i = tid; i < kC * DK; i += 256) {
        const int r = i / DK, c = i % DK;
        const size_t at = ((size_t)bhk * p.N + t0 + r) * DK + c;
        s.K[r][c] = r < rows ? static_cast<const float *>(p.k)[at] : 0.f;
        s.Q[r][c] = r < rows ? static_cast<const float *>(p.q)[at] : 0.f;
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
                s.O[r][c] = r < rows ? p.scale * static_cast<const float *>(p.dout)[at] : 0.f;
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
                static_cast<float *>(p.dq)[at] = dq[i][m];
                static_cast<float *>(p.dk_out)[at] = dk[i][m];
            }
}

// One decode step.  A block takes 32 columns of one head's state: 16 rows of eight lanes with four
// columns each, so that a warp reads four rows of 128 bytes and every thread has DK / 16 loads in flight.  The dot
// products with k and q are taken in the one pass that reads S, as S_t^T q = a S^T q + (k.q) u.
template <typename T, int DK>
__global__ void __launch_bounds__(128) delta_step_kernel(Params p, float *S)
{
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    __shared__ float ks[DK], qs[DK];
    __shared__ float4 part[2][4][8];
    const int slices = p.dv / kStepCols, bh = blockIdx.x / slices, c0 = blockIdx.x % slices * kStepCols;
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

// Calls f with d_k, or with d_k and d_v, as types.
template <typename F> la_status by_width(int d, F f)
{
    return d == 32   ? f(std::integral_constant<int, 32>())
           : d == 64 ? f(std::integral_constant<int, 64>())
                     : f(std::integral_constant<int, 128>());
}
template <typename F> la_status by_widths(const DeltaProblem &p, F f)
{
    return by_width(p.dk, [&](auto dk) { return by_width(p.dv, [&](auto dv) { return f(dk, dv); }); });
}

// A scan's launch, with CB columns of a head's state to a block.
template <int DK, int CB, typename... Args>
la_status launch_scan(const DeltaProblem &p, int scans, void (*kernel)(Params, Args...), const Params &prm, Args... args)
{
    const int smem = (int)sizeof(ScanSmem<DK, CB>);
    const la_status st = ensure_smem(reinterpret_cast<const void *>(kernel), smem);
    if (st != LA_OK) return st;
    count_launches();
    return tc::launch_dependent(kernel, (unsigned)(scans * p.B * p.H * (p.dv / CB)), scan_threads<DK, CB>() + kMakers, smem, p.stream, prm, args...);
}
// Blocks of 32 columns or of 8: a narrow block's chain is shorter (at d_k 32, 64, 128 and 128 value features, 1000 tokens: 57,
// 87, 137 us against 86, 143, 367), but two of them share an SM (75, 132, 270 us a round), a wide one has it alone: wide ones
// where they take fewer rounds (24 heads: 87, 142, 367 us against 142, 212, 400; 19 heads, one round of either: narrow).
bool wide_slices(const DeltaProblem &p, int scans)
{
    const int sms = tc::sm_count();
    const long long columns = (long long)scans * p.B * p.H * p.dv;
    auto rounds = [](long long blocks, int slots) { return (blocks + slots - 1) / slots; };
    return rounds(columns / 32, sms) < rounds(columns / 8, 2 * sms);
}

template <int DK, int DV>
la_status launch_local(const DeltaProblem &p, const Params &prm, const float *errors, const float *dX, const float *before,
                       const float *after)
{
    const int smem = (int)sizeof(LocalSmem<DK, DV>);
    const la_status st = ensure_smem(reinterpret_cast<const void *>(&delta_local<DK, DV>), smem);
    if (st != LA_OK) return st;
    const unsigned grid = (unsigned)p.B * p.Hk * ceil_div(p.N, kC);
    count_launches();
    return tc::launch_dependent(&delta_local<DK, DV>, grid, 256, smem, p.stream, prm, errors, dX, before, after);
}

}  // namespace
}  // namespace delta

using namespace delta;

la_status delta_forward_simt(const DeltaProblem &p)
{
    return by_width(p.dk, [&](auto dk) {
        constexpr int DK = decltype(dk)::value;
        return wide_slices(p, 1) ? launch_scan<DK, 32>(p, 1, &delta_scan<DK, 32>, params_of(p))
                                 : launch_scan<DK, 8>(p, 1, &delta_scan<DK, 8>, params_of(p));
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
    return by_widths(p, [&](auto dk, auto dv) {
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
        const la_status st = wide_slices(p, 2)
                                 ? launch_scan<DK, 32>(p, 2, &delta_scans<DK, 32>, prm, errors, before, dX, after)
                                 : launch_scan<DK, 8>(p, 2, &delta_scans<DK, 8>, prm, errors, before, dX, after);
        if (st != LA_OK || p.N == 0) return st;
        return launch_local<DK, DV>(p, prm, errors, dX, before, after);
    });
}

la_status delta_step(const DeltaProblem &p, float *S)
{
    const Params prm = params_of(p);
    return by_width(p.dk, [&](auto dk) {
        constexpr int DK = decltype(dk)::value;
        const unsigned grid = (unsigned)(p.B * p.H * (p.dv / kStepCols));
        count_launches();
        return p.dtype == LA_F32 ? tc::launch_dependent(&delta_step_kernel<float, DK>, grid, 128, 0, p.stream, prm, S)
                                 : tc::launch_dependent(&delta_step_kernel<__nv_bfloat16, DK>, grid, 128, 0, p.stream, prm, S);
    });
}

}  // namespace la
