// Window attention backward on the tensor cores: bf16, d <= 128 on tiles of 64 or 128
// columns.  D = dO . o of every row first (window_tc_rows), then one launch of two kinds of
// blocks, so that every gradient is summed by one CTA in a fixed order:
//
//   dq      (a CTA: two query tiles of 128 rows, as the forward; key tiles of 64)
//           S = Q K^T, dP = dO V^T, dS = P (dP - D), dQ += dS K;      3 products a tile
//   dk, dv  (a CTA: 128 keys; query tiles of 64 rows, of every head of the group)
//           S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q;   4 products a tile
//
// with P = exp(scale S - lse); scale multiplies dS once, in the epilogues.  A product's left
// operand comes from TMEM where it is P or dS: each is rounded to bf16 and written over the
// columns it was computed from, so nothing of the score matrices reaches shared memory.
// Two groups of four warps work in turn, as in the forward: while one forms P and dS of its
// tile (a thread a row), the tensor core runs the products of the other's.  In dk, dv a
// thread owns a key, for which the visible queries are one interval.  Sums are fp32.
//
// The rounding of P and dS (2^-8 relative at most, each on its own) averages out in a long sum, where the
// gradients' error is about 1.4 times that of their own rounding, but not in a short one: of a row that sees two keys
// the two dS are each other's negatives, and all of dq is off by what they are.  A block whose shortest sum (a
// row's visible keys, a key's query rows) has at most 256 terms therefore multiplies P and dS as two
// bf16 parts each (2^-16): 16 heads on 4, d 128, 128 rows 16.2 us (14.0 with one part), 8192 rows of window 128 98 us (91);
// long sums would pay more for it (8192 rows, window 1024: 277 us instead of 244) and have less need.
//
// A tile of sinks is seen by every later row.  Its rows are shared out over several CTAs,
// each about a window tile's work; their fp32 sums go to scratch and a third, small kernel
// adds them up in order (otherwise those few CTAs outlast all others: 864 us instead of
// 150 at 8192 rows, window 1024).  All tiles are shared out in the same way where the launch has
// fewer CTAs than there are SMs (16 on 4 heads, d 128: 512 rows 34 -> 24 us, 1024 rows 61 -> 42;
// 8 heads on one, 1500 rows 132 -> 37).
//
// Rows and keys of padding: their P and dS are 0, and what a product multiplies by them is
// zeroed in shared memory (0 times a NaN is not 0).
#include <algorithm>
#include <type_traits>

#include "la_tc_window.cuh"

namespace la {
namespace {

using namespace window;

static __device__ unsigned g_winb_status;
std::atomic<bool> g_launched{false};

constexpr int kHalf = 64;  // keys (dq) or query rows (dk, dv) of a streamed tile
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kHalfBox = kHalf * 128;  // one [64 rows x 64 bf16] swizzled box: 8 KB
constexpr uint32_t tS = 0, tP = 128, tG = 256;  // S_s at 64 s, dP_s at 128 + 64 s, gradients from 256
constexpr int kFewTerms = 256;  // of a sum, up to which P and dS are multiplied as two parts
// P and dS lie over the 32 columns that each half of them came from: 16 columns of bf16 pairs, then 16 of
// what their rounding left (where that is multiplied too).
constexpr uint32_t kRest = 16;
__device__ __forceinline__ constexpr uint32_t half_at(int kk) { return (uint32_t)((kk >> 1) * 32 + (kk & 1) * 8); }

// Rounds a half's 32 values to bf16 at TMEM address t, and with kFine the rest behind them.
template <bool kFine>
__device__ __forceinline__ void store_half(uint32_t t, const uint32_t (&x)[32])
{
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) pk[e] = pack_bf16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
    tmem_st16(t, pk);
    if constexpr (kFine) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            pk[e] = pack_bf16(__uint_as_float(x[2 * e]) - __uint_as_float(pk[e] << 16),
                              __uint_as_float(x[2 * e + 1]) - __uint_as_float(pk[e] & 0xffff0000u));
        tmem_st16(t + kRest, pk);
    }
}

__device__ __forceinline__ bool wait_b(int *abort_flag, uint64_t *bar, uint32_t parity)
{
    return wait_bar(&g_winb_status, abort_flag, bar, parity);
}
__device__ __forceinline__ bool wait_w(int *abort_flag, uint64_t *bar, uint32_t parity)
{
    return wait_bar_warp(&g_winb_status, abort_flag, bar, parity);
}
// Descriptors of a 64-row tile.
__device__ __forceinline__ uint64_t kmajor_half(uint32_t tile, int kk)
{
    return desc_sw128(tile + (kk >> 2) * kHalfBox + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t mnmajor_half(uint32_t tile, int kk) { return mnmajor(tile, kk, kHalfBox); }

// Zeroes rows from r0 on of a 64-row tile, by one warp, visible to the tensor core.
template <int DT>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int r0, int lane)
{
    r0 = max(r0, 0);
    for (int e = lane; e < (kHalf - r0) * (DT / 8); e += 32) {
        const int row = r0 + e / (DT / 8), ch = e % (DT / 8);
        *reinterpret_cast<uint4 *>(tile + (ch >> 3) * kHalfBox + row * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Row r of a 128-row output tile: 16 fp32 columns from x of TMEM address ta, times f, as bf16.
__device__ __forceinline__ void stage16(uint8_t *tile, uint32_t ta, int r, int x, float f, bool some)
{
    uint32_t o[16], pk[8];
    tmem_ld16(ta + x, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e)
        pk[e] = some ? pack_bf16(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f) : 0u;
    uint8_t *row = tile + x / 64 * kBox + r * 128;
    const int ch = (x & 63) >> 3;
    *reinterpret_cast<uint4 *>(row + ((ch ^ (r & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    *reinterpret_cast<uint4 *>(row + (((ch + 1) ^ (r & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
}

// ---------------------------------------------------------------- dq
constexpr int kKeyStages = 3;

template <int DT>
struct DqSmem {
    static constexpr uint32_t kTile = kRows * DT * 2, kStage = kHalf * DT * 2;
    uint8_t q[2][kTile];  // then dq, staged
    uint8_t go[2][kTile];
    uint8_t k[kKeyStages][kStage];
    uint8_t v[kKeyStages][kStage];
    uint64_t q_full[2], s_full[2], ds_full[2], g_full[2];
    uint64_t k_full[kKeyStages], k_empty[kKeyStages], v_full[kKeyStages], v_empty[kKeyStages], drain;
    uint32_t tmem_base;
    int abort;
};

// The launch's tensor maps: tiles of 128 rows, and of 64 for what is streamed.
struct Maps {
    CUtensorMap q, go, k, v, q_half, go_half, k_half, v_half, dq, dk, dv;
};

// Whether the first row of a dq block, which sees the fewest keys, has few terms.
__device__ __forceinline__ bool few_keys(const Params &prm, int block)
{
    const int p = Work<kHalf>::first_row(prm, block % prm.units) + prm.Nk - prm.Nq;
    return p < kFewTerms || (prm.window <= kFewTerms && prm.sinks <= kFewTerms - prm.window);
}

// kFine: dS is multiplied as two parts.
template <int DT, bool kFine>
__device__ __forceinline__ void dq_block(const Maps &maps, const Params &prm, const int block, uint8_t *smem_raw)
{
    DqSmem<DT> &sm = *reinterpret_cast<DqSmem<DT> *>(smem_raw);
    constexpr uint32_t kTile = DqSmem<DT>::kTile, kStage = DqSmem<DT>::kStage;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.ds_full[s], 128);
            mbar_init(&sm.g_full[s], 1);
        }
        for (int i = 0; i < kKeyStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = (smem_u32(smem_raw) & 1023u) == 0 ? 0 : 1;
        if (sm.abort) atomicOr(&g_winb_status, kStatusTimeout);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    int *abort_flag = &sm.abort;
    const Work<kHalf> w(prm, block);
    const int U = w.count();

    if (warp == kTmaWarp) {
        if (lane == 0 && !aborted(abort_flag)) {
            const int kz = w.b * prm.Hk + w.hk;
            int loaded = 0;
            for (int u = 0; u < U; ++u) {
                const int st = u % kKeyStages, j0 = w.tile(u) * kHalf;
                const uint32_t ph = (uint32_t)(u / kKeyStages - 1) & 1u;
                if (u >= kKeyStages && !wait_b(abort_flag, &sm.k_empty[st], ph)) break;
                mbar_arrive_expect_tx(&sm.k_full[st], kStage);
#pragma unroll
                for (int x = 0; x < DT; x += 64)
                    tma_load_3d(sm.k[st] + x / 64 * kHalfBox, &maps.k_half, &sm.k_full[st], x, j0, kz);
                if (u == 0)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        if (w.kt[s].count() > 0) {
                            const int z = w.b * prm.Hq + w.h[s];
                            mbar_arrive_expect_tx(&sm.q_full[s], 2 * kTile);
#pragma unroll
                            for (int x = 0; x < DT; x += 64) {
                                tma_load_3d(sm.q[s] + x / 64 * kBox, &maps.q, &sm.q_full[s], x, w.t0[s], z);
                                tma_load_3d(sm.go[s] + x / 64 * kBox, &maps.go, &sm.q_full[s], x, w.t0[s], z);
                            }
                        }
                loaded = u + 1;
                if (u >= kKeyStages && !wait_b(abort_flag, &sm.v_empty[st], ph)) {
                    mbar_arrive_expect_tx(&sm.v_full[st], 0);  // completes the phase that drain() waits for
                    break;
                }
                mbar_arrive_expect_tx(&sm.v_full[st], kStage);
#pragma unroll
                for (int x = 0; x < DT; x += 64)
                    tma_load_3d(sm.v[st] + x / 64 * kHalfBox, &maps.v_half, &sm.v_full[st], x, j0, kz);
            }
            // no copy may still be writing shared memory when the CTA exits
            if (loaded > 0)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (w.kt[s].count() > 0) drain(&sm.q_full[s], 0);
            for (int u = max(loaded - kKeyStages, 0); u < loaded; ++u) {
                drain(&sm.k_full[u % kKeyStages], (uint32_t)(u / kKeyStages) & 1u);
                drain(&sm.v_full[u % kKeyStages], (uint32_t)(u / kKeyStages) & 1u);
            }
        }
    } else if (warp == kMmaWarp) {
        const uint32_t id_s = idesc_bf16_f32(128, kHalf, false, false), id_g = idesc_bf16_f32(128, DT, false, true);
        const uint64_t qd[2] = {kmajor(smem_u32(sm.q[0]), 0), kmajor(smem_u32(sm.q[1]), 0)};
        const uint64_t gd[2] = {kmajor(smem_u32(sm.go[0]), 0), kmajor(smem_u32(sm.go[1]), 0)};
        const uint64_t kd = kmajor_half(smem_u32(sm.k[0]), 0), vd = kmajor_half(smem_u32(sm.v[0]), 0);
        const uint64_t kt = mnmajor_half(smem_u32(sm.k[0]), 0);
        uint32_t st = 0, ph = 0, pst = 0;  // stage and phase of tile u, stage of tile u - 1
        uint32_t fed[2] = {0, 0};          // tiles of s whose dS has been multiplied
        bool pending[2] = {false, false};
        auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(&g_winb_status, abort_flag, bar, parity); };
        for (int u = 0; u <= U; ++u) {
            if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
            const int tile = u < U ? w.tile(u) : 0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (pending[s]) {
                    wait(&sm.ds_full[s], fed[s] & 1u);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t d = kt + pst * (kStage >> 4);
#pragma unroll
                        for (int kk = 0; kk < kHalf / 16; ++kk)
                            mma_ts(tmem + tG + s * DT, tmem + tS + s * kHalf + half_at(kk), d + kk * (2048 >> 4), id_g,
                                   fed[s] > 0 || kk > 0);
                        if (kFine)
#pragma unroll
                            for (int kk = 0; kk < kHalf / 16; ++kk)
                                mma_ts(tmem + tG + s * DT, tmem + tS + s * kHalf + half_at(kk) + kRest, d + kk * (2048 >> 4),
                                       id_g, true);
                    }
                    ++fed[s];
                    pending[s] = false;
                }
                if (s == 1 && u > 0 && elect_one()) mma_commit(&sm.k_empty[pst]);
                if (u < U) {
                    if (s == 0) {
                        wait(&sm.k_full[st], ph);
                        if (u == U - 1 && tile * kHalf + kHalf > w.n) zero_rows<DT>(sm.k[st], w.n - tile * kHalf, lane);
                        wait(&sm.v_full[st], ph);
                    }
                    if (w.reaches(s, tile)) {
                        if (fed[s] == 0) wait(&sm.q_full[s], 0);
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t so = st * (kStage >> 4);
#pragma unroll
                            for (int kk = 0; kk < DT / 16; ++kk)
                                mma_ss(tmem + tS + s * kHalf, qd[s] + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                                       kd + so + (((kk >> 2) * kHalfBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
#pragma unroll
                            for (int kk = 0; kk < DT / 16; ++kk)
                                mma_ss(tmem + tP + s * kHalf, gd[s] + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                                       vd + so + (((kk >> 2) * kHalfBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
                            mma_commit(&sm.s_full[s]);
                        }
                        pending[s] = true;
                    }
                    if (s == 1 && elect_one()) mma_commit(&sm.v_empty[st]);
                }
            }
            pst = st;
            if (++st == kKeyStages) st = 0, ph ^= 1u;
        }
        if (elect_one())
            for (int s = 0; s < 2; ++s) mma_commit(&sm.g_full[s]);
        if (elect_one()) {
            mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
            drain(&sm.drain, 0);
        }
        __syncwarp();
    } else {
        const int s = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + tS + s * kHalf, tp = tl + tP + s * kHalf, tg = tl + tG + s * DT;
        const KeyTiles kt = s ? w.kt[1] : w.kt[0];
        const int t0 = s ? w.t0[1] : w.t0[0], z = w.b * prm.Hq + (s ? w.h[1] : w.h[0]);
        const int t = t0 + r, p = t + w.off, p_first = t0 + w.off, tiles = kt.count();
        const bool live = t < prm.Nq && p < w.n;
        const float c = prm.scale * kLog2e;
        bool ok = !aborted(abort_flag);
        // the row's -lse in units of the raw scores, and its -D
        const size_t at = (size_t)z * prm.padded + t;
        const float delta = t0 < prm.Nq ? __ldcg(prm.delta + at) : 0.f;
        const float base = t0 < prm.Nq ? __ldcg(prm.delta + (size_t)prm.B * prm.Hq * prm.padded + at) : 0.f;
        const uint64_t base2 = pair(base, base), delta2 = pair(delta, delta), c2 = pair(c, c);
        for (int done = 0; ok && done < tiles; ++done) {
            const int j0 = kt.tile(done) * kHalf;
            if (!(ok = wait_w(abort_flag, &sm.s_full[s], (uint32_t)done & 1u))) break;
            tc_fence_after();
            const bool whole = j0 + kHalf - 1 <= p_first && p_first + kRows - 1 < w.n &&
                               (p_first + kRows - 1 - j0 < prm.window || j0 + kHalf <= prm.sinks);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t a[32], b[32];
                tmem_ld32(ts + 32 * g, a);
                tmem_ld32(tp + 32 * g, b);
                tmem_ld_wait();
                const uint32_t bits = whole ? 0xffffffffu : seen_bits(p, j0 + 32 * g, prm.window, prm.sinks, w.n);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float x, y;
                    split(mul2(add2(pair(a[e], a[e + 1]), base2), c2), x, y);
                    const uint64_t d = mul2(pair(ex2(x), ex2(y)), add2(pair(b[e], b[e + 1]), delta2));
                    split(d, x, y);
                    a[e] = __float_as_uint(x);
                    a[e + 1] = __float_as_uint(y);
                }
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((bits >> e) & 1u)) a[e] = 0u;
                }
                store_half<kFine>(ts + 32 * g, a);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.ds_full[s]);
        }
        if (ok) ok = U == 0 || wait_w(abort_flag, &sm.g_full[s], 0);
        if (ok && t0 < prm.Nq) {
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < DT; x += 16) stage16(sm.q[s], tg, r, x, prm.scale, live);
            fence_proxy_async_smem();
        }
        named_bar_sync(1 + s, 128);
        if (ok && t0 < prm.Nq && (warp & 3) == 0 && lane == 0) {
#pragma unroll
            for (int x = 0; x < DT; x += 64)
                tma_store_3d(&maps.dq, sm.q[s] + x / 64 * kBox, x, t0, z);
            tma_store_commit();
            tma_store_wait_all();
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- dk, dv
constexpr int kRowStages = 5;

// Which key tiles are shared out: the first `tiles` per key head, to `parts` CTAs each.  They are the
// tiles of sinks, or all where the launch would leave SMs idle.
struct Split {
    int tiles, parts;
};
Split split_of(const WindowProblem &p)
{
    Split sp{ceil_div(p.sinks, kRows), 1};
    const long long tiles = ceil_div(p.Nk, kRows), whole = ceil_div(p.Nq, kHalf);
    const long long win = std::min<long long>(whole, (p.window + kRows) / kHalf + 1);
    // a share is a window tile's work, or what half a CTA's share of the machine comes to
    const long long total = (long long)p.B * p.Hk * ((tiles - sp.tiles) * win + sp.tiles * whole);
    const long long unit = std::max(win, total / (2 * sm_count()));
    if (sp.tiles > 0) sp.parts = (int)((whole + unit - 1) / unit);
    // room for more CTAs, and shares of 4 query tiles (fewer than 12 are not worth the launch that adds up)
    const long long ctas = (long long)p.B * p.Hk * tiles, dq = (long long)p.B * p.Hk * params_of(p).units;
    const long long streamed = win * (p.Hq / p.Hk), more = std::min((sm_count() - dq) / std::max(ctas, 1LL), streamed / 4);
    if (streamed >= 12 && more > 1 && sp.parts <= more) sp = {(int)tiles, (int)more};
    return sp;
}
size_t split_floats(const WindowProblem &p, const Split &sp, int DT)
{
    return sp.parts > 1 ? (size_t)p.B * p.Hk * sp.tiles * sp.parts * 2 * kRows * DT : 0;
}

// Adds up the shares of the shared tiles, in order: 4 features a thread.
template <int DT>
__global__ void __launch_bounds__(256) window_tc_sum(const float *part, __nv_bfloat16 *dk, __nv_bfloat16 *dv, const Split sp,
                                                     int Nk, int d, float scale)
{
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;  // (bh, tile, dv or dk, row, 4 features)
    const int c = (int)(e % (DT / 4)) * 4, r = (int)(e / (DT / 4) % kRows), which = (int)(e / (DT / 4) / kRows % 2);
    const long long tile = e / (DT / 4) / kRows / 2;
    griddep_wait();
    griddep_launch_dependents();
    const int j = (int)(tile % sp.tiles) * kRows + r;
    if (j >= Nk || c >= d) return;
    const float *src = part + (tile * sp.parts * 2 + which) * (kRows * DT) + r * DT + c;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < sp.parts; ++i) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + (size_t)i * 2 * kRows * DT));
        sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
    }
    const float f = which ? scale : 1.f;
    *reinterpret_cast<uint2 *>((which ? dk : dv) + ((size_t)(tile / sp.tiles) * Nk + j) * d + c) =
        make_uint2(pack_bf16(sum.x * f, sum.y * f), pack_bf16(sum.z * f, sum.w * f));
}

template <int DT>
struct DkvSmem {
    static constexpr uint32_t kTile = kRows * DT * 2, kStage = kHalf * DT * 2;
    uint8_t k[kTile];  // then dk, staged
    uint8_t v[kTile];  // then dv, staged
    uint8_t q[kRowStages][kStage];
    uint8_t go[kRowStages][kStage];
    float delta[kRowStages][kHalf], base[kRowStages][kHalf];  // -D and -lse / scale of the rows
    uint64_t kv_full, s_full[2], ds_full[2], g_full;
    uint64_t q_full[kRowStages], q_empty[kRowStages], drain;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(DkvSmem<128>) <= 232448, "fits an SM's shared memory");

template <int DT>
__device__ __forceinline__ void dkv_block(const Maps &maps, const Params &prm, const Split &sp, float *part, const int block,
                                          uint8_t *smem_raw)
{
    DkvSmem<DT> &sm = *reinterpret_cast<DkvSmem<DT> *>(smem_raw);
    constexpr uint32_t kTile = DkvSmem<DT>::kTile, kStage = DkvSmem<DT>::kStage;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.kv_full, 1);
        mbar_init(&sm.g_full, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.ds_full[s], 128);
        }
        for (int i = 0; i < kRowStages; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = (smem_u32(smem_raw) & 1023u) == 0 ? 0 : 1;
        if (sm.abort) atomicOr(&g_winb_status, kStatusTimeout);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    int *abort_flag = &sm.abort;

    const int tiles = (prm.Nk + kRows - 1) / kRows, group = prm.Hq / prm.Hk, off = prm.Nk - prm.Nq;
    const int units = tiles + sp.tiles * (sp.parts - 1), bh = block / units, unit = block % units;
    const bool shared = unit < sp.tiles * sp.parts && sp.parts > 1;  // a share of a tile
    const int j0 = (shared ? unit / sp.parts : unit - sp.tiles * (sp.parts - 1)) * kRows, b = bh / prm.Hk, hk = bh % prm.Hk;
    const int n = valid(prm.lens, b, prm.Nk);
    const QueryTiles qt(j0, min(j0 + kRows, prm.Nk) - 1, prm.window, prm.sinks, n, off, prm.Nq, kHalf);
    // streamed tile x: head x / per of the group; this CTA's from x0 on, X of them
    const int per = qt.end - qt.begin, all = per * group, share = shared ? unit % sp.parts : 0;
    const int x0 = shared ? (int)((long long)all * share / sp.parts) : 0;
    const int X = (shared ? (int)((long long)all * (share + 1) / sp.parts) : all) - x0;
    const int rows = min(prm.Nq, n - off);  // rows of tokens
    // the query rows that see key j; the fewest of a tile are at its ends, or where the sinks end
    const int j1 = min(j0 + kRows, n) - 1;
    auto few = [&](int j) {
        const int last = j < prm.sinks ? n - 1 : min(n - 1, j + prm.window - 1);
        return (last - max(j, off) + 1) * (long long)group <= kFewTerms;
    };
    const bool fine = few(j0) || few(j1) || (j0 < prm.sinks && prm.sinks <= j1 && few(prm.sinks));

    // the products and the softmax groups, with P and dS in two parts or one
    auto run = [&](auto parts) {
        constexpr bool kFine = decltype(parts)::value;
        if (warp == kMmaWarp) {
            const uint32_t id_s = idesc_bf16_f32(128, kHalf, false, false), id_g = idesc_bf16_f32(128, DT, false, true);
            const uint64_t kd = kmajor(smem_u32(sm.k), 0), vd = kmajor(smem_u32(sm.v), 0);
            const uint64_t qd = kmajor_half(smem_u32(sm.q[0]), 0), gd = kmajor_half(smem_u32(sm.go[0]), 0);
            const uint64_t qt_ = mnmajor_half(smem_u32(sm.q[0]), 0), gt = mnmajor_half(smem_u32(sm.go[0]), 0);
            uint32_t st = 0, ph = 0, bst = 0;  // stage and phase of tile i, stage of tile i - 2
            int at = per > 0 ? x0 % per : 0;   // tile i's place within its head
            auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(&g_winb_status, abort_flag, bar, parity); };
            if (X > 0) wait(&sm.kv_full, 0);
            for (int i = 0; i < (X > 0 ? X + 2 : 0); ++i) {
                if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
                const uint32_t s = i & 1;
                const int back = i - 2;
                if (back >= 0) {  // the tile of this group before: its P and dS are in TMEM
                    wait(&sm.ds_full[s], (uint32_t)(back >> 1) & 1u);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t so = bst * (kStage >> 4);
#pragma unroll
                        for (int kk = 0; kk < kHalf / 16; ++kk)
                            mma_ts(tmem + tG, tmem + tS + s * kHalf + half_at(kk), gt + so + kk * (2048 >> 4), id_g,
                                   back > 0 || kk > 0);
#pragma unroll
                        for (int kk = 0; kk < kHalf / 16; ++kk)
                            mma_ts(tmem + tG + DT, tmem + tP + s * kHalf + half_at(kk), qt_ + so + kk * (2048 >> 4), id_g,
                                   back > 0 || kk > 0);
                        if (kFine)
#pragma unroll
                            for (int kk = 0; kk < kHalf / 16; ++kk) {
                                mma_ts(tmem + tG, tmem + tS + s * kHalf + half_at(kk) + kRest, gt + so + kk * (2048 >> 4),
                                       id_g, true);
                                mma_ts(tmem + tG + DT, tmem + tP + s * kHalf + half_at(kk) + kRest,
                                       qt_ + so + kk * (2048 >> 4), id_g, true);
                            }
                        mma_commit(&sm.q_empty[bst]);
                    }
                    if (++bst == kRowStages) bst = 0;
                }
                if (i < X) {
                    wait(&sm.q_full[st], ph);
                    const int t0 = (qt.begin + at) * kHalf;
                    if (t0 + kHalf > rows) {
                        zero_rows<DT>(sm.q[st], rows - t0, lane);
                        zero_rows<DT>(sm.go[st], rows - t0, lane);
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t so = st * (kStage >> 4);
#pragma unroll
                        for (int kk = 0; kk < DT / 16; ++kk)
                            mma_ss(tmem + tS + s * kHalf, kd + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                                   qd + so + (((kk >> 2) * kHalfBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
#pragma unroll
                        for (int kk = 0; kk < DT / 16; ++kk)
                            mma_ss(tmem + tP + s * kHalf, vd + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                                   gd + so + (((kk >> 2) * kHalfBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
                        mma_commit(&sm.s_full[s]);
                    }
                    if (++st == kRowStages) st = 0, ph ^= 1u;
                    if (++at == per) at = 0;
                }
            }
            if (elect_one()) {
                mma_commit(&sm.g_full);
                mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
                drain(&sm.drain, 0);
            }
            __syncwarp();
        } else {
            const int s = warp >> 2, r = 32 * (warp & 3) + lane, j = j0 + r;
            const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const uint32_t ts = tl + tS + s * kHalf, tp = tl + tP + s * kHalf;
            const float c = prm.scale * kLog2e;
            const uint64_t c2 = pair(c, c);
            // positions [j, last] see key j
            const int last = j >= n ? -1 : j < prm.sinks ? n - 1 : min(n - 1, j + prm.window - 1);
            bool ok = !aborted(abort_flag);
            for (int i = s; ok && i < X; i += 2) {
                const int st = i % kRowStages, p0 = (qt.begin + (x0 + i) % per) * kHalf + off;
                if (!(ok = wait_w(abort_flag, &sm.q_full[st], (uint32_t)(i / kRowStages) & 1u))) break;  // base, delta
                if (!(ok = wait_w(abort_flag, &sm.s_full[s], (uint32_t)(i >> 1) & 1u))) break;
                tc_fence_after();
                const bool whole = j0 + kRows - 1 <= p0 && p0 + kHalf - 1 < n &&
                                   (p0 + kHalf - 1 - j0 < prm.window || j0 + kRows <= prm.sinks);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t a[32], d[32];
                    tmem_ld32(ts + 32 * g, a);
                    tmem_ld32(tp + 32 * g, d);
                    tmem_ld_wait();
                    const ulonglong2 *bp = reinterpret_cast<const ulonglong2 *>(&sm.base[st][32 * g]);
                    const ulonglong2 *dp = reinterpret_cast<const ulonglong2 *>(&sm.delta[st][32 * g]);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 nb = bp[e / 4], nd = dp[e / 4];
#pragma unroll
                        for (int h = 0; h < 4; h += 2) {
                            float x, y;
                            split(mul2(add2(pair(a[e + h], a[e + h + 1]), h ? nb.y : nb.x), c2), x, y);
                            x = ex2(x);
                            y = ex2(y);
                            a[e + h] = __float_as_uint(x);
                            a[e + h + 1] = __float_as_uint(y);
                            split(mul2(pair(x, y), add2(pair(d[e + h], d[e + h + 1]), h ? nd.y : nd.x)), x, y);
                            d[e + h] = __float_as_uint(x);
                            d[e + h + 1] = __float_as_uint(y);
                        }
                    }
                    if (!whole) {
                        const int lo = max(j - (p0 + 32 * g), 0), hi = min(last - (p0 + 32 * g), 31);
                        const uint32_t bits = hi < lo || lo > 31 ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1u)) a[e] = d[e] = 0u;
                    }
                    store_half<kFine>(ts + 32 * g, a);
                    store_half<kFine>(tp + 32 * g, d);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sm.ds_full[s]);
            }
            if (ok && X > 0) ok = wait_w(abort_flag, &sm.g_full, 0);
            uint8_t *out = s == 0 ? sm.v : sm.k;  // group 0: dv, group 1: dk
            if (ok && shared) {
                // this share's sums: [share][dv, dk][128][DT]
                float *dst = part + ((((size_t)bh * sp.tiles + j0 / kRows) * sp.parts + share) * 2 + s) * (kRows * DT) + r * DT;
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < DT; x += 16) {
                    uint32_t o[16];
                    tmem_ld16(tl + tG + s * DT + x, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(dst + x + e) =
                            X > 0 ? make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_uint4(0u, 0u, 0u, 0u);
                }
            } else if (ok) {
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < DT; x += 16) stage16(out, tl + tG + s * DT, r, x, s == 0 ? 1.f : prm.scale, X > 0);
                fence_proxy_async_smem();
            }
            named_bar_sync(1 + s, 128);
            if (ok && !shared && (warp & 3) == 0 && lane == 0) {
#pragma unroll
                for (int x = 0; x < DT; x += 64) tma_store_3d(s == 0 ? &maps.dv : &maps.dk, out + x / 64 * kBox, x, j0, bh);
                tma_store_commit();
                tma_store_wait_all();
            }
            __syncwarp();
        }
    };
    if (warp == kTmaWarp) {
        if (lane == 0 && X > 0 && !aborted(abort_flag)) {
            mbar_arrive_expect_tx(&sm.kv_full, 2 * kTile);
#pragma unroll
            for (int x = 0; x < DT; x += 64) {
                tma_load_3d(sm.k + x / 64 * kBox, &maps.k, &sm.kv_full, x, j0, bh);
                tma_load_3d(sm.v + x / 64 * kBox, &maps.v, &sm.kv_full, x, j0, bh);
            }
            int loaded = 0;
            for (int i = 0; i < X; ++i) {
                const int st = i % kRowStages, x = x0 + i;
                const int t0 = (qt.begin + x % per) * kHalf, z = b * prm.Hq + hk * group + x / per;
                if (i >= kRowStages && !wait_b(abort_flag, &sm.q_empty[st], (uint32_t)(i / kRowStages - 1) & 1u)) break;
                mbar_arrive_expect_tx(&sm.q_full[st], 2 * kStage + 2 * kHalf * 4);
#pragma unroll
                for (int c = 0; c < DT; c += 64) {
                    tma_load_3d(sm.q[st] + c / 64 * kHalfBox, &maps.q_half, &sm.q_full[st], c, t0, z);
                    tma_load_3d(sm.go[st] + c / 64 * kHalfBox, &maps.go_half, &sm.q_full[st], c, t0, z);
                }
                const float *row = prm.delta + (size_t)z * prm.padded + t0;
                bulk_load(sm.delta[st], row, kHalf * 4, &sm.q_full[st]);
                bulk_load(sm.base[st], row + (size_t)prm.B * prm.Hq * prm.padded, kHalf * 4, &sm.q_full[st]);
                loaded = i + 1;
            }
            drain(&sm.kv_full, 0);  // no copy may still be writing shared memory when the CTA exits
            for (int i = max(loaded - kRowStages, 0); i < loaded; ++i)
                drain(&sm.q_full[i % kRowStages], (uint32_t)(i / kRowStages) & 1u);
        }
        __syncwarp();
    } else if (fine) {
        run(std::true_type{});
    } else {
        run(std::false_type{});
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Both kinds of blocks in one launch, the longer dk, dv ones first: neither waits for the other, and the
// last wave is filled by either (8192 rows, d 128, window 1024: 244 us, 268 as two launches of 130
// and 139 us, each with a last wave of its own).
template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
window_tc_backward(const __grid_constant__ Maps maps, const Params prm, const Split sp, float *part, const int dkv_blocks)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if ((int)blockIdx.x < dkv_blocks)
        dkv_block<DT>(maps, prm, sp, part, (int)blockIdx.x, smem_raw);
    else if (few_keys(prm, (int)blockIdx.x - dkv_blocks))
        dq_block<DT, true>(maps, prm, (int)blockIdx.x - dkv_blocks, smem_raw);
    else
        dq_block<DT, false>(maps, prm, (int)blockIdx.x - dkv_blocks, smem_raw);
}

// -D = -dO . o and -lse / scale of every row, rows of an entry padded to whole tiles with zeros: 16
// lanes a row, 64 rows of one head a CTA.
constexpr int kRowsCta = 64;
__global__ void __launch_bounds__(256) window_tc_rows(const __nv_bfloat16 *o, const __nv_bfloat16 *go, const Params prm)
{
    constexpr int kN = kRowsCta / 16;  // rows a thread
    const int per = prm.padded / kRowsCta, z = (int)blockIdx.x / per, t0 = (int)blockIdx.x % per * kRowsCta + threadIdx.x / 16;
    const int lane = threadIdx.x % 16;
    griddep_wait();
    griddep_launch_dependents();
    const int rows = min(prm.Nq, valid(prm.lens, z / prm.Hq, prm.Nk) - (prm.Nk - prm.Nq));  // of tokens
    uint4 a[kN], b[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
        const int t = t0 + 16 * i;
        if (t < rows && lane * 8 < prm.d) {
            const size_t at = ((size_t)z * prm.Nq + t) * prm.d + lane * 8;
            a[i] = __ldg(reinterpret_cast<const uint4 *>(o + at));
            b[i] = __ldg(reinterpret_cast<const uint4 *>(go + at));
        }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const uint32_t as[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bs[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x = fmaf(__uint_as_float(as[e] << 16), __uint_as_float(bs[e] << 16), x);
            x = fmaf(__uint_as_float(as[e] & 0xffff0000u), __uint_as_float(bs[e] & 0xffff0000u), x);
        }
#pragma unroll
        for (int m = 8; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
        const int t = t0 + 16 * i;
        if (lane == 0) {
            const size_t at = (size_t)z * prm.padded + t;
            prm.delta[at] = -x;
            prm.delta[(size_t)prm.B * prm.Hq * prm.padded + at] =
                t < rows ? -__ldg(prm.lse + (size_t)z * prm.Nq + t) / prm.scale : 0.f;
        }
    }
}

// Scratch: -D and -lse / scale of every row (rows of an entry padded to whole tiles), then the shares.
size_t part_offset(const WindowProblem &p) { return (size_t)p.B * p.Hq * ceil_div(p.Nq, kRows) * kRows * 2 * sizeof(float); }

template <int DT>
la_status backward(const WindowProblem &p)
{
    const Params prm = params_of(p);
    const auto kernel = window_tc_backward<DT>;
    const Split sp = split_of(p);
    const long long dq_ctas = (long long)p.B * p.Hk * prm.units;
    const long long dkv_ctas = (long long)p.B * p.Hk * (ceil_div(p.Nk, kRows) + sp.tiles * (sp.parts - 1LL));
    const long long sum_ctas = (long long)split_floats(p, sp, DT) / std::max(sp.parts, 1) / 4 / 256;
    const long long row_ctas = (long long)p.B * p.Hq * (prm.padded / kRowsCta);
    if (dq_ctas + dkv_ctas > 0x7fffffffLL || sum_ctas > 0x7fffffffLL || row_ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    float *part = reinterpret_cast<float *>(reinterpret_cast<char *>(p.delta) + part_offset(p));
    const int bq = p.B * p.Hq, bk = p.B * p.Hk;
    Maps m;
    la_status st = make_map(&m.q, p.q, bq, p.Nq, p.d);
    if (st == LA_OK) st = make_map(&m.go, p.dout, bq, p.Nq, p.d);
    if (st == LA_OK) st = make_map(&m.k, p.k, bk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&m.v, p.v, bk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&m.q_half, p.q, bq, p.Nq, p.d, kHalf);
    if (st == LA_OK) st = make_map(&m.go_half, p.dout, bq, p.Nq, p.d, kHalf);
    if (st == LA_OK) st = make_map(&m.k_half, p.k, bk, p.Nk, p.d, kHalf);
    if (st == LA_OK) st = make_map(&m.v_half, p.v, bk, p.Nk, p.d, kHalf);
    if (st == LA_OK) st = make_map(&m.dq, p.dq, bq, p.Nq, p.d);
    if (st == LA_OK) st = make_map(&m.dk, p.dk, bk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&m.dv, p.dv, bk, p.Nk, p.d);
    constexpr int smem = (int)std::max(sizeof(DqSmem<DT>), sizeof(DkvSmem<DT>));
    if (st == LA_OK) st = ensure_smem((const void *)kernel, smem);
    if (st != LA_OK) return st;
    g_launched = true;
    count_launches(sp.parts > 1 ? 3 : 2);
    st = launch_dependent(window_tc_rows, (unsigned)row_ctas, 256, 0, p.stream, static_cast<const __nv_bfloat16 *>(p.o),
                          static_cast<const __nv_bfloat16 *>(p.dout), prm);
    if (st == LA_OK)
        st = launch_dependent(kernel, (unsigned)(dq_ctas + dkv_ctas), kThreads, smem, p.stream, m, prm, sp, part,
                              (int)dkv_ctas);
    if (st != LA_OK || sp.parts == 1) return st;
    return launch_dependent(window_tc_sum<DT>, (unsigned)sum_ctas, 256, 0, p.stream, (const float *)part,
                            static_cast<__nv_bfloat16 *>(p.dk), static_cast<__nv_bfloat16 *>(p.dv), sp, p.Nk, p.d, p.scale);
}

}  // namespace

size_t window_backward_tc_scratch(const WindowProblem &p)
{
    return part_offset(p) + split_floats(p, split_of(p), p.d <= 64 ? 64 : 128) * 4;
}

la_status window_backward_tc(const WindowProblem &p)
{
    return p.d <= 64 ? backward<64>(p) : backward<128>(p);
}

la_status tc_window_bwd_read_status(cudaStream_t s, unsigned *bits)
{
    return read_status(g_launched, g_winb_status, s, bits);
}

}  // namespace la
