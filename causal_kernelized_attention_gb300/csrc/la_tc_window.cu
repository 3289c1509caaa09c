// Window attention forward on the tensor cores: bf16 q, k, v, any length, d <= 128 on tiles
// of 64 or 128 columns (narrower heads zero-filled by TMA); two kernels, the second further
// down for narrow heads.  The mathematics is la_window.cu's:
// one pass over the key tiles with the running maximum and sum of the softmax.
//
// A CTA takes two query tiles of 128 rows -- the same rows of two heads that share a key
// head, or neighbouring rows of one head -- so each K and V tile brought into shared memory
// feeds two of each product (for short windows one tile: see the dispatch).  TMEM holds S_s
// (128 columns each) and O_s (one per query tile s); the weights P_s, rounded to bf16, are
// written over S_s and read from there by the second product.  Warps 0-3 and 4-7 are the softmax groups of the two tiles (a thread
// owns a row, no shuffles), warp 8 loads by TMA, warp 9 issues the MMAs:
//
//   MMA:      S0(0) S1(0) | PV0(0) S0(1) | PV1(0) S1(1) | PV0(1) S0(2) | ...
//   group 0:         softmax(0)        ---         softmax(1) ...
//   group 1:               softmax(0)        ---         softmax(1) ...
//
// so one tile's softmax runs under the other's products.  The output is rescaled only when
// a row's maximum has grown by more than 8 (log2 units): until then the weights are at most
// 2^8 above the usual, which neither fp32 sums nor bf16's relative rounding notice, and the
// read-modify-write of O leaves the loop.  Tiles that every row sees skip the mask.
//
// The weights' rounding to bf16 (2^-8 relative at most, each on its own) enters the output like the
// rounding of the output itself: the error is 1.3 to 1.4 times that of the latter alone (two-part weights, as the
// decode step has them, would be half as many products again); sums, maxima and the accumulator are fp32.
#include "la_tc_window.cuh"

namespace la {
namespace {

using namespace window;

static __device__ unsigned g_win_status;
std::atomic<bool> g_launched{false};

constexpr int kT = kRows;  // rows and keys of a tile
constexpr float kGrow = 8.f;  // log2 units a maximum may grow before the output is rescaled

// QT query tiles a CTA: two, one CTA an SM, or one, two CTAs an SM.
template <int DT, int QT>
struct Smem {
    static constexpr uint32_t kTile = kT * DT * 2;
    // V(u) is used one step after K(u)
    static constexpr int kKStages = QT == 1 && DT == 128 ? 1 : 2, kVStages = QT == 1 && DT == 128 ? 1 : 3;
    uint8_t q[QT][kTile];  // then the outputs, staged
    uint8_t k[kKStages][kTile];
    uint8_t v[kVStages][kTile];
    uint64_t q_full[QT], s_full[QT], p_full[QT], o_full[QT];
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], drain;
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ bool wait_b(int *abort_flag, uint64_t *bar, uint32_t parity)
{
    return wait_bar(&g_win_status, abort_flag, bar, parity);
}
__device__ __forceinline__ bool wait_w(int *abort_flag, uint64_t *bar, uint32_t parity)
{
    return wait_bar_warp(&g_win_status, abort_flag, bar, parity);
}
// A row's kN scores from TMEM, -inf where the row does not see the key.
template <int kN>
__device__ __forceinline__ void load_scores(uint32_t ts, uint32_t (&a)[kN], bool whole, int p, int j0, const Params &prm, int n)
{
#pragma unroll
    for (int g = 0; g < kN / 32; ++g) tmem_ld32(ts + 32 * g, reinterpret_cast<uint32_t(&)[32]>(a[32 * g]));
    tmem_ld_wait();
    if (!whole) {
#pragma unroll
        for (int g = 0; g < kN / 32; ++g) {
            const uint32_t bits = seen_bits(p, j0 + 32 * g, prm.window, prm.sinks, n);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) a[32 * g + e] = 0xff800000u;
        }
    }
}

template <int kN>
__device__ __forceinline__ float row_max(const uint32_t (&a)[kN])
{
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < kN / 2; ++e) mx[e & 3] = max3(mx[e & 3], __uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
    return max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
}

// exp2((s - m) c) of a row's kN scores, rounded to bf16 into a[0 .. kN / 2 - 1], with the scores'
// maximum and the weights' sum (two halves).
template <int kN>
__device__ __forceinline__ void weights(uint32_t (&a)[kN], float c, float m, float &top, uint64_t &sum)
{
    float base = m == -INFINITY ? 0.f : -m * c, past = 0.f;
    const bool huge = __any_sync(0xffffffffu, fabsf(m) * c > 0x1p100f && m != -INFINITY);
    if (huge) {  // m c may overflow: subtract first
        past = row_max(a);
        const float z = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int e = 0; e < kN; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) - z);
        base = 0.f;
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    const uint64_t c2 = pair(c, c), base2 = pair(base, base);
    uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int e = 0; e < kN / 2; ++e) {
        const uint32_t s0 = a[2 * e], s1 = a[2 * e + 1];
        mx[e & 3] = max3(mx[e & 3], __uint_as_float(s0), __uint_as_float(s1));
        float x, y;
        split(fma2(pair(s0, s1), c2, base2), x, y);
        x = ex2(x);
        y = ex2(y);
        sums[e & 3] = add2(sums[e & 3], pair(x, y));
        a[e] = pack_bf16(x, y);
    }
    top = huge ? past : max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
    sum = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
}

template <int DT, int QT>
__global__ void __launch_bounds__(32 * (4 * QT + 2), 3 - QT)
window_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const Params prm)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    typedef Smem<DT, QT> Sm;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    constexpr uint32_t kTile = Sm::kTile;
    constexpr int kKStages = Sm::kKStages, kVStages = Sm::kVStages, kTmaWarp = 4 * QT, kMmaWarp = kTmaWarp + 1;
    constexpr uint32_t tS = 0, tO = QT * 128, kTmemCols = QT * 256;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < QT; ++s) {
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.p_full[s], 128);
            mbar_init(&sm.o_full[s], 1);
        }
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = (smem_u32(smem_raw) & 1023u) == 0 ? 0 : 1;
        if (sm.abort) atomicOr(&g_win_status, kStatusTimeout);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
        tma_prefetch_map(&map_o);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    int *abort_flag = &sm.abort;
    const Work<kT> w(prm, (int)blockIdx.x);
    const int U = w.count();

    if (warp == kTmaWarp) {
        if (lane == 0 && !aborted(abort_flag)) {
            const int kz = w.b * prm.Hk + w.hk;
            int loaded = 0;
            for (int u = 0; u < U; ++u) {
                const int ks = u % kKStages, vs = u % kVStages, j0 = w.tile(u) * kT;
                if (u >= kKStages && !wait_b(abort_flag, &sm.k_empty[ks], (uint32_t)(u / kKStages - 1) & 1u)) break;
                mbar_arrive_expect_tx(&sm.k_full[ks], kTile);
#pragma unroll
                for (int x = 0; x < DT; x += 64) tma_load_3d(sm.k[ks] + x / 64 * kBox, &map_k, &sm.k_full[ks], x, j0, kz);
                if (u == 0)
#pragma unroll
                    for (int s = 0; s < QT; ++s)
                        if (w.kt[s].count() > 0) {
                            mbar_arrive_expect_tx(&sm.q_full[s], kTile);
#pragma unroll
                            for (int x = 0; x < DT; x += 64)
                                tma_load_3d(sm.q[s] + x / 64 * kBox, &map_q, &sm.q_full[s], x, w.t0[s], w.b * prm.Hq + w.h[s]);
                        }
                loaded = u + 1;
                if (u >= kVStages && !wait_b(abort_flag, &sm.v_empty[vs], (uint32_t)(u / kVStages - 1) & 1u)) {
                    mbar_arrive_expect_tx(&sm.v_full[vs], 0);  // completes the phase that drain() waits for
                    break;
                }
                mbar_arrive_expect_tx(&sm.v_full[vs], kTile);
#pragma unroll
                for (int x = 0; x < DT; x += 64) tma_load_3d(sm.v[vs] + x / 64 * kBox, &map_v, &sm.v_full[vs], x, j0, kz);
            }
            // no copy may still be writing shared memory when the CTA exits
            if (loaded > 0)
#pragma unroll
                for (int s = 0; s < QT; ++s)
                    if (w.kt[s].count() > 0) drain(&sm.q_full[s], 0);
            for (int u = max(loaded - kKStages, 0); u < loaded; ++u)
                drain(&sm.k_full[u % kKStages], (uint32_t)(u / kKStages) & 1u);
            for (int u = max(loaded - kVStages, 0); u < loaded; ++u)
                drain(&sm.v_full[u % kVStages], (uint32_t)(u / kVStages) & 1u);
        }
    } else if (warp == kMmaWarp) {
        const uint32_t id_s = idesc_bf16_f32(128, kT, false, false), id_o = idesc_bf16_f32(128, DT, false, true);
        const uint64_t dq[2] = {kmajor(smem_u32(sm.q[0]), 0), kmajor(smem_u32(sm.q[QT - 1]), 0)};
        const uint64_t dk = kmajor(smem_u32(sm.k[0]), 0), dv = mnmajor(smem_u32(sm.v[0]), 0, kBox);
        uint32_t kst = 0, kph = 0, vst = 0, vph = 0;  // stages and phases of K(u) and V(u - 1)
        uint32_t fed[2] = {0, 0};                     // products of P_s issued
        bool pending[2] = {false, false};
        auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(&g_win_status, abort_flag, bar, parity); };
        for (int u = 0; u <= U; ++u) {
            if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
            const int tile = u < U ? w.tile(u) : 0;
            if (u > 0) {
                wait(&sm.v_full[vst], vph);
                // values of padding (in the last tile only): their weights are 0, but 0 times a
                // NaN is not
                if (u == U && w.tile(u - 1) * kT + kT > w.n) {
                    const int r0 = w.n - w.tile(u - 1) * kT;
                    for (int e = lane; e < (kT - r0) * (DT / 8); e += 32) {
                        const int row = r0 + e / (DT / 8), ch = e % (DT / 8);
                        *reinterpret_cast<uint4 *>(sm.v[vst] + (ch >> 3) * kBox + row * 128 + (ch & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
#pragma unroll
            for (int s = 0; s < QT; ++s) {
                if (pending[s]) {
                    wait(&sm.p_full[s], fed[s] & 1u);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t d = dv + vst * (kTile >> 4);
#pragma unroll
                        for (int kk = 0; kk < kT / 16; ++kk)
                            mma_ts(tmem + tO + s * DT, tmem + tS + s * kT + kk * 8, d + kk * (2048 >> 4), id_o,
                                   fed[s] > 0 || kk > 0);
                        mma_commit(&sm.o_full[s]);
                    }
                    ++fed[s];
                    pending[s] = false;
                }
                if (s == QT - 1 && u > 0 && elect_one()) mma_commit(&sm.v_empty[vst]);
                if (u < U) {
                    if (s == 0) wait(&sm.k_full[kst], kph);
                    if (w.reaches(s, tile)) {
                        if (fed[s] == 0) wait(&sm.q_full[s], 0);
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t d = dk + kst * (kTile >> 4);
#pragma unroll
                            for (int kk = 0; kk < DT / 16; ++kk) {
                                const uint64_t o = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
                                mma_ss(tmem + tS + s * kT, dq[s] + o, d + o, id_s, kk > 0);
                            }
                            mma_commit(&sm.s_full[s]);
                        }
                        pending[s] = true;
                    }
                    if (s == QT - 1 && elect_one()) mma_commit(&sm.k_empty[kst]);
                }
            }
            if (u > 0 && ++vst == kVStages) vst = 0, vph ^= 1u;
            if (++kst == kKStages) kst = 0, kph ^= 1u;
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
            drain(&sm.drain, 0);
        }
        __syncwarp();
    } else {
        const int s = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + tS + s * kT, to = tl + tO + s * DT;
        const KeyTiles kt = s ? w.kt[1] : w.kt[0];
        const int t0 = s ? w.t0[1] : w.t0[0], z = w.b * prm.Hq + (s ? w.h[1] : w.h[0]);
        const int t = t0 + r, p = t + w.off, p_first = t0 + w.off, tiles = kt.count();
        const float c = prm.scale * kLog2e;
        float m = -INFINITY, l = 0.f;
        bool ok = !aborted(abort_flag);
        int done = 0;
        for (; ok && done < tiles; ++done) {
            const int j0 = kt.tile(done) * kT;
            if (!(ok = wait_w(abort_flag, &sm.s_full[s], (uint32_t)done & 1u))) break;
            tc_fence_after();
            const bool whole = j0 + kT - 1 <= p_first && p_first + kT - 1 < w.n &&
                               (p_first + kT - 1 - j0 < prm.window || j0 + kT <= prm.sinks);
            // The weights against the maximum so far, found together with the tile's own maximum:
            // unless that is more than kGrow above they stand, else the scores are taken again.
            uint32_t a[128];
            uint64_t sum;
            bool again;
            do {  // (a row's first visible tile sets its maximum ahead: it has no output to rescale)
                load_scores(ts, a, whole, p, j0, prm, w.n);
                if (__any_sync(0xffffffffu, m == -INFINITY)) {
                    const float first = row_max(a);
                    if (m == -INFINITY) m = first;
                }
                float top;
                weights(a, c, m, top, sum);
                const bool grow = top > m && (top - m) * c > kGrow;
                again = __any_sync(0xffffffffu, grow);
                if (again) {
                    const float keep = grow ? ex2((m - top) * c) : 1.f;
                    if (grow) m = top;
                    l *= keep;
                    if (done > 0) {
                        if (!(ok = wait_w(abort_flag, &sm.o_full[s], (uint32_t)(done - 1) & 1u))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < DT; x += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + x, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                            tmem_st16(to + x, o);
                        }
                    }
                }
            } while (again);
            if (!ok) break;
            float lx, ly;
            split(sum, lx, ly);
            l += lx + ly;
#pragma unroll
            for (int g = 0; g < 4; ++g) tmem_st16(ts + 16 * g, reinterpret_cast<const uint32_t(&)[16]>(a[16 * g]));
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.p_full[s]);
        }
        if (ok && done > 0) ok = wait_w(abort_flag, &sm.o_full[s], (uint32_t)(done - 1) & 1u);
        if (ok && t0 < prm.Nq) {
            tc_fence_after();
            // padding gives zeros whatever TMEM holds, a row of no finite score 0 / 0
            const bool some = p < w.n;
            const float inv = 1.f / l;
#pragma unroll
            for (int x = 0; x < DT; x += 16) {
                uint32_t o[16];
                if (done > 0) {
                    tmem_ld16(to + x, o);
                    tmem_ld_wait();
                }
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    pk[e] = some ? pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv) : 0u;
                uint8_t *row = sm.q[s] + x / 64 * kBox + r * 128;
                const int ch = (x & 63) >> 3;
                *reinterpret_cast<uint4 *>(row + (((ch) ^ (r & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                *reinterpret_cast<uint4 *>(row + (((ch + 1) ^ (r & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            }
            if (t < prm.Nq)
                prm.lse[(size_t)z * prm.Nq + t] =
                    some ? (m == -INFINITY ? 0.f : m) * prm.scale + __log2f(l) * kLn2 : -INFINITY;
            fence_proxy_async_smem();
        }
        named_bar_sync(1 + s, 128);
        if (ok && t0 < prm.Nq && (warp & 3) == 0 && lane == 0) {
#pragma unroll
            for (int x = 0; x < DT; x += 64)
                tma_store_3d(&map_o, sm.q[s] + x / 64 * kBox, x, t0, z);
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

// ---------------------------------------------------------------- narrow heads
// For heads of at most 64: one query tile and key tiles of 64, 128 TMEM columns (S, then P, at 0, O at 64), 48 KB of shared
// memory and five warps, so that four CTAs share an SM and the products, softmax chains, starts and
// ends of each run under the others'; a batch of a few hundred tiles is one wave.  Warp 4 issues both the copies and the MMAs: when the softmax group has given
// up P(u - 1), S(u - 1) and with it P V(u - 2) are complete (products complete in order), so
// their stages are free without barriers of their own.
constexpr int kSmallKeys = 64;
constexpr uint32_t kSmallBox = kSmallKeys * 128;

struct SmallSmem {
    uint8_t q[kT * 128];  // then the output, staged
    uint8_t k[2][kSmallBox];
    uint8_t v[2][kSmallBox];
    uint64_t q_full, s_full, p_full, o_full, k_full[2], v_full[2], drain;
    uint32_t tmem_base;
    int abort;
};

__global__ void __launch_bounds__(160, 4)
window_tc_small_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const Params prm)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    SmallSmem &sm = *reinterpret_cast<SmallSmem *>(smem_raw);
    constexpr uint32_t tS = 0, tO = 64;
    constexpr int KT = kSmallKeys;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    if (tid == 0) {
        uint64_t *bars[] = {&sm.q_full, &sm.s_full, &sm.o_full, &sm.k_full[0], &sm.k_full[1], &sm.v_full[0], &sm.v_full[1], &sm.drain};
        for (uint64_t *b : bars) mbar_init(b, 1);
        mbar_init(&sm.p_full, 128);
        sm.abort = (smem_u32(smem_raw) & 1023u) == 0 ? 0 : 1;
        if (sm.abort) atomicOr(&g_win_status, kStatusTimeout);
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(&sm.tmem_base, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    int *abort_flag = &sm.abort;
    const Work<KT> w(prm, (int)blockIdx.x);
    const int U = w.kt[0].count();

    if (warp == 4) {
        const uint32_t id_s = idesc_bf16_f32(128, KT, false, false), id_o = idesc_bf16_f32(128, 64, false, true);
        const uint64_t dq = kmajor(smem_u32(sm.q), 0), dk = kmajor(smem_u32(sm.k[0]), 0), dv = mnmajor(smem_u32(sm.v[0]), 0, 0);
        const int kz = w.b * prm.Hk + w.hk;
        auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(&g_win_status, abort_flag, bar, parity); };
        auto load = [&](uint8_t (*dst)[kSmallBox], uint64_t *bars, const CUtensorMap *map, int u) {
            if (u < U && elect_one()) {
                mbar_arrive_expect_tx(&bars[u & 1], kSmallBox);
                tma_load_3d(dst[u & 1], map, &bars[u & 1], 0, w.kt[0].tile(u) * KT, kz);
            }
        };
        int loaded = 0;  // tiles whose K has been asked for
        if (U > 0 && !__any_sync(0xffffffffu, aborted(abort_flag))) {
            load(sm.k, sm.k_full, &map_k, 0);
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.q_full, sizeof(sm.q));
                tma_load_3d(sm.q, &map_q, &sm.q_full, 0, w.t0[0], w.b * prm.Hq + w.h[0]);
            }
            load(sm.v, sm.v_full, &map_v, 0);
            load(sm.k, sm.k_full, &map_k, 1);
            load(sm.v, sm.v_full, &map_v, 1);
            loaded = min(U, 2);
            wait(&sm.q_full, 0);
            for (int u = 0; u <= U; ++u) {
                if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
                if (u > 0) {
                    const int x = u - 1;
                    wait(&sm.p_full, (uint32_t)x & 1u);
                    wait(&sm.v_full[x & 1], (uint32_t)(x >> 1) & 1u);
                    if (u == U && w.kt[0].tile(x) * KT + KT > w.n) {  // values of padding
                        const int r0 = w.n - w.kt[0].tile(x) * KT;
                        for (int e = lane; e < (KT - r0) * 8; e += 32)
                            *reinterpret_cast<uint4 *>(sm.v[x & 1] + (r0 + e / 8) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t d = dv + (x & 1) * (kSmallBox >> 4);
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            mma_ts(tmem + tO, tmem + tS + kk * 8, d + kk * (2048 >> 4), id_o, x > 0 || kk > 0);
                        mma_commit(&sm.o_full);
                    }
                    // S(x) and P V(x - 1) are complete: K(x + 2) over K(x), V(x + 1) over V(x - 1)
                    load(sm.k, sm.k_full, &map_k, x + 2);
                    if (x > 0) load(sm.v, sm.v_full, &map_v, x + 1);
                    loaded = max(loaded, min(U, x + 3));
                }
                if (u < U) {
                    wait(&sm.k_full[u & 1], (uint32_t)(u >> 1) & 1u);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t d = dk + (u & 1) * (kSmallBox >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) mma_ss(tmem + tS, dq + kk * 2, d + kk * 2, id_s, kk > 0);
                        mma_commit(&sm.s_full);
                    }
                }
            }
        }
        if (elect_one()) {
            mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
            drain(&sm.drain, 0);
            if (loaded > 0 && aborted(abort_flag)) {  // no copy may still be writing shared memory
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < kDrainNs) {
                }
            }
        }
        __syncwarp();
    } else {
        const int r = 32 * warp + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16), ts = tl + tS, to = tl + tO;
        const KeyTiles kt = w.kt[0];
        const int t0 = w.t0[0], z = w.b * prm.Hq + w.h[0], t = t0 + r, p = t + w.off, p_first = t0 + w.off;
        const float c = prm.scale * kLog2e;
        float m = -INFINITY, l = 0.f;
        bool ok = !aborted(abort_flag);
        int done = 0;
        for (; ok && done < U; ++done) {
            const int j0 = kt.tile(done) * KT;
            if (!(ok = wait_w(abort_flag, &sm.s_full, (uint32_t)done & 1u))) break;
            tc_fence_after();
            const bool whole = j0 + KT - 1 <= p_first && p_first + kT - 1 < w.n &&
                               (p_first + kT - 1 - j0 < prm.window || j0 + KT <= prm.sinks);
            uint32_t a[KT];
            uint64_t sum;
            bool again;
            do {  // as in the larger kernel
                load_scores(ts, a, whole, p, j0, prm, w.n);
                if (__any_sync(0xffffffffu, m == -INFINITY)) {
                    const float first = row_max(a);
                    if (m == -INFINITY) m = first;
                }
                float top;
                weights(a, c, m, top, sum);
                const bool grow = top > m && (top - m) * c > kGrow;
                again = __any_sync(0xffffffffu, grow);
                if (again) {
                    const float keep = grow ? ex2((m - top) * c) : 1.f;
                    if (grow) m = top;
                    l *= keep;
                    if (done > 0) {
                        if (!(ok = wait_w(abort_flag, &sm.o_full, (uint32_t)(done - 1) & 1u))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < 64; x += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + x, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                            tmem_st16(to + x, o);
                        }
                    }
                }
            } while (again);
            if (!ok) break;
            float lx, ly;
            split(sum, lx, ly);
            l += lx + ly;
#pragma unroll
            for (int g = 0; g < KT / 32; ++g) tmem_st16(ts + 16 * g, reinterpret_cast<const uint32_t(&)[16]>(a[16 * g]));
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.p_full);
        }
        if (ok && done > 0) ok = wait_w(abort_flag, &sm.o_full, (uint32_t)(done - 1) & 1u);
        if (ok) {
            tc_fence_after();
            const bool some = p < w.n;
            const float inv = 1.f / l;
#pragma unroll
            for (int x = 0; x < 64; x += 16) {
                uint32_t o[16];
                if (done > 0) {
                    tmem_ld16(to + x, o);
                    tmem_ld_wait();
                }
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    pk[e] = some ? pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv) : 0u;
                uint8_t *row = sm.q + r * 128;
                const int ch = x >> 3;
                *reinterpret_cast<uint4 *>(row + ((ch ^ (r & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                *reinterpret_cast<uint4 *>(row + (((ch + 1) ^ (r & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            }
            if (t < prm.Nq)
                prm.lse[(size_t)z * prm.Nq + t] =
                    some ? (m == -INFINITY ? 0.f : m) * prm.scale + __log2f(l) * kLn2 : -INFINITY;
            fence_proxy_async_smem();
        }
        named_bar_sync(1, 128);
        if (ok && warp == 0 && lane == 0) {
            tma_store_3d(&map_o, sm.q, 0, t0, z);
            tma_store_commit();
            tma_store_wait_all();
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, 128);
}

la_status forward_small(const WindowProblem &p)
{
    const Params prm = params_of(p, true);
    const long long ctas = (long long)p.B * p.Hk * prm.units;
    if (ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    CUtensorMap mq, mk, mv, mo;
    la_status st = make_map(&mq, p.q, p.B * p.Hq, p.Nq, p.d);
    if (st == LA_OK) st = make_map(&mk, p.k, p.B * p.Hk, p.Nk, p.d, kSmallKeys);
    if (st == LA_OK) st = make_map(&mv, p.v, p.B * p.Hk, p.Nk, p.d, kSmallKeys);
    if (st == LA_OK) st = make_map(&mo, p.out, p.B * p.Hq, p.Nq, p.d);
    if (st == LA_OK) st = ensure_smem((const void *)window_tc_small_kernel, (int)sizeof(SmallSmem));
    if (st != LA_OK) return st;
    g_launched = true;
    count_launches();
    return launch_dependent(window_tc_small_kernel, (unsigned)ctas, 160, (int)sizeof(SmallSmem), p.stream, mq, mk, mv, mo, prm);
}

template <int DT, int QT>
la_status forward(const WindowProblem &p)
{
    typedef Smem<DT, QT> Sm;
    const Params prm = params_of(p, QT == 1);
    const long long ctas = (long long)p.B * p.Hk * prm.units;
    if (ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    CUtensorMap mq, mk, mv, mo;
    la_status st = make_map(&mq, p.q, p.B * p.Hq, p.Nq, p.d);
    if (st == LA_OK) st = make_map(&mk, p.k, p.B * p.Hk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&mv, p.v, p.B * p.Hk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&mo, p.out, p.B * p.Hq, p.Nq, p.d);
    if (st == LA_OK) st = ensure_smem((const void *)window_tc_kernel<DT, QT>, (int)sizeof(Sm));
    if (st != LA_OK) return st;
    g_launched = true;
    count_launches();
    return launch_dependent(window_tc_kernel<DT, QT>, (unsigned)ctas, 32 * (4 * QT + 2), (int)sizeof(Sm), p.stream, mq, mk, mv, mo,
                            prm);
}

}  // namespace

// Heads of 64 and less: the small kernel (8 heads, window 512: 4 x 2048 rows 19.1 us, against 23.9
// with one query tile a CTA and key tiles of 128, 25.1 with two; 65536 rows, 16 heads, window 2048:
// 580 / 749 / 690), unless its CTAs do not even fill the SMs once, where what counts is the length of
// one CTA's chain and key tiles of 128 make fewer steps (1 x 2048 rows: 10.7 against 12.1 us).
//
// Heads of 128: two query tiles a CTA, but for short windows, where a CTA's start and end weigh more
// than the second use of each K and V tile, one, with two CTAs an SM (8 heads: window 128 19.3
// against 22.0 us, 512 28.9 / 29.5; from a window of 1024 two tiles are faster: 1 x 8192 rows 72
// against 79 us, 65536 rows, window 2048: 790 / 892).
la_status window_forward_tc(const WindowProblem &p)
{
    if (p.d <= 64)
        return (long long)p.B * p.Hq * ceil_div(p.Nq, kRows) > sm_count() ? forward_small(p) : forward<64, 1>(p);
    return (long long)p.window + p.sinks <= 640 ? forward<128, 1>(p) : forward<128, 2>(p);
}

la_status tc_window_read_status(cudaStream_t s, unsigned *bits)
{
    return read_status(g_launched, g_win_status, s, bits);
}

}  // namespace la
