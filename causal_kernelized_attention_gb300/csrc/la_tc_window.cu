// Window attention forward on the tensor cores: bf16 q, k, v, any length, d <= 128 on tiles
// of 64 or 128 columns (narrower heads zero-filled by TMA).  The mathematics is la_window.cu's:
// one pass over the key tiles with the running maximum and sum of the softmax.
//
// A CTA takes two query tiles of 128 rows -- the same rows of two heads that share a key
// head, or neighbouring rows of one head -- so each K and V tile brought into shared memory
// feeds two of each product.  TMEM holds S_s (128 columns each) and O_s (one per query
// tile s); the weights P_s, rounded to bf16, are written over S_s and read from there by
// the second product.  Warps 0-3 and 4-7 are the softmax groups of the two tiles (a thread
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
// The weights' rounding to bf16 (2^-9 relative each, independent) enters the output like the
// rounding of the output itself; sums, maxima and the accumulator are fp32.
#include "la_tc_window.cuh"

namespace la {
namespace {

using namespace window;

static __device__ unsigned g_win_status;

constexpr int kT = kRows;  // rows and keys of a tile
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kStages = 2;
constexpr uint32_t kTmemCols = 512;
constexpr float kGrow = 8.f;  // log2 units a maximum may grow before the output is rescaled

template <int DT>
struct Smem {
    static constexpr uint32_t kTile = kT * DT * 2;
    uint8_t q[2][kTile];  // then the outputs, staged
    uint8_t k[kStages][kTile];
    uint8_t v[kStages][kTile];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], drain;
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
template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
window_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const Params prm)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<DT> &sm = *reinterpret_cast<Smem<DT> *>(smem_raw);
    constexpr uint32_t kTile = Smem<DT>::kTile;
    constexpr uint32_t tS = 0, tO = 256;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.p_full[s], 128);
            mbar_init(&sm.o_full[s], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
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
                const int st = u % kStages, j0 = w.tile(u) * kT;
                const uint32_t ph = (uint32_t)(u / kStages - 1) & 1u;
                if (u >= kStages && !wait_b(abort_flag, &sm.k_empty[st], ph)) break;
                mbar_arrive_expect_tx(&sm.k_full[st], kTile);
#pragma unroll
                for (int x = 0; x < DT; x += 64) tma_load_3d(sm.k[st] + x / 64 * kBox, &map_k, &sm.k_full[st], x, j0, kz);
                if (u == 0)
                    for (int s = 0; s < 2; ++s)
                        if (w.kt[s].count() > 0) {
                            mbar_arrive_expect_tx(&sm.q_full[s], kTile);
#pragma unroll
                            for (int x = 0; x < DT; x += 64)
                                tma_load_3d(sm.q[s] + x / 64 * kBox, &map_q, &sm.q_full[s], x, w.t0[s], w.b * prm.Hq + w.h[s]);
                        }
                loaded = u + 1;
                if (u >= kStages && !wait_b(abort_flag, &sm.v_empty[st], ph)) {
                    mbar_arrive_expect_tx(&sm.v_full[st], 0);  // completes the phase that drain() waits for
                    break;
                }
                mbar_arrive_expect_tx(&sm.v_full[st], kTile);
#pragma unroll
                for (int x = 0; x < DT; x += 64) tma_load_3d(sm.v[st] + x / 64 * kBox, &map_v, &sm.v_full[st], x, j0, kz);
            }
            // no copy may still be writing shared memory when the CTA exits
            if (loaded > 0)
                for (int s = 0; s < 2; ++s)
                    if (w.kt[s].count() > 0) drain(&sm.q_full[s], 0);
            for (int u = max(loaded - kStages, 0); u < loaded; ++u) {
                drain(&sm.k_full[u % kStages], (uint32_t)(u / kStages) & 1u);
                drain(&sm.v_full[u % kStages], (uint32_t)(u / kStages) & 1u);
            }
        }
    } else if (warp == kMmaWarp) {
        const uint32_t id_s = idesc_bf16_f32(128, kT, false, false), id_o = idesc_bf16_f32(128, DT, false, true);
        int pvs[2] = {0, 0};
        bool pending[2] = {false, false}, ok = !aborted(abort_flag);
        for (int u = 0; ok && u <= U; ++u) {
            const int st = u % kStages, pst = (u + kStages - 1) % kStages;
            const uint32_t ph = (uint32_t)(u / kStages) & 1u, pph = (uint32_t)((u - 1) / kStages) & 1u;
            if (u > 0) {
                if (!(ok = wait_w(abort_flag, &sm.v_full[pst], pph))) break;
                // values of padding: their weights are 0, but 0 times a NaN is not
                const int j0 = w.tile(u - 1) * kT;
                if (j0 + kT > w.n) {
                    const int r0 = w.n - j0;
                    for (int e = lane; e < (kT - r0) * (DT / 8); e += 32) {
                        const int row = r0 + e / (DT / 8), ch = e % (DT / 8);
                        *reinterpret_cast<uint4 *>(sm.v[pst] + (ch >> 3) * kBox + row * 128 + (ch & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (u < U && !(ok = wait_w(abort_flag, &sm.k_full[st], ph))) break;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (pending[s]) {
                    if (!(ok = wait_w(abort_flag, &sm.p_full[s], (uint32_t)pvs[s] & 1u))) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t va = smem_u32(sm.v[pst]);
#pragma unroll
                        for (int kk = 0; kk < kT / 16; ++kk)
                            mma_ts(tmem + tO + s * DT, tmem + tS + s * kT + kk * 8, mnmajor(va, kk, kBox), id_o,
                                   pvs[s] > 0 || kk > 0);
                        mma_commit(&sm.o_full[s]);
                    }
                    ++pvs[s];
                    pending[s] = false;
                }
                if (u < U && w.reaches(s, w.tile(u))) {
                    if (pvs[s] == 0 && !(ok = wait_w(abort_flag, &sm.q_full[s], 0))) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t qa = smem_u32(sm.q[s]), ka = smem_u32(sm.k[st]);
#pragma unroll
                        for (int kk = 0; kk < DT / 16; ++kk)
                            mma_ss(tmem + tS + s * kT, kmajor(qa, kk), kmajor(ka, kk), id_s, kk > 0);
                        mma_commit(&sm.s_full[s]);
                    }
                    pending[s] = true;
                }
            }
            if (ok && lane == 0) {
                if (u < U) mma_commit(&sm.k_empty[st]);
                if (u > 0) mma_commit(&sm.v_empty[pst]);
            }
            __syncwarp();
        }
        if (lane == 0) {
            mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
            drain(&sm.drain, 0);
        }
        __syncwarp();
    } else {
        const int s = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + tS + s * kT, to = tl + tO + s * DT;
        const int t = w.t0[s] + r, p = t + w.off, p_first = w.t0[s] + w.off;
        const float c = prm.scale * kLog2e;
        float m = -INFINITY, l = 0.f;
        int done = 0;
        bool ok = !aborted(abort_flag);
        for (int u = 0; ok && u < U; ++u) {
            const int tile = w.tile(u), j0 = tile * kT;
            if (!w.reaches(s, tile)) continue;
            if (!(ok = wait_w(abort_flag, &sm.s_full[s], (uint32_t)done & 1u))) break;
            tc_fence_after();
            uint32_t a[4][32];
#pragma unroll
            for (int g = 0; g < 4; ++g) tmem_ld32(ts + 32 * g, a[g]);
            tmem_ld_wait();
            const bool whole = j0 + kT - 1 <= p_first && p_first + kT - 1 < w.n &&
                               (p_first + kT - 1 - j0 < prm.window || j0 + kT <= prm.sinks);
            if (!whole) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint32_t bits = seen_bits(p, j0 + 32 * g, prm.window, prm.sinks, w.n);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((bits >> e) & 1u)) a[g][e] = 0xff800000u;  // -inf
                }
            }
            float mx[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                mx[g] = __uint_as_float(a[g][0]);
#pragma unroll
                for (int e = 1; e < 32; ++e) mx[g] = fmaxf(mx[g], __uint_as_float(a[g][e]));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grow = top > m && (m == -INFINITY || (top - m) * c > kGrow);
            if (__any_sync(0xffffffffu, grow)) {
                const float keep = grow ? (m == -INFINITY ? 0.f : ex2((m - top) * c)) : 1.f;
                if (grow) m = top;
                l *= keep;
                if (done > 0) {
                    if (!(ok = wait_w(abort_flag, &sm.o_full[s], (uint32_t)(done - 1) & 1u))) break;
                    tc_fence_after();
#pragma unroll
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
            float base = m == -INFINITY ? 0.f : -m * c;
            if (__any_sync(0xffffffffu, fabsf(m) > 0x1p100f && m != -INFINITY)) {
                // m c may overflow: subtract first
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        a[g][e] = __float_as_uint(__uint_as_float(a[g][e]) - (m == -INFINITY ? 0.f : m));
                base = 0.f;
            }
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = ex2(fmaf(__uint_as_float(a[g][2 * e]), c, base));
                    const float y = ex2(fmaf(__uint_as_float(a[g][2 * e + 1]), c, base));
                    sum[e & 3] += x + y;
                    pk[e] = pack_bf16(x, y);
                }
                tmem_st16(ts + 16 * g, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.p_full[s]);
            ++done;
        }
        if (ok && done > 0) ok = wait_w(abort_flag, &sm.o_full[s], (uint32_t)(done - 1) & 1u);
        if (ok && w.t0[s] < prm.Nq) {
            tc_fence_after();
            // rows that saw nothing (l = 0) are zeros whatever TMEM holds
            const bool some = l != 0.f;
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
                prm.lse[((size_t)w.b * prm.Hq + w.h[s]) * prm.Nq + t] =
                    some ? (m == -INFINITY ? 0.f : m) * prm.scale + __log2f(l) * kLn2 : -INFINITY;
            fence_proxy_async_smem();
        }
        named_bar_sync(1 + s, 128);
        if (ok && w.t0[s] < prm.Nq && (warp & 3) == 0 && lane == 0) {
#pragma unroll
            for (int x = 0; x < DT; x += 64)
                tma_store_3d(&map_o, sm.q[s] + x / 64 * kBox, x, w.t0[s], w.b * prm.Hq + w.h[s]);
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

template <int DT>
la_status forward(const WindowProblem &p)
{
    const Params prm = params_of(p);
    const long long ctas = (long long)p.B * p.Hk * prm.units;
    if (ctas > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    CUtensorMap mq, mk, mv, mo;
    la_status st = make_map(&mq, p.q, p.B * p.Hq, p.Nq, p.d);
    if (st == LA_OK) st = make_map(&mk, p.k, p.B * p.Hk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&mv, p.v, p.B * p.Hk, p.Nk, p.d);
    if (st == LA_OK) st = make_map(&mo, p.out, p.B * p.Hq, p.Nq, p.d);
    if (st == LA_OK) st = ensure_smem((const void *)window_tc_kernel<DT>, (int)sizeof(Smem<DT>));
    if (st != LA_OK) return st;
    count_launches();
    return launch_dependent(window_tc_kernel<DT>, (unsigned)ctas, kThreads, (int)sizeof(Smem<DT>), p.stream, mq, mk, mv, mo,
                            prm);
}

}  // namespace

la_status window_forward_tc(const WindowProblem &p)
{
    return p.d <= 64 ? forward<64>(p) : forward<128>(p);
}

la_status tc_window_read_status(cudaStream_t s, unsigned *bits)
{
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_win_status, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_win_status, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return cuda_status(e);
}

}  // namespace la
