// Gated delta rule on the tensor cores: the backward pass (bf16), three launches: the
// chunks' matrices; the scan of the states forward and of their gradients in reverse, side by side; and
// the gradients of each chunk, all chunks at once.
#include "la_tc_delta_scan.cuh"

namespace la {
namespace delta {
namespace {

// CTAs 0 .. BH - 1 go forward, BH .. 2 BH - 1 in reverse: neither needs the other.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
delta_scans_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do, const Params p,
               const uint8_t *images, uint8_t *before, uint8_t *errors, uint8_t *after, uint8_t *dx)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int n = p.B * p.H, bh = (int)blockIdx.x;
    if (bh < n)
        scan_body<DK, DV, kSave>(map_q, map_k, map_v, map_v, p, p.S0, nullptr, images, nullptr, before, errors, bh, smem_raw);
    else
        scan_body<DK, DV, kReverse>(map_q, map_k, map_do, map_do, p, p.dSN, p.dS0, images, nullptr, after, dx, bh - n, smem_raw);
}

// ---------------------------------------------------------------- gradients of a chunk
// A CTA a (b, key head, chunk), over the heads that share the keys.  With B the state before the chunk, A its gradient
// behind it (each in two parts), E and dX from the scans:
//   lanes 0-63 of one product:  dO E^T, lanes 64-127: dX E^T;  of another: Q K^T and K K^T;
//   DP = scale D beta_j (dO E^T),  M = -D beta_i beta_j (dX E^T) below the diagonal;
//   dq = scale exp(G) B dO + DP K,   dk = -beta exp(G) B dX + beta exp(G_C - G) A E + DP^T Q + (M + M^T) K;
//   dbeta_i = (dX E^T)_ii,   dv = beta dX;
// DP and M are multiplied in two parts as well: dq's two terms nearly cancel where keys overwrite one another, and dk's.
// and g_t stands in each decay that crosses from before t to t or later: dg_t = sum over i >= t > j of (Q K^T DP + K K^T M)_ij
// + the reads of B at i >= t (q.dq, k.dk of the B terms) + the writes into A at j < t + exp(G_C) <B, A>.
// Products with the states have the key features as rows, so that a thread sums its feature's gradients over the
// heads in registers.  Warps 0-7: (w % 4: 32 TMEM lanes, w / 4: half of the columns); 8: products; 9: copies.
constexpr int kLocalWarps = 8, kLocalMma = 8, kLocalCopy = 9, kLocalThreads = 10 * 32;

template <int DK, int DV> struct LocalSmem {
    uint8_t qk[DK / 64][2 * kSq];      // per 64 columns: Q, K; then dq, dk
    uint8_t x[DV / 64][3 * kSq];       // per 64 columns: dO, dX's high part, its low part (then dv)
    uint8_t e[2][DV / 64][kSq];
    uint8_t b[2][DK / 64][DV * 128];
    uint8_t a[DK / 64][DV * 128];      // one part at a time
    uint8_t dp[kSq], m[kSq];           // dp: then partial sums
    uint8_t low[DV == 128 ? 16 : 2 * kSq];  // their low parts (d_v 128: over E's low part, once that has been read)
    Scalars s;
    float row[2][32];                  // sums of the first 32 columns of rows 32-63, of both matrices
    uint64_t keys_in, rows_in, b_in, a_in, mat_full, st_full, wk_full, dp_ready, low_ready, a_free, head_free, drain;
    uint32_t tmem_base;
    int abort;
};
struct Sums {  // over dp
    float pairs[2][4][32], reads[4][kChunk], writes[4][kChunk], whole[kLocalWarps];
};
static_assert(sizeof(Sums) <= kSq, "");

// Sums of v[e] over the warp's lanes: lane l gets that of v[l].
__device__ __forceinline__ float transposed_sums(float (&v)[32], int lane)
{
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int e = 0; e < d; ++e) {
            const float keep = up ? v[e + d] : v[e], give = up ? v[e] : v[e + d];
            v[e] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
    }
    return v[0];
}
__device__ __forceinline__ uint64_t both(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

template <int DK, int DV>
__global__ void __launch_bounds__(kLocalThreads, 1)
delta_local_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_dq,
               const __grid_constant__ CUtensorMap map_dk, const __grid_constant__ CUtensorMap map_dv, const Params p,
               const uint8_t *images, const uint8_t *before, const uint8_t *errors, const uint8_t *after, const uint8_t *dx)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    typedef LocalSmem<DK, DV> Sm;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    constexpr uint32_t tMat = 0, tLow = 64, tKeys = 128, tRq = 192, tRk = 256, tWk = 320, tDq = 384, tDk = 448;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const int chunks = (p.N + kChunk - 1) / kChunk, bhk = blockIdx.x / chunks, chunk = blockIdx.x % chunks, t0 = chunk * kChunk;
    const int group = p.H / p.Hk, bh0 = bhk / p.Hk * p.H + bhk % p.Hk * group;
    if (tid == 0) {
        uint64_t *one[] = {&sm.keys_in, &sm.rows_in, &sm.b_in, &sm.a_in, &sm.mat_full, &sm.st_full, &sm.wk_full, &sm.drain};
        for (uint64_t *b : one) mbar_init(b, 1);
        uint64_t *all[] = {&sm.dp_ready, &sm.low_ready, &sm.a_free, &sm.head_free};
        for (uint64_t *b : all) mbar_init(b, 32 * kLocalWarps);
        sm.abort = (smem_u32(smem_raw) & 1023u) == 0 ? 0 : 1;
        if (sm.abort) atomicOr(&g_delta_status, kStatusTimeout);
        fence_mbar_init();
    }
    if (warp == kLocalMma) {
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
    bool ok = !aborted(abort_flag);
    uint8_t *const low = DV == 128 ? sm.e[1][0] : sm.low;  // of DP, then of M

    if (warp == kLocalCopy) {
        auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_bar_warp(&g_delta_status, abort_flag, bar, parity); };
        if (ok && elect_one()) {
            mbar_arrive_expect_tx(&sm.keys_in, DK / 64 * 2 * kSq);
            for (int x = 0; x < DK / 64; ++x) {
                tma_load_3d(sm.qk[x], &map_q, &sm.keys_in, 64 * x, t0, bhk);
                tma_load_3d(sm.qk[x] + kSq, &map_k, &sm.keys_in, 64 * x, t0, bhk);
            }
        }
        __syncwarp();
        bool all = false;
        for (int h = 0; ok && h < group; ++h) {
            const size_t at = (size_t)(bh0 + h) * chunks + chunk;
            constexpr uint32_t half_state = state_bytes(DK, DV) / 2, half_rows = rows_bytes(DV) / 2;
            if (h > 0 && !(ok = wait(&sm.head_free, (uint32_t)(h - 1) & 1u))) break;
            if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
            if (elect_one()) {
                fence_proxy_async_global();
                mbar_arrive_expect_tx(&sm.rows_in, 5 * half_rows + (uint32_t)sizeof(Scalars));
                for (int x = 0; x < DV / 64; ++x) {
                    tma_load_3d(sm.x[x], &map_do, &sm.rows_in, 64 * x, t0, bh0 + h);
                    bulk_load(sm.x[x] + kSq, dx + at * rows_bytes(DV) + x * kSq, kSq, &sm.rows_in);
                    bulk_load(sm.x[x] + 2 * kSq, dx + at * rows_bytes(DV) + half_rows + x * kSq, kSq, &sm.rows_in);
                }
                bulk_load(sm.e, errors + at * rows_bytes(DV), rows_bytes(DV), &sm.rows_in);
                bulk_load(&sm.s, images + at * Layout<DK>::backward_bytes, sizeof(Scalars), &sm.rows_in);
                mbar_arrive_expect_tx(&sm.b_in, 2 * half_state);
                bulk_load(sm.b, before + at * state_bytes(DK, DV), 2 * half_state, &sm.b_in);
                mbar_arrive_expect_tx(&sm.a_in, half_state);
                bulk_load(sm.a, after + at * state_bytes(DK, DV), half_state, &sm.a_in);
            }
            __syncwarp();
            if (!(ok = wait(&sm.a_free, (uint32_t)h & 1u))) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.a_in, half_state);
                bulk_load(sm.a, after + at * state_bytes(DK, DV) + half_state, half_state, &sm.a_in);
            }
            __syncwarp();
            all = h + 1 == group;
        }
        if (!all) let_copies_land();
    } else if (warp == kLocalMma) {
        constexpr uint32_t id = idesc_bf16_f32(128, kChunk, false, false), id_mn = idesc_bf16_f32(128, kChunk, true, false);
        constexpr uint32_t id_both = idesc_bf16_f32(128, kChunk, true, true);
        constexpr uint32_t kBox = kSq >> 4, kXBox = 3 * kBox, kEPart = DV / 64 * kBox;
        constexpr uint32_t kLboState = DK == 128 ? DV * 128 : 0, kPart = DK / 64 * DV * 128 >> 4;
        constexpr uint32_t kLboKeys = DK == 128 ? 2 * kSq : 0;
        const uint64_t dkeys = rows_k(smem_u32(sm.qk[0]), 0), dx_ = rows_k(smem_u32(sm.x[0]), 0), de = rows_k(smem_u32(sm.e[0][0]), 0);
        const uint64_t db = cols_mn(smem_u32(sm.b[0][0]), 0, kLboState), da = cols_mn(smem_u32(sm.a[0]), 0, kLboState);
        const uint64_t dq = cols_mn(smem_u32(sm.qk[0]), 0, kLboKeys), dp_k = rows_k(smem_u32(sm.dp), 0), dp_mn = cols_mn(smem_u32(sm.dp), 0);
        const uint64_t low_k = rows_k(smem_u32(low), 0), low_mn = cols_mn(smem_u32(low), 0);
        auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(&g_delta_status, abort_flag, bar, parity); };
        // 16-column steps of rows of 64-column boxes `box` apart
        auto step = [](int kk, uint32_t box) { return (uint32_t)(kk >> 2) * box + (uint32_t)(kk & 3) * 2; };
        if (!__any_sync(0xffffffffu, aborted(abort_flag))) {
            wait(&sm.keys_in, 0);
            tc_fence_after();
            if (elect_one()) {  // [Q; K] K^T
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_ss(tmem + tKeys, dkeys + step(kk, 2 * kBox), dkeys + kBox + step(kk, 2 * kBox), id, kk > 0);
            }
            __syncwarp();
        }
        for (int h = 0; h < group; ++h) {
            if (__any_sync(0xffffffffu, aborted(abort_flag))) break;
            const uint32_t ph = (uint32_t)h & 1u;
            wait(&sm.rows_in, ph);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)  // [dO; dX] E^T, and the low part of dX
#pragma unroll
                    for (int kk = 0; kk < DV / 16; ++kk)
                        mma_ss(tmem + tMat, dx_ + step(kk, kXBox), de + part * kEPart + step(kk, kBox), id, part + kk > 0);
#pragma unroll
                for (int kk = 0; kk < DV / 16; ++kk)
                    mma_ss(tmem + tLow, dx_ + kBox + step(kk, kXBox), de + step(kk, kBox), id, kk > 0);
                mma_commit(&sm.mat_full);
            }
            __syncwarp();
            wait(&sm.b_in, ph);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)  // B dO^T
#pragma unroll
                    for (int kk = 0; kk < DV / 16; ++kk)
                        mma_ss(tmem + tRq, db + part * kPart + kk * (2048 >> 4), dx_ + step(kk, kXBox), id_mn, part + kk > 0);
#pragma unroll
                for (int part = 0; part < 3; ++part)  // B dX^T: high high, low high, high low
#pragma unroll
                    for (int kk = 0; kk < DV / 16; ++kk)
                        mma_ss(tmem + tRk, db + (part == 1) * kPart + kk * (2048 >> 4), dx_ + (part == 2 ? 2 : 1) * kBox + step(kk, kXBox),
                               id_mn, part + kk > 0);
            }
            __syncwarp();
            wait(&sm.a_in, 0);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)  // A's high part times E^T
#pragma unroll
                    for (int kk = 0; kk < DV / 16; ++kk)
                        mma_ss(tmem + tWk, da + kk * (2048 >> 4), de + part * kEPart + step(kk, kBox), id_mn, part + kk > 0);
                mma_commit(&sm.st_full);
            }
            __syncwarp();
            wait(&sm.dp_ready, ph);
            tc_fence_after();
            auto within = [&](uint64_t p_k, uint64_t p_mn, bool add) {
                const uint64_t k = dq + kBox, m_k = p_k + kBox, m_mn = p_mn + kBox;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_ss(tmem + tDq, k + kk * (2048 >> 4), p_k + kk * 2, id_mn, add || kk > 0);  // DP K
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(tmem + tDk, dq + kk * (2048 >> 4), p_mn + kk * (2048 >> 4), id_both, add || kk > 0);  // DP^T Q
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_ss(tmem + tDk, k + kk * (2048 >> 4), m_k + kk * 2, id_mn, 1);  // M K
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_ss(tmem + tDk, k + kk * (2048 >> 4), m_mn + kk * (2048 >> 4), id_both, 1);  // M^T K
            };
            if (elect_one()) within(dp_k, dp_mn, h > 0);
            __syncwarp();
            wait(&sm.low_ready, ph);
            tc_fence_after();
            if (elect_one()) within(low_k, low_mn, true);
            __syncwarp();
            wait(&sm.a_in, 1);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < DV / 16; ++kk)  // A's low part times E^T
                    mma_ss(tmem + tWk, da + kk * (2048 >> 4), de + step(kk, kBox), id_mn, 1);
                mma_commit(&sm.wk_full);
            }
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(&sm.drain);  // every MMA issued completes before TMEM is freed
            drain(&sm.drain, 0);
        }
        __syncwarp();
    } else {
        auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_bar_warp(&g_delta_status, abort_flag, bar, parity); };
        const int q = warp & 3, half = warp >> 2, f = 32 * q + lane, c0 = 32 * half;
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        const bool live = 32 * q < DK;  // the lanes are key features of the products with the states
        float dq[32], dk[32];           // of feature f, tokens c0 ..
#pragma unroll
        for (int e = 0; e < 32; ++e) dq[e] = dk[e] = 0.f;
        uint32_t at[8];  // (row e, feature f) of Q's tile
#pragma unroll
        for (int e = 0; e < 8; ++e) at[e] = ((f & (DK - 1)) >> 6) * 2 * kSq + sw128_offset(e, f & 63);
        Sums &sums = *reinterpret_cast<Sums *>(sm.dp);
        for (int h = 0; ok && h < group; ++h) {
            const uint32_t ph = (uint32_t)h & 1u;
            const size_t gates = (size_t)(bh0 + h) * p.N + t0;
            if (!(ok = wait(&sm.rows_in, ph) && wait(&sm.mat_full, ph))) break;
            tc_fence_after();
            // ---- the matrices of the chunk: row i of DP (lanes 0-63) or of M, columns c0 ..
            float pairs = 0.f;
            uint32_t lows[16];
            {
                const int i = f & 63;
                const bool is_m = q >= 2, upper = half == 1 && (q & 1) == 0, diagonal = half == (q & 1);
                float r[32];
                if (upper) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = 0.f, lows[e / 2] = 0u;
                    uint8_t *to = is_m ? sm.m : sm.dp;
#pragma unroll
                    for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4 *>(to + sw128_offset(i, c0 + 8 * c)) = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const uint64_t hi = pair(sm.s.hi[i], sm.s.hi[i]), lo = pair(sm.s.lo[i], sm.s.lo[i]);
                    const float own = is_m ? -sm.s.beta[i] : p.scale;
                    uint8_t *to = is_m ? sm.m : sm.dp;
#pragma unroll
                    for (int y = 0; y < 32; y += 16) {
                        uint32_t a[16], b[16];
                        tmem_ld16(tl + tMat + c0 + y, a);
                        if (is_m) tmem_ld16(tl + tLow + c0 + y, b);
                        tmem_ld_wait();
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(a[e]) + (is_m ? __uint_as_float(b[e]) : 0.f);
                        if (is_m && diagonal) {
                            float d = 0.f;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (y + e == lane) d = v[e];
                            if (lane >= y && lane < y + 16 && t0 + i < p.N) p.dbeta[gates + i] = d;
                        }
                        tmem_ld16(tl + tKeys + c0 + y, a);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const int j = c0 + y + e;
                            const uint64_t w = decay2(hi, lo, *reinterpret_cast<const float2 *>(&sm.s.hi[j]), *reinterpret_cast<const float2 *>(&sm.s.lo[j]));
                            const float2 b2 = *reinterpret_cast<const float2 *>(&sm.s.beta[j]);
                            unpair(mul2(w, mul2(pair(own * b2.x, own * b2.y), pair(v[e], v[e + 1]))), v[e], v[e + 1]);
                        }
                        if (diagonal) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (y + e > lane || (is_m && y + e == lane)) v[e] = 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            uint32_t hi4[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) split2(v[e + 2 * u], v[e + 2 * u + 1], hi4[u], lows[(y + e) / 2 + u]);
                            *reinterpret_cast<uint4 *>(to + sw128_offset(i, c0 + y + e)) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
                        }
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) r[y + e] = (diagonal && y + e == lane) ? 0.f : v[e] * __uint_as_float(a[e]);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&sm.dp_ready);
                // column t of r: the row's sum over j < t, for t up to i
                float run = 0.f;
                if (half == 0) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float x = r[e];
                        r[e] = (q & 1) || e <= lane ? run : 0.f;
                        run += x;
                    }
                    if (q & 1) sm.row[q >> 1][lane] = run;
                }
                named_bar_sync(1, 256);
                if (half == 1) {
                    run = (q & 1) ? sm.row[q >> 1][lane] : 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float x = r[e];
                        r[e] = (q & 1) && e <= lane ? run : 0.f;
                        run += x;
                    }
                }
                pairs = transposed_sums(r, lane);
            }
            // ---- <B, A>, with A's high part
            float whole = 0.f;
            if (!(ok = wait(&sm.b_in, ph) && wait(&sm.a_in, 0))) break;
            {
                uint64_t acc = 0;
                const uint4 *bh = reinterpret_cast<const uint4 *>(sm.b[0][0]), *bl = reinterpret_cast<const uint4 *>(sm.b[1][0]);
                const uint4 *ah = reinterpret_cast<const uint4 *>(sm.a[0]);
#pragma unroll 2
                for (int i = tid; i < DK * DV / 8; i += 256) {
                    const uint4 x = bh[i], y = bl[i], z = ah[i];
                    acc = fma2(add2(both(x.x), both(y.x)), both(z.x), acc);
                    acc = fma2(add2(both(x.y), both(y.y)), both(z.y), acc);
                    acc = fma2(add2(both(x.z), both(y.z)), both(z.z), acc);
                    acc = fma2(add2(both(x.w), both(y.w)), both(z.w), acc);
                }
                float x, y;
                unpair(acc, x, y);
                whole = x + y;
            }
            if (!(ok = wait(&sm.st_full, ph))) break;
            tc_fence_after();
            mbar_arrive(&sm.a_free);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4 *>(low + (q >= 2) * kSq + sw128_offset(f & 63, c0 + 8 * c)) =
                    make_uint4(lows[4 * c], lows[4 * c + 1], lows[4 * c + 2], lows[4 * c + 3]);
            fence_proxy_async_smem();
            mbar_arrive(&sm.low_ready);
            // ---- reads of B
            float reads = 0.f, writes = 0.f;
            if (live) {
                float v[32];
#pragma unroll
                for (int y = 0; y < 32; y += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16(tl + tRq + c0 + y, a);
                    tmem_ld16(tl + tRk + c0 + y, b);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = y + e;
                        const uint8_t *row = sm.qk[0] + (c0 + t) / 8 * 1024 + at[e & 7];
                        const float x = p.scale * sm.s.first[c0 + t] * __uint_as_float(a[e]), z = sm.s.back[c0 + t] * __uint_as_float(b[e]);
                        dq[t] += x;
                        dk[t] += z;
                        v[t] = fmaf(bf16_at(row), x, bf16_at(row + kSq) * z);
                    }
                }
                reads = transposed_sums(v, lane);
            }
            // ---- dv = beta dX over dX's low part, which the products have read
            for (int i = tid; i < kChunk * DV / 8; i += 256) {
                const int box = i / (kChunk * 8), u = i % (kChunk * 8), r = u >> 3;
                uint8_t *at_hi = sm.x[box] + kSq + u * 16, *at_lo = at_hi + kSq;
                const uint4 x = *reinterpret_cast<const uint4 *>(at_hi), y = *reinterpret_cast<const uint4 *>(at_lo);
                const uint64_t b = pair(sm.s.beta[r], sm.s.beta[r]);
                auto one = [&](uint32_t u, uint32_t v) {
                    float s, t;
                    unpair(mul2(b, add2(both(u), both(v))), s, t);
                    return pack_bf16(s, t);
                };
                *reinterpret_cast<uint4 *>(at_lo) = make_uint4(one(x.x, y.x), one(x.y, y.y), one(x.z, y.z), one(x.w, y.w));
            }
            fence_proxy_async_smem();
            // ---- A's low part
            if (!(ok = wait(&sm.a_in, 1))) break;
            {
                uint64_t acc = 0;
                const uint4 *bh = reinterpret_cast<const uint4 *>(sm.b[0][0]), *al = reinterpret_cast<const uint4 *>(sm.a[0]);
#pragma unroll 2
                for (int i = tid; i < DK * DV / 8; i += 256) {
                    const uint4 x = bh[i], z = al[i];
                    acc = fma2(both(x.x), both(z.x), acc);
                    acc = fma2(both(x.y), both(z.y), acc);
                    acc = fma2(both(x.z), both(z.z), acc);
                    acc = fma2(both(x.w), both(z.w), acc);
                }
                float x, y;
                unpair(acc, x, y);
                whole += x + y;
            }
            if (!(ok = wait(&sm.wk_full, ph))) break;
            tc_fence_after();
            if (live) {
                float v[32];
#pragma unroll
                for (int y = 0; y < 32; y += 16) {
                    uint32_t a[16];
                    tmem_ld16(tl + tWk + c0 + y, a);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = y + e;
                        const float x = sm.s.write[c0 + t] * __uint_as_float(a[e]);
                        dk[t] += x;
                        v[t] = x * bf16_at(sm.qk[0] + kSq + (c0 + t) / 8 * 1024 + at[e & 7]);
                    }
                }
                writes = transposed_sums(v, lane);
            }
            for (int d = 1; d < 32; d *= 2) whole += __shfl_xor_sync(0xffffffffu, whole, d);
            // the products have read DP: the sums over lanes and warps go there
            sums.pairs[half][q][lane] = pairs;
            sums.reads[q][c0 + lane] = reads;
            sums.writes[q][c0 + lane] = writes;
            if (lane == 0) sums.whole[warp] = whole;
            tc_fence_before();
            named_bar_sync(1, 256);
            if (warp == 0) {
                if (lane == 0) {
                    for (int x = 0; x < DV / 64; ++x) tma_store_3d(&map_dv, sm.x[x] + 2 * kSq, 64 * x, t0, bh0 + h);
                    tma_store_commit();
                }
                float pr[2], rd[2], wr[2], total = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = 32 * u + lane;
                    pr[u] = (sums.pairs[u][0][lane] + sums.pairs[u][1][lane]) + (sums.pairs[u][2][lane] + sums.pairs[u][3][lane]);
                    rd[u] = (sums.reads[0][t] + sums.reads[1][t]) + (sums.reads[2][t] + sums.reads[3][t]);
                    wr[u] = (sums.writes[0][t] + sums.writes[1][t]) + (sums.writes[2][t] + sums.writes[3][t]);
                }
                for (int w = 0; w < kLocalWarps; ++w) total += sums.whole[w];
                for (int d = 1; d < 32; d *= 2) {  // reads from t on, writes up to t
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float x = __shfl_down_sync(0xffffffffu, rd[u], d), y = __shfl_up_sync(0xffffffffu, wr[u], d);
                        if (lane + d < 32) rd[u] += x;
                        if (lane >= d) wr[u] += y;
                    }
                }
                rd[0] += __shfl_sync(0xffffffffu, rd[1], 0);
                const float first_half = __shfl_sync(0xffffffffu, wr[0], 31);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float up = __shfl_up_sync(0xffffffffu, wr[u], 1);  // writes before t
                    const float w = (lane ? up : 0.f) + (u ? first_half : 0.f);
                    if (t0 + 32 * u + lane < p.N)
                        p.dg[gates + 32 * u + lane] = pr[u] + rd[u] + w + sm.s.first[kChunk - 1] * total;
                }
                if (lane == 0) tma_store_wait_read_all();
                __syncwarp();
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.head_free);
        }
        if (ok) {  // dq over Q, dk over K, which every product has read
            named_bar_sync(1, 256);
            if (live)
#pragma unroll
                for (int y = 0; y < 32; y += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16(tl + tDq + c0 + y, a);
                    tmem_ld16(tl + tDk + c0 + y, b);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        uint8_t *row = sm.qk[0] + (c0 + y + e) / 8 * 1024 + at[e & 7];
                        *reinterpret_cast<__nv_bfloat16 *>(row) = __float2bfloat16_rn(dq[y + e] + __uint_as_float(a[e]));
                        *reinterpret_cast<__nv_bfloat16 *>(row + kSq) = __float2bfloat16_rn(dk[y + e] + __uint_as_float(b[e]));
                    }
                }
            fence_proxy_async_smem();
            named_bar_sync(1, 256);
            if (warp == 0 && lane == 0) {
                for (int x = 0; x < DK / 64; ++x) {
                    tma_store_3d(&map_dq, sm.qk[x], 64 * x, t0, bhk);
                    tma_store_3d(&map_dk, sm.qk[x] + kSq, 64 * x, t0, bhk);
                }
                tma_store_commit();
            }
        }
        if (warp == 0 && lane == 0) tma_store_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kLocalMma) tmem_dealloc(tmem, 512);
}

template <int DK, int DV> struct Scratch4 {  // what the launches leave for one another, per (b, h, chunk)
    static constexpr size_t images = Layout<DK>::backward_bytes, state = state_bytes(DK, DV), rows = rows_bytes(DV);
    static constexpr size_t total = images + 2 * state + 2 * rows;
};

template <int DK, int DV> la_status backward(const DeltaProblem &p)
{
    typedef ScanSmem<DK, DV, kSave> Save;
    typedef ScanSmem<DK, DV, kReverse> Rev;
    typedef LocalSmem<DK, DV> Loc;
    typedef Scratch4<DK, DV> Sc;
    constexpr size_t scans = sizeof(Save) > sizeof(Rev) ? sizeof(Save) : sizeof(Rev);
    static_assert(scans <= 227 * 1024 && sizeof(Loc) <= 227 * 1024, "");
    const Params prm = params_of(p);
    const size_t n = (size_t)p.B * p.H * ceil_div(p.N, kChunk);
    uint8_t *images = reinterpret_cast<uint8_t *>(p.scratch), *before = images + n * Sc::images, *after = before + n * Sc::state;
    uint8_t *errors = after + n * Sc::state, *dx = errors + n * Sc::rows;
    CUtensorMap mq, mk, mv, mo, mdq, mdk, mdv;
    la_status st = make_map(&mv, p.v, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = make_map(&mo, p.dout, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = make_map(&mdq, p.dq, p.B * p.Hk, p.N, p.dk, kChunk);
    if (st == LA_OK) st = make_map(&mdk, p.dk_out, p.B * p.Hk, p.N, p.dk, kChunk);
    if (st == LA_OK) st = make_map(&mdv, p.dv_out, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = ensure_smem((const void *)delta_scans_tc<DK, DV>, (int)scans);
    if (st == LA_OK) st = ensure_smem((const void *)delta_local_tc<DK, DV>, (int)sizeof(Loc));
    if (st == LA_OK) st = prepare<DK, true>(p, prm, images, &mq, &mk);
    if (st != LA_OK) return st;
    count_launches();
    st = launch_dependent(delta_scans_tc<DK, DV>, (unsigned)(2 * p.B * p.H), kThreads, (int)scans, p.stream, mq, mk, mv, mo, prm,
                          (const uint8_t *)images, before, errors, after, dx);
    if (st != LA_OK) return st;
    count_launches();
    return launch_dependent(delta_local_tc<DK, DV>, (unsigned)(p.B * p.Hk * ceil_div(p.N, kChunk)), kLocalThreads, (int)sizeof(Loc),
                            p.stream, mq, mk, mo, mdq, mdk, mdv, prm, (const uint8_t *)images, (const uint8_t *)before,
                            (const uint8_t *)errors, (const uint8_t *)after, (const uint8_t *)dx);
}

}  // namespace
}  // namespace delta

using namespace delta;

size_t delta_backward_tc_scratch(const DeltaProblem &p)
{
    const size_t n = (size_t)p.B * p.H * ceil_div(p.N, kChunk);
    if (p.dk <= 64) return n * (p.dv <= 64 ? Scratch4<64, 64>::total : Scratch4<64, 128>::total);
    return n * (p.dv <= 64 ? Scratch4<128, 64>::total : Scratch4<128, 128>::total);
}

la_status delta_backward_tc(const DeltaProblem &p)
{
    if (p.dk <= 64) return p.dv <= 64 ? backward<64, 64>(p) : backward<64, 128>(p);
    return p.dv <= 64 ? backward<128, 64>(p) : backward<128, 128>(p);
}

la_status tc_delta_bwd_read_status(cudaStream_t s, unsigned *bits) { return read_status(g_launched, g_delta_status, s, bits); }

}  // namespace la
