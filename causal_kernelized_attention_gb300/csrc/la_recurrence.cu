// Gated recurrence, each channel on its own:
//
//   forward    h_t = alpha_t h_{t-1} + x_t                       (h_{-1} = h0, or 0)
//   backward   g_t = dh_t + alpha_{t+1} g_{t+1}                  (g_{N-1} = dh_{N-1} + dhN)
//              dx_t = g_t,  dalpha_t = g_t h_{t-1},  dh0 = alpha_0 g_0
//
// The backward pass is the forward's scan over reversed time with the gates moved by one
// token, so one kernel does both.  A run of tokens maps the state before it, c, to A c + H
// with A the product of its gates and H its result from zero; runs compose as
// (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2), without a division, so gates of 0 are exact.
// With the state before its run a warp then steps through the run itself, so every h_t is
// rounded as the recurrence rounds it.
//
// Bound by memory: alpha and x are read once, h written once (4 + 2 e bytes an element,
// e the size of x).  A CTA takes a tile of consecutive tokens of neighbouring channels, a
// warp a run of them, a lane its channels; runs are joined through shared memory.  A cluster
// of CTAs takes consecutive tiles of the same channels and its CTAs send each other their
// (A, H) once a step, so a sequence is split over the machine when there are few channels, in
// one pass over the data and without a flag in global memory to wait for.  The sends are
// asynchronous stores counted on mbarriers: a cluster barrier in their place also waits for
// the step's global stores (695 us instead of 347 at 65536 x 4096, forward, on tiles of 64).
//
// Measured at 65536 x 4096, bf16: forward 326 us (6.6 TB/s), backward 540 us (7.0 TB/s); fp32
// backward 852 us (6.3 TB/s).  4 x 2048 x 512 forward 7.2 us (4.6 TB/s, two steps of a cluster).
//
// Where the largest clusters leave half of the machine idle and a sequence is 32 tiles or longer, it
// is split into segments instead, one CTA each: one launch finds every segment's (A, H), a
// second joins those before its own and runs it.  That reads alpha and x twice but takes no step for
// step exchange: 65536 x 64 forward 19 us instead of 102, 30000 x 33 backward 27 instead of 161, 16384 x
// 512 forward 18 instead of 28; 4096 x 64 forward 7.6 instead of 8.5, below that the launch costs more
// than it saves (2048 x 64: 7.2 instead of 5.6).
//
// Rows of whole 16-byte vectors come in by TMA, kStages tiles of 128 tokens x 64 channels deep,
// so that the bytes in flight depend neither on registers nor on occupancy; other widths by
// plain loads, one channel a lane.
#include <algorithm>
#include <type_traits>

#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRun = 16;             // tokens of a warp's run
constexpr int kTok = kWarps * kRun;  // tokens of a tile

static __device__ unsigned g_rec_status;
std::atomic<bool> g_launched{false};

// V neighbouring elements of type T.
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T x[V]; };
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ld(const T *p) { return *reinterpret_cast<const Vec<T, V> *>(p); }
template <typename T, int V>
__device__ __forceinline__ void st(T *p, const Vec<T, V> &v) { *reinterpret_cast<Vec<T, V> *>(p) = v; }
template <typename T, int V>
__device__ __forceinline__ Vec<float, V> ldf(const T *p)
{
    const Vec<T, V> v = ld<T, V>(p);
    Vec<float, V> f;
#pragma unroll
    for (int i = 0; i < V; ++i) f.x[i] = Elem<T>::to_f32(v.x[i]);
    return f;
}
template <typename T, int V>
__device__ __forceinline__ void stf(T *p, const Vec<float, V> &f)
{
    Vec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v.x[i] = Elem<T>::from_f32(f.x[i]);
    st<T, V>(p, v);
}

template <typename T>
struct Args {
    const T *x;          // forward: x; backward: dh
    const float *alpha;
    const T *h_in;       // backward: h
    const float *h0;     // may be null
    const float *dhN;    // backward, may be null
    T *out;              // forward: h; backward: dx
    float *dalpha;       // backward
    float *last;         // forward: hN; backward: dh0; may be null
    float *fold;         // [units][segs][A, H][kCh] where segs > 1
    int N, D, steps, segs;
};

template <typename T, bool kH, bool kDeep>
struct Tiles {  // the TMA ring
    static constexpr int kBytes = kTok * 64 * (4 + (kH ? 2 : 1) * (int)sizeof(T));
    static constexpr int kStages = (kDeep ? 196 : 100) * 1024 / kBytes;
    float alpha[kStages][kTok][64];
    T x[kStages][kTok][64];
    T h[kH ? kStages : 1][kH ? kTok : 1][64];
};
struct NoTiles {
    static constexpr int kStages = 1;
};

template <typename T, bool kH, bool kTma, bool kDeep>
struct Smem {
    static constexpr int kPer = kTma ? 2 : 1, kCh = 32 * kPer;  // channels of a lane, of a CTA
    typedef typename std::conditional<kTma, Tiles<T, kH, kDeep>, NoTiles>::type Ring;
    Ring t;
    alignas(16) float wA[2][kWarps][kCh];  // the warps' runs, by step parity
    float wH[2][kWarps][kCh];
    float cA[2][kMaxCluster][kCh], cH[2][kMaxCluster][kCh];  // the cluster's tiles
    uint64_t full[Ring::kStages], sent[2];
    int abort;
};

// kWhole: a cluster has a whole sequence.  The other two split it into a.segs segments.
enum Mode { kWhole, kFolds, kSegment };

template <typename T, bool kBack, bool kTma, bool kDeep, Mode kMode>
__global__ void __launch_bounds__(kThreads)
recurrence_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_h, const __grid_constant__ Args<T> a)
{
    extern __shared__ __align__(128) uint8_t smem_raw[];
    constexpr bool kFold = kMode == kFolds, kH = kBack && !kFold;
    typedef Smem<T, kH, kTma, kDeep> S_;
    S_ &sm = *reinterpret_cast<S_ *>(smem_raw);
    constexpr int kPer = S_::kPer, kCh = S_::kCh, kStages = S_::Ring::kStages;
    typedef Vec<float, kPer> F;
    constexpr uint32_t kBytes = kTok * kCh * (4 + (kH ? 2 : 1) * sizeof(T));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lc = kPer * lane;
    const uint32_t S = cluster_size(), rank = S > 1 ? cluster_ctarank() : 0;
    const int groups = (a.D + kCh - 1) / kCh, segs = kMode == kWhole ? 1 : a.segs, at_seg = (int)(blockIdx.x / S);
    const int unit = at_seg / segs, seg = kMode == kWhole ? 0 : at_seg % segs;
    if (kFold && seg == segs - 1) return;  // (no segment is after the last)
    const int b = unit / groups, c0 = (unit % groups) * kCh, ch = c0 + lc;
    const bool live = ch < a.D;  // (D is even where a lane has two channels)

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.sent[i], 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (S > 1)
        cluster_sync_all();  // every CTA of the cluster runs before its memory is written
    else
        __syncthreads();

    // scan index of this CTA's first token of a step; token t = i (forward), N - 1 - i (backward):
    // the backward's tiles lie in memory order, and are read from their last row
    auto first_of = [&](int step) { return (((long long)seg * a.steps + step) * S + rank) * kTok; };
    auto fetch = [&](int step) {
        if constexpr (kTma) {
            const long long i0 = first_of(step);
            if (step >= a.steps || i0 >= a.N) return;
            const int s = step % kStages, t0 = kBack ? (int)(a.N - i0 - kTok) : (int)i0;
            mbar_arrive_expect_tx(&sm.full[s], kBytes);
            tma_load_3d(sm.t.alpha[s], &map_a, &sm.full[s], c0, kBack ? t0 + 1 : t0, b);
            tma_load_3d(sm.t.x[s], &map_x, &sm.full[s], c0, t0, b);
            if (kH) tma_load_3d(sm.t.h[s], &map_h, &sm.full[s], c0, t0 - 1, b);
        }
    };
    if (kTma && tid == 0)
        for (int i = 0; i < kStages; ++i) fetch(i);

    F carry, h0;  // carry: the state before the cluster's step
#pragma unroll
    for (int v = 0; v < kPer; ++v) carry.x[v] = h0.x[v] = 0.f;
    const size_t base = (size_t)b * a.N * a.D + ch, at_b = (size_t)b * a.D + ch;
    F whole;  // the gates' product over this segment
#pragma unroll
    for (int v = 0; v < kPer; ++v) whole.x[v] = 1.f;
    float *const fold = a.fold + (size_t)unit * segs * 2 * kCh + lc;
    if (!kFold && live && (kBack ? a.dhN : a.h0)) carry = ld<float, kPer>((kBack ? a.dhN : a.h0) + at_b);
    if (kMode == kSegment && live) {
#pragma unroll 8
        for (int i = 0; i < seg; ++i) {
            const F xa = ld<float, kPer>(fold + i * 2 * kCh), xh = ld<float, kPer>(fold + (i * 2 + 1) * kCh);
#pragma unroll
            for (int v = 0; v < kPer; ++v) carry.x[v] = fmaf(xa.x[v], carry.x[v], xh.x[v]);
        }
    }
    if (kH && live && a.h0) h0 = ld<float, kPer>(a.h0 + at_b);

    bool ok = true;
    for (int step = 0; step < a.steps; ++step) {
        const int par = step & 1;
        const long long i0 = first_of(step);
        const int left = (int)min((long long)kTok, max(a.N - i0, 0ll));  // tokens of this tile
        F al[kRun], xv[kRun], hv[kRun];
        if constexpr (kTma) {
            const int s = step % kStages;
            if (left > 0) {
                if (ok) ok = tc::wait_bar(&g_rec_status, &sm.abort, &sm.full[s], (uint32_t)(step / kStages) & 1u);
#pragma unroll
                for (int r = 0; r < kRun; ++r) {
                    const int k = warp * kRun + r, row = kBack ? kTok - 1 - k : k;
                    al[r] = ld<float, kPer>(&sm.t.alpha[s][row][lc]);
                    xv[r] = ldf<T, kPer>(&sm.t.x[s][row][lc]);
                    if (kH) hv[r] = ldf<T, kPer>(&sm.t.h[s][row][lc]);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                const int k = warp * kRun + r;
                if (k < left && live) {
                    const long long t = kBack ? a.N - 1 - (i0 + k) : i0 + k;
                    const size_t o = base + (size_t)t * a.D;
                    if (!kBack || i0 + k > 0) al[r] = ld<float, kPer>(a.alpha + o + (kBack ? a.D : 0));
                    xv[r] = ldf<T, kPer>(a.x + o);
                    if (kH && t > 0) hv[r] = ldf<T, kPer>(a.h_in + o - a.D);
                }
            }
        }
        if (left < kTok || (kBack && i0 == 0)) {
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                const int k = warp * kRun + r;
#pragma unroll
                for (int v = 0; v < kPer; ++v) {
                    // past the end: the identity; the last token's state has no later gate
                    if (k >= left || (kBack && i0 + k == 0)) al[r].x[v] = 1.f;
                    if (k >= left) xv[r].x[v] = 0.f;
                }
            }
        }
        F A, H;
#pragma unroll
        for (int v = 0; v < kPer; ++v) {
            A.x[v] = 1.f;
            H.x[v] = 0.f;
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                H.x[v] = fmaf(al[r].x[v], H.x[v], xv[r].x[v]);
                A.x[v] *= al[r].x[v];
            }
        }
        st<float, kPer>(&sm.wA[par][warp][lc], A);
        st<float, kPer>(&sm.wH[par][warp][lc], H);
        __syncthreads();  // the runs are written, and the stage is read
        if (tid == 0) {
            if (kTma) fetch(step + kStages);
            if (S > 1) mbar_arrive_expect_tx(&sm.sent[par], S * kCh * 2 * 4);
        }
        // the runs before this warp's in the CTA, and the whole CTA's
        F pA, pH, tA, tH;
#pragma unroll
        for (int v = 0; v < kPer; ++v) {
            pA.x[v] = tA.x[v] = 1.f;
            pH.x[v] = tH.x[v] = 0.f;
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) {
                pA = tA;
                pH = tH;
            }
            const F xa = ld<float, kPer>(&sm.wA[par][w][lc]), xh = ld<float, kPer>(&sm.wH[par][w][lc]);
#pragma unroll
            for (int v = 0; v < kPer; ++v) {
                tH.x[v] = fmaf(xa.x[v], tH.x[v], xh.x[v]);
                tA.x[v] *= xa.x[v];
            }
        }
        F at = carry;  // the state before this CTA's tile
        if (S > 1) {
            // Warp w sends to rank w.  The slots alternate: a CTA that still reads this step's has
            // not sent its next tile, which whoever writes the slot again waits for first.
            if (warp < (int)S) {
                const uint32_t bar = mapa_shared(smem_u32(&sm.sent[par]), warp);
                const uint32_t da = mapa_shared(smem_u32(&sm.cA[par][rank][lc]), warp);
                const uint32_t dh = mapa_shared(smem_u32(&sm.cH[par][rank][lc]), warp);
                if constexpr (kPer == 2) {
                    st_async_f32x2(da, tA.x[0], tA.x[1], bar);
                    st_async_f32x2(dh, tH.x[0], tH.x[1], bar);
                } else {
                    st_async_f32(da, tA.x[0], bar);
                    st_async_f32(dh, tH.x[0], bar);
                }
            }
            if (ok) ok = tc::wait_bar(&g_rec_status, &sm.abort, &sm.sent[par], (uint32_t)(step >> 1) & 1u);
            for (uint32_t w = 0; w < S; ++w) {
                const F xa = ld<float, kPer>(&sm.cA[par][w][lc]), xh = ld<float, kPer>(&sm.cH[par][w][lc]);
                if (w == rank) at = carry;
#pragma unroll
                for (int v = 0; v < kPer; ++v) carry.x[v] = fmaf(xa.x[v], carry.x[v], xh.x[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < kPer; ++v) carry.x[v] = fmaf(tA.x[v], carry.x[v], tH.x[v]);
        }
        if constexpr (kFold) {
#pragma unroll
            for (int v = 0; v < kPer; ++v) whole.x[v] *= tA.x[v];
        } else {
            F c;
#pragma unroll
            for (int v = 0; v < kPer; ++v) c.x[v] = fmaf(pA.x[v], at.x[v], pH.x[v]);
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                const int k = warp * kRun + r;
#pragma unroll
                for (int v = 0; v < kPer; ++v) c.x[v] = fmaf(al[r].x[v], c.x[v], xv[r].x[v]);
                if (k < left && live) {
                    const long long t = kBack ? a.N - 1 - (i0 + k) : i0 + k;
                    const size_t o = base + (size_t)t * a.D;
                    stf<T, kPer>(a.out + o, c);
                    if (kBack) {
                        F da;
#pragma unroll
                        for (int v = 0; v < kPer; ++v) da.x[v] = c.x[v] * (t == 0 ? h0.x[v] : hv[r].x[v]);
                        st<float, kPer>(a.dalpha + o, da);
                    }
                }
            }
        }
    }
    if constexpr (kFold) {
        if (warp == 0 && live) {
            st<float, kPer>(fold + seg * 2 * kCh, whole);
            st<float, kPer>(fold + (seg * 2 + 1) * kCh, carry);
        }
    }
    // the state after the last token (forward), or alpha_0 g_0 (backward)
    if (!kFold && a.last && seg == segs - 1 && rank == 0 && warp == 0 && live) {
        if (kBack && a.N > 0) {
            const F f = ld<float, kPer>(a.alpha + base);
#pragma unroll
            for (int v = 0; v < kPer; ++v) carry.x[v] *= f.x[v];
        }
        st<float, kPer>(a.last + at_b, carry);
    }
    if (!ok) {  // a wait ran out: nothing may still arrive in this CTA's shared memory when it exits
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000000ull) {
        }
    }
}

// [B, N, D] as a 3-D tensor (D, N, B); box = 64 channels x 128 tokens.
la_status tile_map(CUtensorMap *m, const void *ptr, bool f32, int B, int N, int D)
{
    tc::EncodeTiledFn enc;
    la_status st = tc::encode_fn(&enc);
    if (st == LA_OK) st = tc::bind_thread_context();
    if (st != LA_OK) return st;
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t strides[2] = {(cuuint64_t)D * e, (cuuint64_t)N * D * e};
    const cuuint32_t box[3] = {64, kTok, 1}, estr[3] = {1, 1, 1};
    const CUresult r = enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? LA_OK : cuda_status(cudaErrorInvalidValue);
}

template <typename T, bool kBack, bool kTma, bool kDeep, Mode kMode>
la_status launch(const RecurrenceProblem &p, const Args<T> &a, long long units, int S)
{
    auto kern = recurrence_kernel<T, kBack, kTma, kDeep, kMode>;
    constexpr bool kH = kBack && kMode != kFolds;
    constexpr size_t smem = sizeof(Smem<T, kH, kTma, kDeep>);
    CUtensorMap ma{}, mx{}, mh{};
    la_status st = ensure_smem((const void *)kern, (int)smem);
    if (kTma) {
        if (st == LA_OK) st = tile_map(&ma, p.alpha, true, p.B, p.N, p.D);
        if (st == LA_OK) st = tile_map(&mx, a.x, sizeof(T) == 4, p.B, p.N, p.D);
        if (st == LA_OK && kH) st = tile_map(&mh, p.h_in, sizeof(T) == 4, p.B, p.N, p.D);
    }
    if (st != LA_OK) return st;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(units * a.segs * S));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = p.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = S > 1 ? 1 : 0;
    g_launched = true;
    count_launches();
    return cuda_status(cudaLaunchKernelEx(&lc, kern, ma, mx, mh, a));
}

// Runs the problem, or with `bytes` only finds the scratch that it needs.
template <typename T, bool kBack, bool kTma, bool kDeep = false>
la_status run(const RecurrenceProblem &p, size_t *bytes)
{
    typedef Smem<T, kBack, kTma, kDeep> S_;
    const long long units = (long long)p.B * ceil_div(p.D, S_::kCh);
    const long long tiles = ((long long)p.N + kTok - 1) / kTok;
    // CTAs a sequence and group of channels: as many as run at once (two an SM where shared
    // memory allows), none without a tile of its own.
    constexpr int resident = sizeof(S_) <= 113 * 1024 ? 2 : 1;
    const long long room = (long long)resident * tc::sm_count() / units;
    int S = 1;
    while (S < kMaxCluster && S < tiles && S * 2 <= room) S *= 2;
    if (units * S > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    Args<T> a;
    a.segs = 1;
    if (!kDeep && room >= 2 * kMaxCluster && tiles >= 4 * kMaxCluster) {  // segments (see above)
        a.segs = (int)std::min(room, tiles);
        S = 1;
    }
    a.steps = (int)((tiles + a.segs * S - 1) / (a.segs * S));
    if (a.segs > 1) a.segs = (int)((tiles + a.steps - 1) / a.steps);  // none without a tile
    if (bytes) {
        *bytes = a.segs > 1 ? (size_t)units * a.segs * 2 * S_::kCh * sizeof(float) : 0;
        return LA_OK;
    }
    a.x = static_cast<const T *>(kBack ? p.dh : p.x);
    a.alpha = p.alpha;
    a.h_in = static_cast<const T *>(p.h_in);
    a.h0 = p.h0;
    a.dhN = p.dhN;
    a.out = static_cast<T *>(kBack ? p.dx : p.h);
    a.dalpha = p.dalpha;
    a.last = kBack ? p.dh0 : p.hN;
    a.fold = p.fold;
    a.N = p.N;
    a.D = p.D;
    if constexpr (!kDeep)
        if (a.segs > 1) {
            const la_status st = launch<T, kBack, kTma, false, kFolds>(p, a, units, 1);
            return st == LA_OK ? launch<T, kBack, kTma, false, kSegment>(p, a, units, 1) : st;
        }
    return launch<T, kBack, kTma, kDeep, kWhole>(p, a, units, S);
}

template <typename T, bool kBack>
la_status pick(const RecurrenceProblem &p, size_t *bytes)
{
    // TMA wants rows of whole 16-byte vectors, and a sequence to describe
    if (p.D % (int)(16 / sizeof(T)) != 0 || p.N == 0) return run<T, kBack, false>(p, bytes);
    // The bf16 backward's tile is 64 KB.  Where clusters of at most two fill the machine, one
    // CTA an SM with three tiles in its ring measures 538 us at 65536 x 4096 (7.0 TB/s), two
    // CTAs with one tile each 630; with larger clusters, which then need whole groups of free
    // SMs, it is 289 against 203 us (65536 x 1024).  The other forms' tiles fit twice in 100 KB
    // (or are within 2% either way).
    if (kBack && sizeof(T) == 2 && (long long)p.B * ceil_div(p.D, 64) * 4 > tc::sm_count())
        return run<T, kBack, true, (kBack && sizeof(T) == 2)>(p, bytes);
    return run<T, kBack, true>(p, bytes);
}

// ---------------------------------------------------------------- one token
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads)
step_kernel(float *state, const T *x, const float *alpha, T *h, long long n)
{
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * kVec;
    if (i >= n) return;
    Vec<float, kVec> s = ld<float, kVec>(state + i);
    const Vec<float, kVec> al = ld<float, kVec>(alpha + i);
    const Vec<T, kVec> xv = ld<T, kVec>(x + i);
    Vec<T, kVec> o;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
        s.x[v] = fmaf(al.x[v], s.x[v], Elem<T>::to_f32(xv.x[v]));
        o.x[v] = Elem<T>::from_f32(s.x[v]);
    }
    st<float, kVec>(state + i, s);
    st<T, kVec>(h + i, o);
}

template <typename T>
la_status step(float *state, const void *x, const float *alpha, void *h, long long n, cudaStream_t s)
{
    count_launches();
    if (n % 4 == 0)
        step_kernel<T, 4><<<(unsigned)((n / 4 + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            state, static_cast<const T *>(x), alpha, static_cast<T *>(h), n);
    else
        step_kernel<T, 1><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            state, static_cast<const T *>(x), alpha, static_cast<T *>(h), n);
    return cuda_status(cudaGetLastError());
}

}  // namespace

static la_status any(const RecurrenceProblem &p, size_t *bytes)
{
    if (p.dtype == LA_BF16) return p.backward ? pick<__nv_bfloat16, true>(p, bytes) : pick<__nv_bfloat16, false>(p, bytes);
    return p.backward ? pick<float, true>(p, bytes) : pick<float, false>(p, bytes);
}
size_t recurrence_scratch(const RecurrenceProblem &p)
{
    size_t bytes = 0;
    return any(p, &bytes) == LA_OK ? bytes : 0;
}
la_status recurrence(const RecurrenceProblem &p) { return any(p, nullptr); }

la_status recurrence_read_status(cudaStream_t s, unsigned *bits)
{
    return tc::read_status(g_launched, g_rec_status, s, bits);
}

la_status recurrence_step(float *state, const void *x, const float *alpha, void *h, int B, int D, la_dtype dtype,
                          cudaStream_t stream)
{
    const long long n = (long long)B * D;
    if (dtype == LA_BF16) return step<__nv_bfloat16>(state, x, alpha, h, n, stream);
    return step<float>(state, x, alpha, h, n, stream);
}

}  // namespace la
