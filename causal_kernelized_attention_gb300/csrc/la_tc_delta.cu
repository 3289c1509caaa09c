// Gated delta rule on the tensor cores: the forward pass (bf16): the chunks' matrices, then the scan, in two
// launches or, for calls that are long enough, side by side in one.
#include "la_tc_delta_scan.cuh"

namespace la {
namespace delta {
namespace {

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
delta_scan_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const Params p,
              const uint8_t *images)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    scan_body<DK, DV, kForward>(map_q, map_k, map_v, map_o, p, p.S0, p.SN, images, nullptr, nullptr, nullptr, (int)blockIdx.x, smem_raw);
}

// Both at once, where the heads leave SMs idle: the first `workers` CTAs prepare chunks, four at a time, in the order
// in which the scans come to them, and publish each one's image (mostly read from L2); the others scan, one head
// each.  Workers wait for nobody and come first, so the scans' waits end whatever else runs on the device.
constexpr int kSets = 4;  // of four warps
template <int DK, int DV> union BothSmem {
    ScanSmem<DK, DV, kForward> scan;
    PrepSmem<DK, false> prep[kSets];
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
delta_both_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const Params p,
              uint8_t *images, unsigned *ready, int workers)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if ((int)blockIdx.x >= workers) {
        scan_body<DK, DV, kForward>(map_q, map_k, map_v, map_o, p, p.S0, p.SN, images, ready, nullptr, nullptr,
                                    (int)blockIdx.x - workers, smem_raw);
        return;
    }
    BothSmem<DK, DV> &sm = *reinterpret_cast<BothSmem<DK, DV> *>(smem_raw);
    constexpr uint32_t kColumns = kSets * prep_columns(DK, false);
    const int warp = uniform_warp(), set = warp >> 2, tid = threadIdx.x & 127;
    const int chunks = (p.N + kChunk - 1) / kChunk, heads = p.B * p.H;
    if (set < kSets && tid == 0) prepare_start(sm.prep[set]);
    if (threadIdx.x == 0) fence_mbar_init();
    if (warp == 0) {
        tmem_alloc(&sm.prep[0].tmem_base, kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    if (set < kSets) {
        PrepSmem<DK, false> &mine = sm.prep[set];
        const uint32_t tmem = sm.prep[0].tmem_base + set * prep_columns(DK, false);
        const long long items = (long long)chunks * heads, step = (long long)workers * kSets;
        long long last = -1;  // stored, not yet published
        auto publish = [&]() {
            if ((warp & 3) == 0 && elect_one() && last >= 0) {
                tma_store_wait_all();
                st_release_gpu(ready + last, 1u);
            }
            __syncwarp();
        };
        uint32_t turn = 0;
        const long long start = (long long)blockIdx.x * kSets + set;
        float2 gates = start < items ? load_gates(p, (int)(start % heads), (int)(start / heads), tid) : make_float2(0.f, 0.f);
        for (long long i = start; i < items; i += step, ++turn) {
            if (__any_sync(0xffffffffu, aborted(&mine.abort))) break;
            const int chunk = (int)(i / heads), bh = (int)(i % heads);
            const long long at = (long long)bh * chunks + chunk;
            const float2 now = gates;
            const long long next = i + step;
            if (next < items) gates = load_gates(p, (int)(next % heads), (int)(next / heads), tid);
            named_bar_sync(1 + set, 128);  // the last chunk's operands are read
            prepare_chunk<DK, false>(mine, map_q, map_k, p, images + at * Layout<DK>::forward_bytes, now, bh, chunk, tid, warp & 3, tmem, turn,
                                     true, 1 + set, true, [&] { named_bar_sync(1 + set, 128); });
            // (a chunk whose own wait has run out is not published: its scan's wait runs out, too)
            last = __any_sync(0xffffffffu, aborted(&mine.abort)) || i == p.drop ? -1 : at;
            publish();
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(sm.prep[0].tmem_base, kColumns);
}

template <int DK, int DV> la_status forward_both(const DeltaProblem &p)
{
    typedef BothSmem<DK, DV> Sm;
    static_assert(sizeof(Sm) <= 227 * 1024, "");
    const Params prm = params_of(p);
    const size_t n = (size_t)p.B * p.H * ceil_div(p.N, kChunk);
    uint8_t *images = reinterpret_cast<uint8_t *>(p.scratch);
    unsigned *ready = reinterpret_cast<unsigned *>(images + n * Layout<DK>::forward_bytes);
    CUtensorMap mq, mk, mv, mo;
    la_status st = make_map(&mq, p.q, p.B * p.Hk, p.N, p.dk, kChunk);
    if (st == LA_OK) st = make_map(&mk, p.k, p.B * p.Hk, p.N, p.dk, kChunk);
    if (st == LA_OK) st = make_map(&mv, p.v, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = make_map(&mo, p.o, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = ensure_smem((const void *)delta_both_tc<DK, DV>, (int)sizeof(Sm));
    if (st != LA_OK) return st;
    g_launched = true;
    count_launches(2);
    if ((st = cuda_status(cudaMemsetAsync(ready, 0, n * sizeof(unsigned), p.stream))) != LA_OK) return st;
    const int heads = p.B * p.H, workers = sm_count() - heads;
    return launch_dependent(delta_both_tc<DK, DV>, (unsigned)(heads + workers), kThreads, (int)sizeof(Sm), p.stream, mq, mk, mv, mo,
                            prm, images, ready, workers);
}

// One launch clears its flags and fills its pipeline first (7 us), and hides the preparing kernel behind the scan: it pays from 5
// chunks an SM, at 16 chunks a head and more (with fewer the scan is over before the rest is hidden), while half of the
// SMs are left to prepare.  One launch against two, us, d 64 / d 128: 32 heads of 8 chunks 34 / 40 against 28 / 34, of 16
// 45 / 55 against 46 / 54, of 24 57 / 73 against 60 / 77, of 64 114 / 150 against 152 / 177; 64 of 12 46 / 55 against
// 44 / 55, of 16 53 / 64 against 55 / 67, of 64 146 / 170 against 184 / 218; 8 of 32 66 / 83 against 60 / 79, of
// 64 110 / 144 against 125 / 144; 90 of 64 261 / 293 against 208 / 250.
bool one_launch(const DeltaProblem &p)
{
    const long long heads = (long long)p.B * p.H, chunks = ceil_div(p.N, kChunk);
    return heads * 2 <= sm_count() && chunks >= 16 && heads * chunks >= 5LL * sm_count();
}

template <int DK, int DV> la_status forward(const DeltaProblem &p)
{
    if (one_launch(p)) return forward_both<DK, DV>(p);
    typedef ScanSmem<DK, DV, kForward> Sm;
    static_assert(sizeof(Sm) <= 227 * 1024, "");
    const Params prm = params_of(p);
    uint8_t *images = reinterpret_cast<uint8_t *>(p.scratch);
    CUtensorMap mq, mk, mv, mo;
    la_status st = make_map(&mv, p.v, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = make_map(&mo, p.o, p.B * p.H, p.N, p.dv, kChunk);
    if (st == LA_OK) st = ensure_smem((const void *)delta_scan_tc<DK, DV>, (int)sizeof(Sm));
    if (st == LA_OK) st = prepare<DK, false>(p, prm, images, &mq, &mk);
    if (st != LA_OK) return st;
    count_launches();
    return launch_dependent(delta_scan_tc<DK, DV>, (unsigned)(p.B * p.H), kThreads, (int)sizeof(Sm), p.stream, mq, mk, mv, mo, prm,
                            (const uint8_t *)images);
}

}  // namespace
}  // namespace delta

using namespace delta;

bool delta_tc_eligible(const DeltaProblem &p)
{
    return p.dtype == LA_BF16 && p.N > 0;
}

size_t delta_forward_tc_scratch(const DeltaProblem &p)
{
    return (size_t)p.B * p.H * ceil_div(p.N, kChunk) *
           ((p.dk <= 64 ? Layout<64>::forward_bytes : Layout<128>::forward_bytes) + sizeof(unsigned));
}

la_status delta_forward_tc(const DeltaProblem &p)
{
    if (p.dk <= 64) return p.dv <= 64 ? forward<64, 64>(p) : forward<64, 128>(p);
    return p.dv <= 64 ? forward<128, 64>(p) : forward<128, 128>(p);
}

la_status tc_delta_read_status(cudaStream_t s, unsigned *bits) { return read_status(g_launched, g_delta_status, s, bits); }

}  // namespace la
