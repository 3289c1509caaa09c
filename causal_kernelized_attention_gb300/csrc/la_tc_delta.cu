// Gated delta rule on the tensor cores: the forward pass (bf16), two launches: the
// chunks' matrices, then the scan.
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
    scan_body<DK, DV, kForward>(map_q, map_k, map_v, map_o, p, p.S0, p.SN, images, nullptr, nullptr, (int)blockIdx.x, smem_raw);
}

template <int DK, int DV> la_status forward(const DeltaProblem &p)
{
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
    return (size_t)p.B * p.H * ceil_div(p.N, kChunk) * (p.dk <= 64 ? Layout<64>::forward_bytes : Layout<128>::forward_bytes);
}

la_status delta_forward_tc(const DeltaProblem &p)
{
    if (p.dk <= 64) return p.dv <= 64 ? forward<64, 64>(p) : forward<64, 128>(p);
    return p.dv <= 64 ? forward<128, 64>(p) : forward<128, 128>(p);
}

la_status tc_delta_read_status(cudaStream_t s, unsigned *bits) { return read_status(g_launched, g_delta_status, s, bits); }

}  // namespace la
