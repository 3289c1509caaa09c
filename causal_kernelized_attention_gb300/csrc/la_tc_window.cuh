// Shared pieces of the tensor-core window-attention kernels (la_tc_window.cu,
// la_tc_window_bwd.cu): a CTA's pair of query tiles and the key tiles they reach, the mask
// as bits, and small device helpers.
#pragma once

#include <math.h>

#include "la_tc_common.cuh"
#include "la_window.cuh"

namespace la {
namespace window {

using namespace sm100;
using namespace tc;

constexpr int kRows = 128;  // rows of a query tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint64_t kDrainNs = 100000000ull;

struct Params {
    float *lse;        // forward: written; backward: read
    float *delta;      // backward: -dO . o of every row, then -lse / scale, rows of an entry `padded`
    const int *lens;
    int B, Hq, Hk, Nq, Nk, window, sinks, d;
    int padded;  // Nq rounded up to whole tiles
    int units;   // CTAs per (entry, key head)
    int pairs;   // 1: the two tiles are the same rows of heads 2i, 2i + 1 of the group; 0: neighbouring rows; 2: one tile
    float scale;
};

__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kDrainNs) {
    }
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The warp's index as a value the compiler knows to be the same in every lane, and one
// elected lane: the MMA warp's loop then runs on the uniform datapath, where descriptors
// and addresses live in the registers that tcgen05.mma reads.  (With threadIdx-derived
// branches each MMA cost about 85 cycles to issue, more than it takes to run.)
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// For the MMA warp, whose lanes must stay together: waits like wait_bar but returns nothing.
// When the wait has run out the abort flag is set, every later wait returns at once, and
// the loop ends at its next check of the flag; what is issued until then multiplies
// whatever is there, which the launch's outputs being undefined allows.
__device__ __forceinline__ void wait_or_abort(unsigned *status, int *abort_flag, uint64_t *bar, uint32_t parity)
{
    if (!mbar_try_wait(bar, parity)) wait_bar(status, abort_flag, bar, parity);
    __syncwarp();
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float &x, float &y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// This CTA's two query tiles and the key tiles either of them reaches.
template <int KT>  // keys of a tile
struct Work {
    int b, hk, h[2], t0[2], n, off;
    KeyTiles kt[2];
    int sink_end, begin, end;
    __device__ __forceinline__ static KeyTiles keys(const Params &p, int t0, int n, int off)
    {
        return KeyTiles(t0 + off, t0 < p.Nq ? min(t0 + kRows, p.Nq) - 1 + off : t0 + off - 1, p.window, p.sinks, n, KT);
    }
    // The first tile's first row, of unit u of an (entry, key head).
    __device__ __forceinline__ static int first_row(const Params &p, int u)
    {
        const int group = p.Hq / p.Hk, tiles = (p.Nq + kRows - 1) / kRows;
        if (p.pairs == 2) return u / group * kRows;
        return p.pairs ? u / (group / 2) * kRows : u % ((tiles + 1) / 2) * 2 * kRows;
    }
    __device__ __forceinline__ Work(const Params &p, int cta)
        : b(cta / p.units / p.Hk), hk(cta / p.units % p.Hk), n(valid(p.lens, b, p.Nk)), off(p.Nk - p.Nq),
          kt{{0, -1, 1, 0, 0, KT}, {0, -1, 1, 0, 0, KT}}
    {
        const int u = cta % p.units, group = p.Hq / p.Hk, tiles = (p.Nq + kRows - 1) / kRows;
        if (p.pairs == 2) {  // one query tile: unit = (row tile, head), heads of one row tile together
            h[0] = h[1] = hk * group + u % group;
            t0[0] = first_row(p, u);
            t0[1] = p.Nq;
        } else if (p.pairs) {  // unit = (row tile, head pair), pairs of one row tile together
            const int hp = u % (group / 2);
            h[0] = hk * group + 2 * hp;
            h[1] = h[0] + 1;
            t0[0] = t0[1] = first_row(p, u);
        } else {
            const int duos = (tiles + 1) / 2;
            h[0] = h[1] = hk * group + u / duos;
            t0[0] = first_row(p, u);
            t0[1] = t0[0] + kRows;
        }
        kt[0] = keys(p, t0[0], n, off);
        kt[1] = keys(p, t0[1], n, off);
        sink_end = max(kt[0].sink_end, kt[1].sink_end);
        const bool e0 = kt[0].count() == 0, e1 = kt[1].count() == 0;
        begin = max(e0 ? kt[1].begin : e1 ? kt[0].begin : min(kt[0].begin, kt[1].begin), sink_end);
        end = max(max(kt[0].end, kt[1].end), begin);
    }
    __device__ __forceinline__ int count() const { return sink_end + (end - begin); }
    __device__ __forceinline__ int tile(int u) const { return u < sink_end ? u : begin + (u - sink_end); }
    __device__ __forceinline__ bool reaches(int s, int tile) const
    {
        return tile < kt[s].sink_end || (tile >= kt[s].begin && tile < kt[s].end);
    }
};

// Bits c of the 32 keys from j on that a row at position p sees.
__device__ __forceinline__ uint32_t seen_bits(int p, int j, int window, int sinks, int n)
{
    if (p >= n) return 0u;
    const int hi = min(p - j, 31), lo = max(p - window + 1 - j, 0), sk = min(sinks - 1 - j, hi);
    const uint32_t up = hi < 0 ? 0u : 0xffffffffu >> (31 - hi);
    const uint32_t win = lo > 31 ? 0u : up & (0xffffffffu << lo);
    return win | (sk < 0 ? 0u : 0xffffffffu >> (31 - sk));
}

// The launch's sizes; the two tiles of a CTA are heads of one group where groups are even
// (they reach exactly the same key tiles), else neighbouring rows (all but one).
inline Params params_of(const WindowProblem &p, bool single = false)
{
    const int group = p.Hq / p.Hk, tiles = ceil_div(p.Nq, kRows);
    Params prm;
    prm.lse = p.lse;
    prm.delta = p.delta;
    prm.lens = p.lens;
    prm.padded = tiles * kRows;
    prm.B = p.B; prm.Hq = p.Hq; prm.Hk = p.Hk; prm.Nq = p.Nq; prm.Nk = p.Nk;
    prm.window = p.window; prm.sinks = p.sinks; prm.d = p.d;
    prm.scale = p.scale;
    prm.pairs = single ? 2 : group % 2 == 0;
    prm.units = single ? tiles * group : prm.pairs ? tiles * (group / 2) : (tiles + 1) / 2 * group;
    return prm;
}

}  // namespace window
}  // namespace la
