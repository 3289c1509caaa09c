// What the window-attention kernels share: which keys a query sees.
//
// Query row t of an entry with n valid tokens stands at position p = t + off (off =
// Nk - Nq: the queries are the last ones of the keys) and sees the keys j <= p with
// p - j < window or j < sinks; rows at p >= n are padding and see nothing.
#pragma once

#include "la_common.cuh"
#include "la_internal.h"

namespace la {
namespace window {

// Valid tokens of batch entry b.
__device__ __forceinline__ int valid(const int *lens, int b, int Nk)
{
    return lens ? min(max(__ldg(lens + b), 0), Nk) : Nk;
}

__device__ __forceinline__ bool sees(int p, int j, int window, int sinks, int n)
{
    return j <= p && p < n && (p - j < window || j < sinks);
}

// The key tiles (T keys each) that rows at positions [p0, p1] reach: the tiles of sinks
// [0, sink_end) and those of the window [begin, end), in this order and disjoint.
struct KeyTiles {
    int sink_end, begin, end;
    __device__ __forceinline__ KeyTiles(int p0, int p1, int window, int sinks, int n, int T)
    {
        p1 = min(p1, n - 1);
        if (p1 < p0) {
            sink_end = begin = end = 0;
            return;
        }
        end = p1 / T + 1;
        begin = max(p0 - window + 1, 0) / T;
        sink_end = min((min(sinks, p1 + 1) + T - 1) / T, end);
        begin = max(begin, sink_end);
        end = max(end, begin);
    }
    __device__ __forceinline__ int count() const { return sink_end + (end - begin); }
    __device__ __forceinline__ int tile(int i) const { return i < sink_end ? i : begin + (i - sink_end); }
};

// The query tiles (T rows each, by row index t) that see a key of [j0, j1]: [begin, end).
struct QueryTiles {
    int begin, end;
    __device__ __forceinline__ QueryTiles(int j0, int j1, int window, int sinks, int n, int off, int Nq, int T)
    {
        j1 = min(j1, n - 1);
        int last = j0 < sinks ? n - 1 : min(n - 1, j1 + window - 1);  // the last position that sees one
        last = min(last - off, Nq - 1);
        const int first = max(j0 - off, 0);
        begin = first / T;
        end = j1 < j0 || last < first ? begin : last / T + 1;
    }
};

}  // namespace window
}  // namespace la
