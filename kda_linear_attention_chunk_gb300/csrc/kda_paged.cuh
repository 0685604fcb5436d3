// kda_paged.cuh -- what the kernels around paged caches share: the sequence and
// position of a row, and the page of a position.  Not installed.
#pragma once

#include <stdint.h>

#include "kda_common.cuh"
#include "kda_paged.h"
#include "kda_window.h"

namespace kda {

// positions that a table row has pages for (at most 2^30)
__device__ __forceinline__ int capacity(const PagedCache &c) { return c.max_pages << c.page_log2; }

// The page of position pos of a table row, -1 if there is none (an id out of range, or a
// position behind the table's end).
__device__ __forceinline__ int page_at(const PagedCache &c, int entry, int pos)
{
    if (pos >= capacity(c)) return -1;
    const int id = __ldg(c.table + (int64_t)entry * c.max_pages + (pos >> c.page_log2));
    return id >= 0 && id < c.num_pages ? id : -1;
}

// The last i in [0, n) with table[i] <= x, for a nondecreasing table, by a converged warp: 32
// probes at a time.  0 where there is none.
__device__ __forceinline__ int last_at_or_below(const int32_t *table, int n, int x, int lane)
{
    int a = 0;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool le = i < n && __ldg(table + a + i) <= x;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le || lane == 0));
        n = min(step, n - last * step);
        a += last * step;
    }
    return a;
}

// The sequence whose rows include row t, by a converged warp; -1: none.
__device__ __forceinline__ int sequence_with(const int32_t *cu, int N, int t, int lane)
{
    const int n = last_at_or_below(cu, N, t, lane);
    return __ldg(cu + n) <= t && t < __ldg(cu + n + 1) ? n : -1;
}

// A sequence's rows and the position of its first one, clamped: at least `least`, and all of
// them within the table where that is possible.  err: where to report, or nullptr.
struct RowsAt {
    int bos, len, start;
};
// cu0, cu1, was: the sequence's table entries as they are.
__device__ __forceinline__ RowsAt rows_at(int cu0, int cu1, int was, const PagedCache &c, int T, int least, int *err)
{
    RowsAt r;
    r.bos = clamp_row(cu0, T, err);
    r.len = max(0, clamp_row(cu1, T, err) - r.bos);
    r.start = max(least, min(was, capacity(c) - min(r.len, capacity(c))));
    if (err && r.len && (r.start != was || r.len > capacity(c) - r.start)) atomicOr(err, kErrBadPosition);
    return r;
}

}  // namespace kda
