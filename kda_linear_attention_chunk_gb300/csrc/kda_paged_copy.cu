// kda_paged_copy.cu -- copies of position ranges between slots in several paged
// caches at once: pure data movement, bound by HBM.
//
// A page holds 2 Hk blocks (a head's keys or values) of `page` rows each; the rows of
// a range that lie in one page are one contiguous run of each block.  A warp takes
// the runs of a page one after another, kVecs 16-byte vectors a lane on their way; the
// grid is moves x caches x shares of a move's blocks of pages.  60 moves of 150 to 300
// positions in four caches (397 MB in all) take 66 us on a GB300, 6.0 TB/s; 13 of up to 5001 in
// pages of 16 small rows (114 MB) 22 us, 5.1 TB/s with the launch.
#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8, kVecs = 4;

struct CopyParams {
    SlotPools caches;
    PagedCache cache;
    const int32_t *src, *dst, *start, *end;
    int row_vecs;                    // 16-byte vectors of a row
    int *err;
};

__global__ void __launch_bounds__(kWarps * 32) pages_copy_kernel(const __grid_constant__ CopyParams p)
{
    const int m = blockIdx.y, which = blockIdx.z, lane = threadIdx.x & 31;
    const bool reports = threadIdx.x == 0 && blockIdx.x == 0 && which == 0;
    const int src = p.src[m], dst = p.dst[m];
    if (src < 0 || src >= p.cache.num_slots || dst < 0 || dst >= p.cache.num_slots) {
        if (reports && (src < -1 || src >= p.cache.num_slots || dst < -1 || dst >= p.cache.num_slots))
            atomicOr(p.err, kErrBadSlot);
        return;
    }
    const int from = p.start ? p.start[m] : 0, to = p.end[m], most = capacity(p.cache);
    const int lo = min(max(from, 0), most), hi = min(max(to, 0), most);
    if (reports && (lo != from || hi != to)) atomicOr(p.err, kErrBadPosition);
    if (src == dst || lo >= hi) return;
    const int page = 1 << p.cache.page_log2, first = lo >> p.cache.page_log2;
    const int pages = ((hi - 1) >> p.cache.page_log2) - first + 1;
    const int64_t entry = p.caches.entry_bytes[which] / 16;           // in vectors
    const int block = page * p.row_vecs, blocks = (int)(entry / block);
    uint4 *base = (uint4 *)p.caches.base[which];
    // runs: (page, block), blocks innermost
    const int64_t runs = (int64_t)pages * blocks;
    for (int64_t run = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); run < runs; run += (int64_t)gridDim.x * kWarps) {
        const int j = (int)(run / blocks), b = (int)(run - (int64_t)j * blocks);
        const int pos = (first + j) << p.cache.page_log2;
        const int a = page_at(p.cache, src, pos), z = page_at(p.cache, dst, pos);
        if (a < 0 || z < 0) {
            if (lane == 0 && b == 0 && which == 0) atomicOr(p.err, kErrBadPage);
            if (z < 0) continue;
        }
        const int r0 = max(lo - pos, 0), n = (min(hi - pos, page) - r0) * p.row_vecs;
        const uint4 *from_v = base + (int64_t)max(a, 0) * entry + (int64_t)b * block + r0 * p.row_vecs;
        uint4 *to_v = base + (int64_t)z * entry + (int64_t)b * block + r0 * p.row_vecs;
        for (int e0 = lane; e0 < n; e0 += 32 * kVecs) {
            uint4 v[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; i++)
                if (e0 + 32 * i < n) v[i] = a >= 0 ? __ldcs(from_v + e0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kVecs; i++)
                if (e0 + 32 * i < n) __stcs(to_v + e0 + 32 * i, v[i]);
        }
    }
}

}  // namespace

cudaError_t launch_pages_copy(const PagesCopyArgs &a)
{
    CopyParams p;
    p.caches = a.caches; p.cache = a.cache;
    p.src = a.src; p.dst = a.dst; p.start = a.start; p.end = a.end;
    p.row_vecs = a.row_bytes / 16; p.err = a.err_word;
    // shares of a move: as many CTAs as fill the card some times over, and no more than
    // there can be runs
    int64_t blocks = 0;
    for (int i = 0; i < a.caches.n; i++) {
        const int64_t b = a.caches.entry_bytes[i] / ((int64_t)a.row_bytes << a.cache.page_log2);
        blocks = b > blocks ? b : blocks;
    }
    const int64_t most = ((int64_t)a.cache.max_pages * blocks + kWarps - 1) / kWarps, rows = (int64_t)a.M * a.caches.n;
    int64_t shares = ((int64_t)a.num_sms * 64 + rows - 1) / rows;
    shares = shares < most ? shares : most;
    // grid.y holds 65535 moves: more take several launches
    for (int at = 0; at < a.M; at += 65535) {
        const int n = a.M - at < 65535 ? a.M - at : 65535;
        pages_copy_kernel<<<dim3((unsigned)shares, n, a.caches.n), kWarps * 32, 0, a.stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        p.src += n; p.dst += n; p.end += n;
        if (p.start) p.start += n;
    }
    return cudaSuccess;
}

}  // namespace kda
