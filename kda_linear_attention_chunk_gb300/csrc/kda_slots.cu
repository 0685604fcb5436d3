// kda_slots.cu -- copies, clears and compaction of slot entries in several pools
// at once: pure data movement, bound by HBM.
//
// The work is cut into pieces of kPiece bytes of one entry; a CTA copies one
// piece with four 16-byte loads in flight per thread.  Pieces are ordered with
// the moves innermost, so the forks of one source read each of its pieces
// together (from L2 after the first).  16 forks of 12.7 MB each take 41.7 us on a GB300,
// 6.1 TB/s of algorithmic bytes (32 KB pieces 43.5 us).
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_hybrid.h"
#include "kda_pdl.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                              // 16-byte vectors per thread and piece
constexpr int64_t kPiece = kThreads * kVecs * 16;     // 16 KB

struct MoveParams {
    SlotPools pools;
    const int32_t *src, *dst;
    int M, num_slots;
    int64_t pieces;              // of one entry of every pool
    int *err;
};

__global__ void __launch_bounds__(kThreads) move_kernel(const __grid_constant__ MoveParams p)
{
    grid_wait();                                      // for the plan, where there is one
    const int64_t items = p.pieces * p.M;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        int64_t piece = item / p.M;
        const int m = (int)(item - piece * p.M);
        const int src = p.src[m], dst = p.dst[m];
        if (src < -1 || src >= p.num_slots || dst < -1 || dst >= p.num_slots) {
            if (piece == 0 && threadIdx.x == 0) atomicOr(p.err, kErrBadSlot);
            continue;
        }
        if (dst < 0 || src == dst) continue;
        int i = 0;
        for (;; i++) {
            const int64_t n = (p.pools.entry_bytes[i] + kPiece - 1) / kPiece;
            if (piece < n) break;
            piece -= n;
        }
        const int64_t bytes = p.pools.entry_bytes[i], at = piece * kPiece;
        const int n = (int)((bytes - at < kPiece ? bytes - at : kPiece) / 16);
        uint8_t *base = (uint8_t *)p.pools.base[i] + at;
        uint4 *to = (uint4 *)(base + dst * bytes);
        uint4 r[kVecs];
        if (src >= 0) {
            const uint4 *from = (const uint4 *)(base + src * bytes);
#pragma unroll
            for (int j = 0; j < kVecs; j++) {
                const int e = threadIdx.x + j * kThreads;
                if (e < n) r[j] = from[e];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVecs; j++) r[j] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kVecs; j++) {
            const int e = threadIdx.x + j * kThreads;
            if (e < n) to[e] = r[j];
        }
    }
}

// The plan of a compaction, one CTA: a bitmap of the live ids, the number of
// live ids before each of its words, and from both the rank of an id among the
// high ones (>= m) and the free id below m of the same rank.
constexpr int kPlanThreads = 1024;
constexpr int kMaxPlanBytes = kMaxPoolSlots / 32 * 8;

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const int32_t *slots, int32_t *new_slots, int N, int num_slots, int *err)
{
    extern __shared__ uint32_t sm[];
    grid_go_on();
    const int words = (num_slots + 31) / 32, tid = threadIdx.x;
    uint32_t *map = sm, *before = sm + words;     // before[w]: live ids in words < w
    __shared__ uint32_t part[kPlanThreads / 32];
    __shared__ uint32_t total;
    for (int w = tid; w < words; w += kPlanThreads) map[w] = 0;
    __syncthreads();
    for (int i = tid; i < N; i += kPlanThreads) {
        const int s = slots[i];
        if (s >= 0 && s < num_slots) atomicOr(&map[s >> 5], 1u << (s & 31));
        else if (s != -1) atomicOr(err, kErrBadSlot);
    }
    __syncthreads();
    // each thread takes a run of words; exclusive scan of the runs' counts
    const int run = (words + kPlanThreads - 1) / kPlanThreads, w0 = min(words, tid * run), w1 = min(words, w0 + run);
    uint32_t mine = 0;
    for (int w = w0; w < w1; w++) mine += __popc(map[w]);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if ((tid & 31) >= o) inc += x;
    }
    if ((tid & 31) == 31) part[tid >> 5] = inc;
    __syncthreads();
    if (tid < 32) {
        uint32_t x = part[tid];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (tid >= o) x += y;
        }
        part[tid] = x;
        if (tid == 31) total = x;
    }
    __syncthreads();
    uint32_t at = inc - mine + (tid >= 32 ? part[(tid >> 5) - 1] : 0);
    for (int w = w0; w < w1; w++) {
        before[w] = at;
        at += __popc(map[w]);
    }
    __syncthreads();
    const int m = (int)total;                     // live ids
    // live ids below x
    auto live_below = [&](int x) {
        return x >= words * 32 ? m : (int)(before[x >> 5] + __popc(map[x >> 5] & ((1u << (x & 31)) - 1)));
    };
    const int low = live_below(m);
    for (int i = tid; i < N; i += kPlanThreads) {
        const int s = slots[i];
        int to = s;
        if (s < 0 || s >= num_slots) {
            to = -1;
        } else if (s >= m) {
            const int rank = live_below(s) - low;  // among the high ids
            int a = 0, b = words - 1;              // the last word with at most `rank` free ids before it
            while (a < b) {
                const int c = (a + b + 1) / 2;
                if (32 * c - (int)before[c] <= rank) a = c; else b = c - 1;
            }
            uint32_t free_bits = ~map[a];
            for (int k = rank - (32 * a - (int)before[a]); k > 0; k--) free_bits &= free_bits - 1;
            to = 32 * a + __ffs(free_bits) - 1;
        }
        new_slots[i] = to;
    }
}

// planned: behind the plan kernel, whose end its CTAs, already there, wait for
cudaError_t move(const SlotMoveArgs &a, bool planned)
{
    MoveParams p;
    p.pools = a.pools;
    p.src = a.src; p.dst = a.dst; p.M = a.M; p.num_slots = a.num_slots; p.err = a.err_word;
    p.pieces = 0;
    for (int i = 0; i < a.pools.n; i++) p.pieces += (a.pools.entry_bytes[i] + kPiece - 1) / kPiece;
    const int64_t items = p.pieces * a.M, most = (int64_t)a.num_sms * 64;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items < most ? items : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = planned;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, move_kernel, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_slots_copy(const SlotMoveArgs &a) { return move(a, false); }

cudaError_t launch_slots_compact(const SlotMoveArgs &a)
{
    const size_t smem = (size_t)((a.num_slots + 31) / 32) * 2 * sizeof(uint32_t);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, a.device, []() {
        return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxPlanBytes);
    });
    if (e != cudaSuccess) return e;
    plan_kernel<<<1, kPlanThreads, smem, a.stream>>>(a.src, a.new_slots, a.M, a.num_slots, a.err_word);
    e = cudaGetLastError();
    return e == cudaSuccess ? move(a, true) : e;
}

}  // namespace kda
