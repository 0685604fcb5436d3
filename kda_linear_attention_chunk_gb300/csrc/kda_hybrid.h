// kda_hybrid.h -- launch interface of the kernels around a hybrid stack's
// softmax layers (kda_norm_rope.cu, kda_window.cu, kda_window_rows.cu,
// kda_slots.cu) for the C ABI (kda_api_hybrid.cu).  Not installed; the public
// interface is include/kda.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kda {

// A position or context length outside its range (clamped): the bit of the
// sticky device error word that only these kernels set.
constexpr int kErrBadPosition = 64;

// kda_api.cu: ordinal (below 64), SM count and error word of the current device
// (checked to be an sm_103 device); returns a kda_status
int device_facts(int *device, int *num_sms, int **err_word);

// Runs `prepare` (a kernel's attributes) once for each device; a failure is
// returned and tried again by the next call.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &done, int device, F prepare)
{
    const uint64_t bit = (uint64_t)1 << device;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    const cudaError_t e = prepare();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// per-head RMS norm and rotation of q and k
struct NormRopeArgs {
    const void *q, *k;               // rows of [Hq|Hk][d], q_stride / k_stride elements apart
    int64_t q_stride, k_stride;
    const float *q_weight, *k_weight;   // [d] or nullptr (ones)
    const float *table;              // [max_pos][rotary]: cos | sin
    const int32_t *positions;        // [T]
    void *q_out, *k_out;             // [T][Hq|Hk][d]
    int T, Hq, Hk, d, rotary, max_pos, layout, norm;
    float eps;
    bool f16;
    cudaStream_t stream;
    int *err_word;
};
cudaError_t launch_norm_rope(const NormRopeArgs &a);

// attention over a sliding window and the first `sinks` positions
struct WindowArgs {
    const void *q, *k, *v;           // rows of [Hq|Hk|Hk][d], strides in elements
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_seqlens;       // [N+1] (prefill)
    const int32_t *starts;           // [N] positions before the first row, or nullptr (0)
    const int32_t *slots;            // [N] or nullptr (entry n)
    void *pool;                      // [num_slots][2][Hk][pool_rows][d] or nullptr (prefill without a cache)
    void *out;                       // [T][Hq][d]
    int N, T, Hq, Hk, d, num_slots, pool_rows, window, sinks;
    float scale;
    bool f16;
    int device, num_sms;
    cudaStream_t stream;
    int *err_word;
};
cudaError_t launch_window_prefill(const WindowArgs &a);
cudaError_t launch_window_decode(const WindowArgs &a);   // T unused; starts = the tokens' positions

// moves of slot entries in several pools at once
constexpr int kMaxPools = 128, kMaxPoolSlots = 524288;
struct SlotPools {
    void *base[kMaxPools];
    int64_t entry_bytes[kMaxPools];
    int n;
};
struct SlotMoveArgs {
    SlotPools pools;
    const int32_t *src, *dst;        // [M]
    int32_t *new_slots;              // compaction: written from src by the plan kernel, then used as dst
    int M, num_slots;
    int device, num_sms;
    cudaStream_t stream;
    int *err_word;
};
cudaError_t launch_slots_copy(const SlotMoveArgs &a);
cudaError_t launch_slots_compact(const SlotMoveArgs &a);

}  // namespace kda
