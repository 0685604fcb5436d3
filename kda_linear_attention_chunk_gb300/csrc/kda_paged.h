// kda_paged.h -- launch interface of the kernels around paged caches and beams
// (kda_paged_append.cu, kda_paged_copy.cu, kda_paged_attention.cu, kda_beam.cu) for
// the C ABI (kda_api_paged.cu).  Not installed; the public interface is include/kda.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_hybrid.h"

namespace kda {

// A page id outside [0, num_pages) where a page was needed.
constexpr int kErrBadPage = 128;

// a paged cache's pages and page table
struct PagedCache {
    uint16_t *pages;                 // [num_pages][2 (k, v)][Hk][page][d]
    const int32_t *table;            // [num_slots][max_pages]
    int num_pages, page_log2, num_slots, max_pages;
};

struct PagedAppendArgs {
    const void *q, *k, *v;           // rows of [Hq|Hk|Hk][d], strides in elements
    int64_t q_stride, k_stride, v_stride;
    const float *q_weight, *k_weight;   // [d] or nullptr (ones)
    const float *angles;             // [max_pos][rotary]: cos | sin
    const int32_t *cu_seqlens;       // [N+1], or nullptr: a row each
    const int32_t *starts, *slots;   // [N] or nullptr
    PagedCache cache;
    void *q_out;                     // [T][Hq][d]
    int N, T, Hq, Hk, d, rotary, max_pos, layout, norm;
    float eps;
    bool f16;
    cudaStream_t stream;
    int *err_word;
};
cudaError_t launch_paged_append(const PagedAppendArgs &a);

struct PagedAttentionArgs {
    const void *q;
    int64_t q_stride;
    const int32_t *cu_seqlens, *starts, *slots;
    PagedCache cache;
    const int32_t *groups, *prefix_lens, *prefix_slots;   // [P+1], [P], [P]; P = 0: nullptr
    void *out;
    void *workspace;
    int N, T, P, Hq, Hk, d;
    float scale;
    bool f16;
    int device, num_sms;
    cudaStream_t stream;
    int *err_word;
};
int64_t paged_attention_workspace(int N, int T, int P, int Hq, int Hk, int d);
cudaError_t launch_paged_attention(const PagedAttentionArgs &a);

struct PagesCopyArgs {
    SlotPools caches;                // entries are pages
    PagedCache cache;                // the table that they share (no pages here)
    const int32_t *src, *dst, *start, *end;
    int M, row_bytes;
    int num_sms;
    cudaStream_t stream;
    int *err_word;
};
cudaError_t launch_pages_copy(const PagesCopyArgs &a);

struct BeamArgs {
    const void *logits;
    int64_t row_stride;
    int dtype;                       // kda_dtype
    const float *scores;
    const int32_t *ended;
    int end_token;
    const int32_t *slots;
    float *scores_out;
    int32_t *parents, *tokens, *ended_out, *new_slots, *src, *dst;
    void *workspace;
    int G, B, V;
    cudaStream_t stream;
};
int64_t beam_workspace(int G, int B, int V);
cudaError_t launch_beam_select(const BeamArgs &a);

}  // namespace kda
