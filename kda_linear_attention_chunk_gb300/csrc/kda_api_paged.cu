// kda_api_paged.cu -- the C ABI of the kernels around paged caches and beams
// (include/kda.h): argument validation and dispatch.  Validation is synchronous and
// happens before any CUDA call, as in kda_api.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_paged.h"

namespace {

using namespace kda::checks;

// the page table and, where there are any, the pages; *log2: of the page's rows
int check_table(int num_pages, int page, int num_slots, int max_pages, int *log2)
{
    if (num_pages < 1 || page < 1 || num_slots < 1 || max_pages < 1) return KDA_ERR_SHAPE;
    if (page < 16 || page > 256 || (page & (page - 1))) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page > (1 << 30)) return KDA_ERR_SHAPE;   // so that a tile behind any position fits in 32 bits
    if ((double)num_slots * max_pages * 4 >= (double)kMaxBytes) return KDA_ERR_SHAPE;
    for (*log2 = 4; 1 << *log2 < page;) ++*log2;
    return KDA_OK;
}

int64_t table_bytes(int num_slots, int max_pages) { return (int64_t)num_slots * max_pages * 4; }

// the pages' size in bytes, or -1
int64_t pages_bytes(int num_pages, int page, int Hk, int d)
{
    const double bytes = (double)num_pages * 2 * Hk * page * d * 2;
    if (bytes >= (double)kMaxBytes || (double)num_pages * 2 * Hk > 2147483647.0) return -1;
    return (int64_t)num_pages * 2 * Hk * page * d * 2;
}

}  // namespace

extern "C" {

int kda_paged_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                     int64_t v_stride, const float *q_weight, const float *k_weight, const float *table,
                     int max_pos, const int32_t *cu_seqlens, const int32_t *starts, const int32_t *slots,
                     void *kv_pages, int num_pages, int page, const int32_t *page_table, int num_slots,
                     int max_pages, void *q_out, int N, int T, int Hq, int Hk, int d, int rotary, int layout,
                     int norm, float eps, int dtype, void *stream)
{
    if (!kv_pages || !page_table || (T > 0 && (!q || !k || !v || !q_out || (rotary > 0 && !table)))) return KDA_ERR_NULL;
    if (N < 1 || T < 0 || rotary < 0 || (rotary > 0 && max_pos < 1) || (!cu_seqlens && T != N)) return KDA_ERR_SHAPE;
    int st = check_heads(Hq, Hk, d, dtype), log2;
    if (st != KDA_OK) return st;
    if ((st = check_table(num_pages, page, num_slots, max_pages, &log2)) != KDA_OK) return st;
    if (rotary > d || (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED) || (norm != 0 && norm != 1) ||
        !(eps >= 0.f && eps <= 3.0e38f) || (!slots && num_slots < N))
        return KDA_ERR_SHAPE;
    if (rotary % 16) return KDA_ERR_UNSUPPORTED;
    const int64_t wq = (int64_t)Hq * d, wk = (int64_t)Hk * d, cache = pages_bytes(num_pages, page, Hk, d);
    if (cache < 0 || (int64_t)max_pos * rotary * 4 >= kMaxBytes) return KDA_ERR_SHAPE;
    const int rows[] = {check_rows(T, q_stride, wq), check_rows(T, k_stride, wk), check_rows(T, v_stride, wk)};
    for (const int s : rows)
        if (s == KDA_ERR_SHAPE) return s;
    for (const int s : rows)
        if (s != KDA_OK) return s;
    const void *tensors[] = {q, k, v, q_weight, k_weight, table, kv_pages, q_out};
    for (const void *p : tensors)
        if (misaligned(p, 16)) return KDA_ERR_ALIGN;
    const void *tables[] = {cu_seqlens, starts, slots, page_table};
    for (const void *p : tables)
        if (misaligned(p, 4)) return KDA_ERR_ALIGN;
    const Span iq = span(q, strided_bytes(T, q_stride, wq)), out = span(q_out, T * wq * 2), pool = span(kv_pages, cache);
    const Span in[] = {span(k, strided_bytes(T, k_stride, wk)), span(v, strided_bytes(T, v_stride, wk)),
                       span(q_weight, (int64_t)d * 4), span(k_weight, (int64_t)d * 4),
                       span(table, (int64_t)max_pos * rotary * 4), span(cu_seqlens, ((int64_t)N + 1) * 4),
                       span(starts, (int64_t)N * 4), span(slots, (int64_t)N * 4),
                       span(page_table, table_bytes(num_slots, max_pages))};
    for (const Span &s : in)
        if (overlap(out, s) || overlap(pool, s)) return KDA_ERR_ALIAS;
    // in place only where the rows lie the same way: each vector is read whole before it is written
    if ((overlap(out, iq) && !(q == q_out && q_stride == wq)) || overlap(pool, iq) || overlap(out, pool)) return KDA_ERR_ALIAS;
    kda::PagedAppendArgs a;
    int device, sms;
    if ((st = kda::device_facts(&device, &sms, &a.err_word)) != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.q_weight = q_weight; a.k_weight = k_weight; a.angles = table;
    a.cu_seqlens = cu_seqlens; a.starts = starts; a.slots = slots;
    a.cache = {(uint16_t *)kv_pages, page_table, num_pages, log2, num_slots, max_pages};
    a.q_out = q_out;
    a.N = N; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rotary = rotary; a.max_pos = max_pos; a.layout = layout;
    a.norm = norm; a.eps = eps; a.f16 = dtype == KDA_F16;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_paged_append(a));
}

int64_t kda_paged_attention_workspace(int N, int T, int P, int Hq, int Hk, int d)
{
    if (N < 1 || T < 0 || P < 0 || check_heads(Hq, Hk, d, KDA_BF16) != KDA_OK || Hq % Hk || Hq / Hk > 128) return -1;
    return kda::paged_attention_workspace(N, T, P, Hq, Hk, d);
}

int kda_paged_attention(const void *q, int64_t q_stride, const int32_t *cu_seqlens, const int32_t *starts,
                        const int32_t *slots, const void *kv_pages, int num_pages, int page,
                        const int32_t *page_table, int num_slots, int max_pages, const int32_t *groups,
                        const int32_t *prefix_lens, const int32_t *prefix_slots, int P, void *out, void *workspace,
                        int64_t workspace_bytes, int N, int T, int Hq, int Hk, int d, float scale, int dtype,
                        void *stream)
{
    if (!kv_pages || !page_table || (T > 0 && (!q || !out))) return KDA_ERR_NULL;
    if (P > 0 ? !groups || !prefix_lens || !prefix_slots : groups || prefix_lens || prefix_slots) return KDA_ERR_NULL;
    if (N < 1 || T < 0 || P < 0 || (!cu_seqlens && T != N)) return KDA_ERR_SHAPE;
    int st = check_heads(Hq, Hk, d, dtype), log2;
    if (st != KDA_OK) return st;
    if (Hq % Hk) return KDA_ERR_SHAPE;
    if (Hq / Hk > 128) return KDA_ERR_UNSUPPORTED;
    if ((st = check_table(num_pages, page, num_slots, max_pages, &log2)) != KDA_OK) return st;
    if (!(scale > 0.f && scale <= 1.0e37f) || (!slots && num_slots < N)) return KDA_ERR_SHAPE;   // also rejects NaN
    const int64_t wq = (int64_t)Hq * d, cache = pages_bytes(num_pages, page, Hk, d);
    const int64_t needed = kda::paged_attention_workspace(N, T, P, Hq, Hk, d);
    if (cache < 0 || needed < 0) return KDA_ERR_SHAPE;
    if ((st = check_rows(T, q_stride, wq)) != KDA_OK) return st;
    if (needed > 0 && !workspace) return KDA_ERR_NULL;
    if (workspace_bytes < needed) return KDA_ERR_SHAPE;
    const void *tensors[] = {q, kv_pages, out, workspace};
    for (const void *p : tensors)
        if (misaligned(p, 16)) return KDA_ERR_ALIGN;
    const void *tables[] = {cu_seqlens, starts, slots, page_table, groups, prefix_lens, prefix_slots};
    for (const void *p : tables)
        if (misaligned(p, 4)) return KDA_ERR_ALIGN;
    const Span to = span(out, T * wq * 2), work = span(workspace, needed);
    const Span in[] = {span(q, strided_bytes(T, q_stride, wq)), span(kv_pages, cache), span(cu_seqlens, ((int64_t)N + 1) * 4),
                       span(starts, (int64_t)N * 4), span(slots, (int64_t)N * 4),
                       span(page_table, table_bytes(num_slots, max_pages)), span(groups, ((int64_t)P + 1) * 4),
                       span(prefix_lens, (int64_t)P * 4), span(prefix_slots, (int64_t)P * 4)};
    for (const Span &s : in)
        if (overlap(to, s) || overlap(work, s)) return KDA_ERR_ALIAS;
    if (overlap(to, work)) return KDA_ERR_ALIAS;
    kda::PagedAttentionArgs a;
    if ((st = kda::device_facts(&a.device, &a.num_sms, &a.err_word)) != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    a.q = q; a.q_stride = q_stride;
    a.cu_seqlens = cu_seqlens; a.starts = starts; a.slots = slots;
    a.cache = {(uint16_t *)kv_pages, page_table, num_pages, log2, num_slots, max_pages};
    a.groups = groups; a.prefix_lens = prefix_lens; a.prefix_slots = prefix_slots;
    a.out = out; a.workspace = workspace;
    a.N = N; a.T = T; a.P = P; a.Hq = Hq; a.Hk = Hk; a.d = d; a.scale = scale; a.f16 = dtype == KDA_F16;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_paged_attention(a));
}

int kda_pages_copy(const kda_pool *caches, int num_caches, int num_pages, int page, int row_bytes,
                   const int32_t *page_table, int num_slots, int max_pages, const int32_t *src, const int32_t *dst,
                   const int32_t *start, const int32_t *end, int M, void *stream)
{
    if (!caches || !page_table || !src || !dst || !end) return KDA_ERR_NULL;
    if (M < 1 || row_bytes < 1) return KDA_ERR_SHAPE;
    kda::PagesCopyArgs a;
    int st = check_pools(caches, num_caches, num_pages, 0x7fffffff, &a.caches), log2;
    if (st != KDA_OK) return st;
    if ((st = check_table(num_pages, page, num_slots, max_pages, &log2)) != KDA_OK) return st;
    if (row_bytes > 1024) return KDA_ERR_UNSUPPORTED;
    if (row_bytes % 16) return KDA_ERR_ALIGN;
    const int64_t block = (int64_t)row_bytes * page;
    for (int i = 0; i < num_caches; i++)
        if (a.caches.entry_bytes[i] % block || a.caches.entry_bytes[i] / block > (1 << 20)) return KDA_ERR_SHAPE;
    const int32_t *tables[] = {page_table, src, dst, start, end};
    for (const void *p : tables)
        if (misaligned(p, 4)) return KDA_ERR_ALIGN;
    if (in_pools(a.caches, num_pages, span(page_table, table_bytes(num_slots, max_pages)))) return KDA_ERR_ALIAS;
    for (int i = 1; i < 5; i++)
        if (in_pools(a.caches, num_pages, span(tables[i], (int64_t)M * 4))) return KDA_ERR_ALIAS;
    int device;
    if ((st = kda::device_facts(&device, &a.num_sms, &a.err_word)) != KDA_OK) return st;
    a.cache = {nullptr, page_table, num_pages, log2, num_slots, max_pages};
    a.src = src; a.dst = dst; a.start = start; a.end = end; a.M = M; a.row_bytes = row_bytes;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_pages_copy(a));
}

int64_t kda_beam_select_workspace(int G, int B, int V) { return kda::beam_workspace(G, B, V); }

int kda_beam_select(const void *logits, int64_t row_stride, int dtype, const float *scores, const int32_t *ended,
                    int end_token, const int32_t *slots, float *scores_out, int32_t *parents, int32_t *tokens,
                    int32_t *ended_out, int32_t *new_slots, int32_t *src, int32_t *dst, void *workspace,
                    int64_t workspace_bytes, int G, int B, int V, void *stream)
{
    if (!logits || !scores || !scores_out || !parents || !tokens || !workspace) return KDA_ERR_NULL;
    if ((ended || ended_out) && end_token < 0) return KDA_ERR_SHAPE;
    if (!ended != !ended_out && !ended_out) return KDA_ERR_NULL;
    if (slots ? !new_slots || !src || !dst : new_slots || src || dst) return KDA_ERR_NULL;
    if (G < 1 || B < 1 || V < 1 || end_token < -1 || end_token >= V) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_F16 && dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
    if (B > 64 || V > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    const int64_t needed = kda::beam_workspace(G, B, V), rows = (int64_t)G * B;
    const int size = dtype == KDA_F32 ? 4 : 2;
    if (needed < 0 || workspace_bytes < needed) return KDA_ERR_SHAPE;
    if (row_stride < V || row_stride >= kMaxBytes || (double)rows * row_stride * size >= (double)kMaxBytes) return KDA_ERR_SHAPE;
    if (misaligned(workspace, 16) || misaligned(logits, size)) return KDA_ERR_ALIGN;
    const void *in4[] = {scores, ended, slots};
    const void *out4[] = {scores_out, parents, tokens, ended_out, new_slots, src, dst};
    Span out[8];
    for (int i = 0; i < 7; i++) {
        if (misaligned(out4[i], 4)) return KDA_ERR_ALIGN;
        out[i] = span(out4[i], rows * 4);
    }
    out[7] = span(workspace, needed);
    for (int i = 0; i < 8; i++) {
        if (overlap(out[i], span(logits, ((rows - 1) * row_stride + V) * size))) return KDA_ERR_ALIAS;
        for (const void *p : in4) {
            if (misaligned(p, 4)) return KDA_ERR_ALIGN;
            if (overlap(out[i], span(p, rows * 4))) return KDA_ERR_ALIAS;
        }
        for (int j = 0; j < i; j++)
            if (overlap(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    int device, sms, *word, st;
    if ((st = kda::device_facts(&device, &sms, &word)) != KDA_OK) return st;
    kda::BeamArgs a;
    a.logits = logits; a.row_stride = row_stride; a.dtype = dtype;
    a.scores = scores; a.ended = ended; a.end_token = end_token; a.slots = slots;
    a.scores_out = scores_out; a.parents = parents; a.tokens = tokens; a.ended_out = ended_out;
    a.new_slots = new_slots; a.src = src; a.dst = dst; a.workspace = workspace;
    a.G = G; a.B = B; a.V = V;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_beam_select(a));
}

}  // extern "C"
