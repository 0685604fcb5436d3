// kda_api_hybrid.cu -- the C ABI of the kernels around a hybrid stack's softmax
// layers (include/kda.h): argument validation and dispatch.  Validation is
// synchronous and happens before any CUDA call, as in kda_api.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_hybrid.h"

namespace {

static_assert(kda::kMaxPools == KDA_MAX_POOLS && kda::kMaxPoolSlots == KDA_MAX_POOL_SLOTS, "the header's limits");

constexpr int64_t kMaxBytes = (int64_t)1 << 40;   // a tensor's span; keeps every product below in 64 bits

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

Span span(const void *p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (p && bytes > 0 ? (uintptr_t)bytes : 0)}; }
bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
bool misaligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

// rows of `width` elements, `stride` apart, 2 bytes an element
int64_t strided_bytes(int T, int64_t stride, int64_t width) { return T > 0 ? ((T - 1) * stride + width) * 2 : 0; }

// row widths and strides: whole 16-byte pieces, rows that do not overlap
int check_rows(int T, int64_t stride, int64_t width)
{
    if (stride < width || stride >= ((int64_t)1 << 31)) return KDA_ERR_SHAPE;
    if (T > 0 && (int64_t)T * stride * 2 >= kMaxBytes) return KDA_ERR_SHAPE;
    return stride % 8 ? KDA_ERR_ALIGN : KDA_OK;
}

int check_heads(int Hq, int Hk, int d, int dtype)
{
    if (Hq < 1 || Hk < 1 || Hq > (1 << 16) || Hk > (1 << 16) || d < 1) return KDA_ERR_SHAPE;
    if ((d != 64 && d != 128) || (dtype != KDA_BF16 && dtype != KDA_F16)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// what the two attention calls share; rows = T (prefill) or N (decode)
int check_window(const kda::WindowArgs &a, int rows, int dtype)
{
    int st = check_heads(a.Hq, a.Hk, a.d, dtype);
    if (st != KDA_OK) return st;
    if (a.Hq % a.Hk || a.window < 1 || a.sinks < 0) return KDA_ERR_SHAPE;
    if (!(a.scale > 0.f && a.scale <= 1.0e37f)) return KDA_ERR_SHAPE;   // also rejects NaN
    if (a.Hq / a.Hk > 128) return KDA_ERR_UNSUPPORTED;
    const int64_t wq = (int64_t)a.Hq * a.d, wk = (int64_t)a.Hk * a.d;
    const int64_t strides[] = {a.q_stride, a.k_stride, a.v_stride};
    int64_t pool_bytes = 0;
    for (int i = 0; i < 3; i++)
        if ((st = check_rows(rows, strides[i], i ? wk : wq)) != KDA_OK && st != KDA_ERR_ALIGN) return st;
    if (a.pool) {
        if (a.num_slots < 1 || (!a.slots && a.num_slots < a.N)) return KDA_ERR_SHAPE;
        if ((int64_t)a.window + a.sinks > a.pool_rows) return KDA_ERR_SHAPE;
        if ((int64_t)a.num_slots * 2 * a.Hk > 0x7fffffff) return KDA_ERR_SHAPE;
        const double bytes = (double)a.num_slots * 2 * (double)wk * a.pool_rows * 2;
        if (bytes >= (double)kMaxBytes) return KDA_ERR_SHAPE;
        pool_bytes = (int64_t)a.num_slots * 2 * wk * a.pool_rows * 2;
    }
    for (const int64_t s : strides)
        if (s % 8) return KDA_ERR_ALIGN;
    const void *tensors[] = {a.q, a.k, a.v, a.out, a.pool};
    for (const void *p : tensors)
        if (misaligned(p, 16)) return KDA_ERR_ALIGN;
    const void *tables[] = {a.cu_seqlens, a.starts, a.slots};
    for (const void *p : tables)
        if (misaligned(p, 4)) return KDA_ERR_ALIGN;
    const Span in[] = {span(a.q, strided_bytes(rows, a.q_stride, wq)), span(a.k, strided_bytes(rows, a.k_stride, wk)),
                       span(a.v, strided_bytes(rows, a.v_stride, wk)), span(a.cu_seqlens, ((int64_t)a.N + 1) * 4),
                       span(a.starts, (int64_t)a.N * 4), span(a.slots, (int64_t)a.N * 4)};
    const Span out = span(a.out, (int64_t)rows * wq * 2), pool = span(a.pool, pool_bytes);
    for (const Span &s : in)
        if (overlap(out, s) || overlap(pool, s)) return KDA_ERR_ALIAS;
    return overlap(out, pool) ? KDA_ERR_ALIAS : KDA_OK;
}

int check_pools(const kda_pool *pools, int num_pools, int num_slots, kda::SlotPools *to)
{
    if (num_pools < 1 || num_slots < 1) return KDA_ERR_SHAPE;
    if (num_pools > KDA_MAX_POOLS || num_slots > KDA_MAX_POOL_SLOTS) return KDA_ERR_UNSUPPORTED;
    for (int i = 0; i < num_pools; i++) {
        if (!pools[i].base) return KDA_ERR_NULL;
        if (pools[i].entry_bytes < 1 || pools[i].entry_bytes >= kMaxBytes / num_slots) return KDA_ERR_SHAPE;
        if (misaligned(pools[i].base, 16) || pools[i].entry_bytes % 16) return KDA_ERR_ALIGN;
        to->base[i] = pools[i].base;
        to->entry_bytes[i] = pools[i].entry_bytes;
        for (int j = 0; j < i; j++)
            if (overlap(span(to->base[i], to->entry_bytes[i] * num_slots),
                        span(to->base[j], to->entry_bytes[j] * num_slots)))
                return KDA_ERR_ALIAS;
    }
    to->n = num_pools;
    return KDA_OK;
}

bool in_pools(const kda::SlotPools &p, int num_slots, Span s)
{
    for (int i = 0; i < p.n; i++)
        if (overlap(span(p.base[i], p.entry_bytes[i] * num_slots), s)) return true;
    return false;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

int kda_head_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const float *q_weight,
                       const float *k_weight, const float *table, int max_pos, const int32_t *positions, void *q_out,
                       void *k_out, int T, int Hq, int Hk, int d, int rotary, int layout, int norm, float eps,
                       int dtype, void *stream)
{
    if (T > 0 && (!q || !k || !q_out || !k_out || (rotary > 0 && (!table || !positions)))) return KDA_ERR_NULL;
    if (T < 0 || rotary < 0 || (rotary > 0 && max_pos < 1)) return KDA_ERR_SHAPE;
    int st = check_heads(Hq, Hk, d, dtype);
    if (st != KDA_OK) return st;
    if (rotary > d || (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED) || (norm != 0 && norm != 1) ||
        !(eps >= 0.f && eps <= 3.0e38f))
        return KDA_ERR_SHAPE;
    if (rotary % 16) return KDA_ERR_UNSUPPORTED;
    const int64_t wq = (int64_t)Hq * d, wk = (int64_t)Hk * d;
    const int sq = check_rows(T, q_stride, wq), sk = check_rows(T, k_stride, wk);
    if (sq == KDA_ERR_SHAPE || sk == KDA_ERR_SHAPE) return KDA_ERR_SHAPE;
    if (sq != KDA_OK || sk != KDA_OK) return KDA_ERR_ALIGN;
    const void *tensors[] = {q, k, q_weight, k_weight, table, q_out, k_out};
    for (const void *p : tensors)
        if (misaligned(p, 16)) return KDA_ERR_ALIGN;
    if (misaligned(positions, 4)) return KDA_ERR_ALIGN;
    const Span iq = span(q, strided_bytes(T, q_stride, wq)), ik = span(k, strided_bytes(T, k_stride, wk));
    const Span oq = span(q_out, T * wq * 2), ok = span(k_out, T * wk * 2);
    // in place only where the rows lie the same way: each vector is read whole before it is written
    const bool same_q = q == q_out && q_stride == wq, same_k = k == k_out && k_stride == wk;
    const Span in[] = {span(q_weight, d * 4), span(k_weight, d * 4), span(table, (int64_t)max_pos * rotary * 4),
                       span(positions, (int64_t)T * 4)};
    for (const Span &s : in)
        if (overlap(oq, s) || overlap(ok, s)) return KDA_ERR_ALIAS;
    if ((overlap(oq, iq) && !same_q) || (overlap(ok, ik) && !same_k) || overlap(oq, ik) || overlap(ok, iq) ||
        overlap(oq, ok))
        return KDA_ERR_ALIAS;
    kda::NormRopeArgs a;
    int device, sms;
    if ((st = kda::device_facts(&device, &sms, &a.err_word)) != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
    a.q_weight = q_weight; a.k_weight = k_weight; a.table = table; a.positions = positions;
    a.q_out = q_out; a.k_out = k_out;
    a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rotary = rotary; a.max_pos = max_pos; a.layout = layout; a.norm = norm;
    a.eps = eps; a.f16 = dtype == KDA_F16;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_norm_rope(a));
}

int kda_window_prefill(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                       int64_t v_stride, const int32_t *cu_seqlens, const int32_t *starts, const int32_t *slots,
                       void *kv_pool, int num_slots, int pool_rows, void *out, int N, int T, int Hq, int Hk, int d,
                       int window, int sinks, float scale, int dtype, void *stream)
{
    if (!cu_seqlens || (T > 0 && (!q || !k || !v || !out)) || (!kv_pool && (starts || slots))) return KDA_ERR_NULL;
    if (N < 1 || T < 0) return KDA_ERR_SHAPE;
    kda::WindowArgs a;
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.cu_seqlens = cu_seqlens; a.starts = starts; a.slots = slots; a.pool = kv_pool; a.out = out;
    a.N = N; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.num_slots = num_slots; a.pool_rows = pool_rows;
    a.window = window; a.sinks = sinks; a.scale = scale; a.f16 = dtype == KDA_F16;
    a.stream = (cudaStream_t)stream;
    int st = check_window(a, T, dtype);
    if (st != KDA_OK) return st;
    if ((st = kda::device_facts(&a.device, &a.num_sms, &a.err_word)) != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    if (!kv_pool) {              // every position is below T: neither needs to be larger
        if (a.window > T) a.window = T;
        if (a.sinks > T) a.sinks = T;
    }
    return status_of(kda::launch_window_prefill(a));
}

int kda_window_decode(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                      int64_t v_stride, const int32_t *positions, const int32_t *slots, void *kv_pool, int num_slots,
                      int pool_rows, void *out, int N, int Hq, int Hk, int d, int window, int sinks, float scale,
                      int dtype, void *stream)
{
    if (!q || !k || !v || !positions || !kv_pool || !out) return KDA_ERR_NULL;
    if (N < 1) return KDA_ERR_SHAPE;
    kda::WindowArgs a;
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.cu_seqlens = nullptr; a.starts = positions; a.slots = slots; a.pool = kv_pool; a.out = out;
    a.N = N; a.T = N; a.Hq = Hq; a.Hk = Hk; a.d = d; a.num_slots = num_slots; a.pool_rows = pool_rows;
    a.window = window; a.sinks = sinks; a.scale = scale; a.f16 = dtype == KDA_F16;
    a.stream = (cudaStream_t)stream;
    int st = check_window(a, N, dtype);
    if (st != KDA_OK) return st;
    if ((int64_t)N * Hq > 0x3fffffff) return KDA_ERR_SHAPE;
    if ((st = kda::device_facts(&a.device, &a.num_sms, &a.err_word)) != KDA_OK) return st;
    return status_of(kda::launch_window_decode(a));
}

int kda_slots_copy(const kda_pool *pools, int num_pools, int num_slots, const int32_t *src, const int32_t *dst, int M,
                   void *stream)
{
    if (!pools || !src || !dst) return KDA_ERR_NULL;
    if (M < 1) return KDA_ERR_SHAPE;
    kda::SlotMoveArgs a;
    int st = check_pools(pools, num_pools, num_slots, &a.pools);
    if (st != KDA_OK) return st;
    if (misaligned(src, 4) || misaligned(dst, 4)) return KDA_ERR_ALIGN;
    if (in_pools(a.pools, num_slots, span(src, (int64_t)M * 4)) ||
        in_pools(a.pools, num_slots, span(dst, (int64_t)M * 4)))
        return KDA_ERR_ALIAS;
    if ((st = kda::device_facts(&a.device, &a.num_sms, &a.err_word)) != KDA_OK) return st;
    a.src = src; a.dst = dst; a.new_slots = nullptr; a.M = M; a.num_slots = num_slots;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_slots_copy(a));
}

int kda_slots_compact(const kda_pool *pools, int num_pools, int num_slots, const int32_t *slots, int32_t *new_slots,
                      int N, void *stream)
{
    if (!pools || !slots || !new_slots) return KDA_ERR_NULL;
    if (N < 1) return KDA_ERR_SHAPE;
    kda::SlotMoveArgs a;
    int st = check_pools(pools, num_pools, num_slots, &a.pools);
    if (st != KDA_OK) return st;
    if (misaligned(slots, 4) || misaligned(new_slots, 4)) return KDA_ERR_ALIGN;
    const Span si = span(slots, (int64_t)N * 4), so = span(new_slots, (int64_t)N * 4);
    if (overlap(si, so) || in_pools(a.pools, num_slots, si) || in_pools(a.pools, num_slots, so)) return KDA_ERR_ALIAS;
    if ((st = kda::device_facts(&a.device, &a.num_sms, &a.err_word)) != KDA_OK) return st;
    a.src = slots; a.dst = new_slots; a.new_slots = new_slots; a.M = N; a.num_slots = num_slots;
    a.stream = (cudaStream_t)stream;
    return status_of(kda::launch_slots_compact(a));
}

}  // extern "C"
