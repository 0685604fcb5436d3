// kda_checks.h -- argument checks that the C ABI's files share.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"
#include "kda_hybrid.h"

namespace kda {
namespace checks {

constexpr int64_t kMaxBytes = (int64_t)1 << 40;   // a tensor's span; keeps every product of sizes in 64 bits

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Span span(const void *p, int64_t bytes)
{
    return {(uintptr_t)p, (uintptr_t)p + (p && bytes > 0 ? (uintptr_t)bytes : 0)};
}
inline bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
inline bool misaligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

// rows of `width` elements, `stride` apart, 2 bytes an element
inline int64_t strided_bytes(int T, int64_t stride, int64_t width) { return T > 0 ? ((T - 1) * stride + width) * 2 : 0; }

// row widths and strides: whole 16-byte pieces, rows that do not overlap
inline int check_rows(int T, int64_t stride, int64_t width)
{
    if (stride < width || stride >= ((int64_t)1 << 31)) return KDA_ERR_SHAPE;
    if (T > 0 && (int64_t)T * stride * 2 >= kMaxBytes) return KDA_ERR_SHAPE;
    return stride % 8 ? KDA_ERR_ALIGN : KDA_OK;
}

inline int check_heads(int Hq, int Hk, int d, int dtype)
{
    if (Hq < 1 || Hk < 1 || Hq > (1 << 16) || Hk > (1 << 16) || d < 1) return KDA_ERR_SHAPE;
    if ((d != 64 && d != 128) || (dtype != KDA_BF16 && dtype != KDA_F16)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// pools of `entries` entries each, at most `most`
inline int check_pools(const kda_pool *pools, int num_pools, int entries, int most, SlotPools *to)
{
    if (num_pools < 1 || entries < 1) return KDA_ERR_SHAPE;
    if (num_pools > KDA_MAX_POOLS || entries > most) return KDA_ERR_UNSUPPORTED;
    for (int i = 0; i < num_pools; i++) {
        if (!pools[i].base) return KDA_ERR_NULL;
        if (pools[i].entry_bytes < 1 || pools[i].entry_bytes >= kMaxBytes / entries) return KDA_ERR_SHAPE;
        if (misaligned(pools[i].base, 16) || pools[i].entry_bytes % 16) return KDA_ERR_ALIGN;
        to->base[i] = pools[i].base;
        to->entry_bytes[i] = pools[i].entry_bytes;
        for (int j = 0; j < i; j++)
            if (overlap(span(to->base[i], to->entry_bytes[i] * entries), span(to->base[j], to->entry_bytes[j] * entries)))
                return KDA_ERR_ALIAS;
    }
    to->n = num_pools;
    return KDA_OK;
}

inline bool in_pools(const SlotPools &p, int entries, Span s)
{
    for (int i = 0; i < p.n; i++)
        if (overlap(span(p.base[i], p.entry_bytes[i] * entries), s)) return true;
    return false;
}

inline int status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace checks
}  // namespace kda
