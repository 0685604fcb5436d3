// kda_paged_rows.cu -- attention over a paged cache for parts of at most 16 query rows a
// key head: a sequence's new token or few (decode, drafts), a small group's prefix.
//
// A part's keys are read once for its 16 query rows (the G query heads that share a key
// head, of 16 / G tokens), 4 d bytes against 64 d operations, so HBM bounds it as long as
// enough loads are in flight.  Every warp is a worker of its own: it takes an equal share
// of the line of all steps of 16 keys, whatever the contexts' lengths, and copies its steps
// ahead (cp.async) into a ring; the eight warps of an SM keep 128 KB on their way.  The
// query rows are the 16 rows of the warp MMA: S = Q K^T, then O += P V with a running
// maximum and sum.  The order of the summed index is free, so a lane reads 16 contiguous
// bytes of a key row and uses them as the operands of two MMAs; the value rows come
// transposed by ldmatrix.
//
// On a GB300, 32 query heads on 8 key heads of 128: 64 contexts of up to 16,384 positions 420 us,
// 6.8 TB/s, the copy bandwidth; one of 20,000 17.5 us, of which 12 are its bytes and the rest the
// way to the first step: the plan's entry, the page table's, the first keys.
#include <stdint.h>

#include "kda_paged_attend.cuh"
#include "kda_warp_mma.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4, kCtasPerSm = kRowWorkersPerSm / kWarps;
constexpr int kStages = 3;           // steps in a warp's ring

// 16 bytes, or zeros where there is nothing to copy
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
paged_rows_kernel(const __grid_constant__ AttendParams p)
{
    // (a ring that starts inside a 128-byte line costs 20 %: each copied row then ends in another)
    extern __shared__ __align__(128) uint8_t smem_raw[];
    constexpr int kTile = kStepKeys * D * 2;             // bytes of a step's keys or values
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int64_t worker = (int64_t)blockIdx.x * kWarps + warp;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem_raw) + warp * kStages * 2 * kTile;
    const PagedCache &cache = p.cache;
    const int page = 1 << cache.page_log2, parts = p.P + p.N;

    // The plan is complete: waited for here, or by the tiles kernel before it let this one start.
    if (!p.after_tiles) grid_wait();
    grid_go_on();
    const Lines lines = load_lines(p.lines);
    const int64_t total = lines.total[1], share = lines.share[1];
    const int64_t from = worker * share, to = min(total * p.Hk, from + share);
    int64_t at = from;
    while (at < to) {
        // the part and key head of this place in the line, and the worker's steps of it
        const int hk = (int)quotient(at, total), part = part_at(p.steps, parts, at - hk * total, lane);
        const bool shared = part < p.P;
        const Part x = load_part(p.parts + part);
        const int64_t begin = hk * total + x.begin + steps_set_up(x), end = begin + part_steps(x);
        if (at < begin) at = begin;
        if (at >= to) break;
        const int step0 = x.key0 / kStepKeys + (int)(at - begin);
        const int steps = (int)(min(end, to) - at);
        at += steps;
        const int rows = x.tokens * p.G;
        const int32_t *table = cache.table + (int64_t)x.entry * cache.max_pages;
        const int64_t head = (int64_t)D << cache.page_log2;  // elements of a head's rows in a page
        const uint16_t *heads = cache.pages + hk * head;

        // q in the order of the key loads: rows g and g + 8, elements 32 kk + 8c .. + 7
        uint4 qa[D / 32], qb[D / 32];
        const int tok_a = g / p.G, tok_b = (g + 8) / p.G;
        const uint16_t *qp = p.q + x.t0 * p.q_stride + (int64_t)hk * p.G * D + 8 * c;
        const uint16_t *qpa = qp + tok_a * p.q_stride + (g - tok_a * p.G) * D;
        const uint16_t *qpb = qp + tok_b * p.q_stride + (g + 8 - tok_b * p.G) * D;
#pragma unroll
        for (int kk = 0; kk < D / 32; kk++) {
            qa[kk] = g < rows ? *reinterpret_cast<const uint4 *>(qpa + 32 * kk) : make_uint4(0, 0, 0, 0);
            qb[kk] = g + 8 < rows ? *reinterpret_cast<const uint4 *>(qpb + 32 * kk) : make_uint4(0, 0, 0, 0);
        }
        // behind the last key that each row sees
        const int see_a = shared ? x.key1 : min(x.key1, x.first + tok_a + 1);
        const int see_b = shared ? x.key1 : min(x.key1, x.first + tok_b + 1);

        float o[D / 8][4];           // tiles of 8 columns
#pragma unroll
        for (int j = 0; j < D / 8; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        // 32 entries of the page table, a lane each
        int ids_from = -1, ids = 0;
        constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;   // 16-byte pieces of a row, rows that a warp copies at once
        const int piece = lane % kPieces, row = lane / kPieces;
        auto fetch = [&](int s, int stage) {
            const int pos = (step0 + s) * kStepKeys, j = pos >> cache.page_log2;
            if (ids_from < 0 || j >= ids_from + 32) {
                ids_from = j;
                ids = j + lane < cache.max_pages ? __ldg(table + j + lane) : -1;
            }
            const int id = __shfl_sync(0xffffffffu, ids, j - ids_from);
            const bool there = id >= 0 && id < cache.num_pages;
            if (!there && lane == 0) atomicOr(p.err, kErrBadPage);
            const uint16_t *ks = heads + (int64_t)(there ? id : 0) * 2 * p.Hk * head + (int64_t)(pos & (page - 1)) * D + 8 * piece;
            const uint16_t *vs = ks + p.Hk * head;
            const uint32_t dst = ring + stage * 2 * kTile;
            if (there && pos >= x.key0 && pos + kStepKeys <= x.key1) {
#pragma unroll
                for (int i = 0; i < kStepKeys / kAtOnce; i++) {
                    const int k = i * kAtOnce + row;
                    copy16(dst + place_key<D>(k, piece), ks + k * D);
                    copy16(dst + kTile + place_value<D>(k, piece), vs + k * D);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kStepKeys / kAtOnce; i++) {
                    const int k = i * kAtOnce + row;
                    const bool in = there && pos + k >= x.key0 && pos + k < x.key1;
                    copy16_or_zero(dst + place_key<D>(k, piece), ks + k * D, in);
                    copy16_or_zero(dst + kTile + place_value<D>(k, piece), vs + k * D, in);
                }
            }
        };
#pragma unroll
        for (int s = 0; s < kStages - 1; s++) {
            if (s < steps) fetch(s, s);
            copy_commit();
        }
        int stage = 0;
        for (int s = 0; s < steps; s++) {
            copy_wait<kStages - 2>();
            __syncwarp();
            if (s + kStages - 1 < steps) fetch(s + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
            copy_commit();
            const uint32_t kt = ring + stage * 2 * kTile, vt = kt + kTile;
            stage = stage + 1 == kStages ? 0 : stage + 1;
            float z[2][4];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                z[j][0] = z[j][1] = z[j][2] = z[j][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 32; kk++) {
                    const uint4 kr = shared16(kt + place_key<D>(8 * j + g, 4 * kk + c));
                    mma16816<E>(z[j], qa[kk].x, qb[kk].x, qa[kk].y, qb[kk].y, kr.x, kr.y);
                    mma16816<E>(z[j], qa[kk].z, qb[kk].z, qa[kk].w, qb[kk].w, kr.z, kr.w);
                }
            }
            const int pos = (step0 + s) * kStepKeys;
            if (pos < x.key0 || pos + kStepKeys > (shared ? x.key1 : min(x.key1, x.first + 1))) {
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int k = pos + 8 * j + 2 * c + e;
                        if (k < x.key0 || k >= see_a) z[j][e] = -INFINITY;
                        if (k < x.key0 || k >= see_b) z[j][2 + e] = -INFINITY;
                    }
            }
            float a = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
            float b = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 2));
            a = fmaxf(a, m0);
            b = fmaxf(b, m1);
            if (__any_sync(0xffffffffu, a > m0 || b > m1)) {
                // a row whose maximum is still -inf keeps zeros: 2^(-inf - 0) = 0
                const float f0 = a == -INFINITY ? 1.f : ex2((m0 - a) * p.scale_log2);
                const float f1 = b == -INFINITY ? 1.f : ex2((m1 - b) * p.scale_log2);
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int j = 0; j < D / 8; j++) {
                    o[j][0] *= f0;
                    o[j][1] *= f0;
                    o[j][2] *= f1;
                    o[j][3] *= f1;
                }
                m0 = a;
                m1 = b;
            }
            // the difference first: rounded products with the scale would not cancel where a
            // maximum changes or two are joined (by 2^-24 of their size, which has no bound)
            const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                z[j][0] = ex2((z[j][0] - z0) * p.scale_log2);
                z[j][1] = ex2((z[j][1] - z0) * p.scale_log2);
                z[j][2] = ex2((z[j][2] - z1) * p.scale_log2);
                z[j][3] = ex2((z[j][3] - z1) * p.scale_log2);
                l0 += z[j][0] + z[j][1];
                l1 += z[j][2] + z[j][3];
            }
            // probabilities in 16 bits, as the tensor cores take them; their sum stays fp32
            const uint32_t p0 = Half2<E>::pack(z[0][0], z[0][1]), p1 = Half2<E>::pack(z[0][2], z[0][3]);
            const uint32_t p2 = Half2<E>::pack(z[1][0], z[1][1]), p3 = Half2<E>::pack(z[1][2], z[1][3]);
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
                uint32_t v[4];
                load_matrices_t(vt + place_value<D>(lane & 15, j + (lane >> 4)), v);
                mma16816<E>(o[j], p0, p1, p2, p3, v[0], v[1]);
                mma16816<E>(o[j + 1], p0, p1, p2, p3, v[2], v[3]);
            }
        }
        copy_wait<0>();
        __syncwarp();                // everyone is done with the ring
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

        const int where = goes_to(x, shared, begin, end, from, to);
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int r = g + 8 * half, tok = half ? tok_b : tok_a;
            if (r >= rows) continue;
            const float l = half ? l1 : l0;
            const int64_t dense = (int64_t)(x.t0 + tok) * p.Hq + hk * p.G + (r - tok * p.G);   // row of [T][Hq]
            if (where == kToOut) {
                const float inv = 1.f / l;
                uint32_t *out = reinterpret_cast<uint32_t *>(p.out + dense * D) + c;
#pragma unroll
                for (int j = 0; j < D / 8; j++) out[4 * j] = Half2<E>::pack(o[j][2 * half] * inv, o[j][2 * half + 1] * inv);
                continue;
            }
            const int64_t i = where == kToCut ? cut_piece(worker, begin, from) * kFewRows + r : dense;
            float2 *to_o = reinterpret_cast<float2 *>((where == kToCut ? p.cut_rows : p.whole[shared]) + i * D) + c;
#pragma unroll
            for (int j = 0; j < D / 8; j++) to_o[4 * j] = make_float2(o[j][2 * half], o[j][2 * half + 1]);
            if (c == 0) (where == kToCut ? p.cut_rows_ml : p.whole_ml[shared])[i] = make_float2(half ? m1 : m0, l);
        }
    }
    // the join waits for this grid's end, and so has to for the tiles kernel's
    if (p.after_tiles) grid_wait();
}

template <typename E, int D>
cudaError_t launch(const PagedAttentionArgs &a, const AttendParams &p)
{
    constexpr int smem = kWarps * kStages * 2 * kStepKeys * D * 2;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, a.device, [&]() {
        return cudaFuncSetAttribute(paged_rows_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.row_workers / kWarps));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_rows_kernel<E, D>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_rows(const PagedAttentionArgs &a, const AttendParams &p)
{
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
