// kda_window_decode.cu -- window attention of one new token per sequence over
// the ring cache; the token's key and value enter the cache.
//
// For a sequence at position p and key head h, with the visible list of p's sinks
// and window, o = sum_j softmax_j(scale q . k_j) v_j for the G query heads of h.
// Each cached row is read once for all G heads (2 x 2 d bytes against 4 G d
// operations), so HBM bounds it as long as enough loads are in flight.
//
// A CTA of four warps takes (sequence, key head, up to 16 query heads); a
// cluster of CTAs shares one such unit where there are too few units to fill the
// SMs.  The list of visible rows is dealt to all warps in steps of 16 keys, which
// each warp copies ahead (cp.async) into a ring of kStages steps of its own: the
// eight warps of an SM keep 128 KB on their way, several times what the latency of
// HBM asks for.  The heads are the 16 rows of the warp MMA: S = Q K^T, then O += P V with a
// running maximum and sum per warp.  The order of the summed index is free, so a
// lane reads 16 contiguous bytes of a key row and uses them as the operands of two
// MMAs (q is held in the same order); of the value rows it reads 16 bytes of two
// neighbouring keys and interleaves them, which permutes only the output columns.
// Warps, then CTAs of a cluster (through distributed shared memory), join their
// (maximum, sum, O) at the end.  The new token's rows are taken from the call's
// arguments by everyone, so nobody reads the cache row being written.
#include <cooperative_groups.h>
#include <stdint.h>

#include "kda_window.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 2;  // finer shares of an SM than one CTA of eight warps: 163 us instead of 174 (64 x 8 units)
constexpr int kHeads = 16;      // query heads of a CTA: the rows of the MMA
constexpr int kStep = 16;       // keys of a warp at a time
constexpr int kStages = 3;      // steps in a warp's ring

// 16 bytes from global to shared memory, asynchronously
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// Place of 16-byte piece c of row r in a step's tile: the pieces that eight lanes
// read together (of a key tile four pieces of rows 2i and 2i + 1; of a value tile
// pieces 2i and 2i + 1 of four rows of one parity) lie in different banks.
template <int D> __device__ __forceinline__ uint32_t place(int r, int c)
{
    return r * (D * 2) + ((c ^ ((r & 6) ^ ((r & 1) << 2))) << 4);
}

struct DecodeWinParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *positions, *slots;
    uint16_t *pool, *out;
    int N, Hq, Hk, groups;      // groups of up to 16 query heads per key head
    int num_slots, pool_rows, window, sinks;
    float scale_log2;
    int *err;
};

template <typename E>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// shared memory of a CTA: every warp's O, then maxima and sums; after the warps
// are joined, the CTA's own in part[0]
template <int D> struct DecodeSmem {
    float o[kWarps][kHeads][D];
    float m[kWarps][kHeads], l[kWarps][kHeads];
};

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
window_decode_kernel(const __grid_constant__ DecodeWinParams p)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DecodeSmem<D> &sm = *reinterpret_cast<DecodeSmem<D> *>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

    int unit = blockIdx.x / ranks;
    const int group = unit % p.groups;
    unit /= p.groups;
    const int hk = unit % p.Hk, n = unit / p.Hk;
    const bool reports = threadIdx.x == 0 && rank == 0 && hk == 0 && group == 0;
    const int entry = entry_of(p.slots, n, p.num_slots, p.err, reports);
    if (entry < 0) return;      // the whole cluster
    int pos = p.positions[n];
    if (pos < 0) {
        if (reports) atomicOr(p.err, kErrBadPosition);
        pos = 0;
    }
    const int G = p.Hq / p.Hk, head0 = hk * G + group * kHeads, heads = min(kHeads, G - group * kHeads);

    // list of visible positions: sinks before the window, then the window
    const int lo = max(0, pos - p.window + 1), ns = min(p.sinks, lo), count = ns + pos - lo + 1;
    const int ring = p.pool_rows - p.sinks, wrap0 = max(lo, p.sinks);
    const int ring0 = (wrap0 - p.sinks) % ring;
    const int64_t head_rows = (int64_t)p.pool_rows * D;
    uint16_t *kc = p.pool + ((int64_t)entry * 2 * p.Hk + hk) * head_rows, *vc = kc + p.Hk * head_rows;
    const uint16_t *kn = p.k + n * p.k_stride + hk * D, *vn = p.v + n * p.v_stride + hk * D;
    // element offset of list item i's row in the cache, -1 for the new token
    auto row_of = [&](int i) -> int64_t {
        if (i >= count - 1) return -1;             // also past the end: any valid row will do
        int at = i;                                // a sink
        if (i >= ns) {
            const int pp = lo + i - ns;
            if (pp < p.sinks) at = pp;
            else {
                at = ring0 + (pp - wrap0);
                at = p.sinks + (at >= ring ? at - ring : at);
            }
        }
        return (int64_t)at * D;
    };
    if (rank == 0 && group == 0 && threadIdx.x < D / 4) {   // the new rows enter the cache
        const int64_t at = (int64_t)ring_row(pos, p.sinks, p.pool_rows) * D;
        const int e = (threadIdx.x & (D / 8 - 1)) * 8;
        if (threadIdx.x < D / 8) *reinterpret_cast<uint4 *>(kc + at + e) = *reinterpret_cast<const uint4 *>(kn + e);
        else *reinterpret_cast<uint4 *>(vc + at + e) = *reinterpret_cast<const uint4 *>(vn + e);
    }

    // q in the order of the key loads: rows g and g + 8, elements 32 kk + 8c .. + 7
    uint4 qa[D / 32], qb[D / 32];
    const uint16_t *qp = p.q + n * p.q_stride + (int64_t)head0 * D + 8 * c;
#pragma unroll
    for (int kk = 0; kk < D / 32; kk++) {
        qa[kk] = g < heads ? *reinterpret_cast<const uint4 *>(qp + g * D + 32 * kk) : make_uint4(0, 0, 0, 0);
        qb[kk] = g + 8 < heads ? *reinterpret_cast<const uint4 *>(qp + (g + 8) * D + 32 * kk) : make_uint4(0, 0, 0, 0);
    }

    float o[D / 64][8][4];
#pragma unroll
    for (int i = 0; i < D / 64; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // this warp's ring; a stage is 16 key rows, then 16 value rows
    constexpr int kTile = kStep * D * 2;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(smem_raw) + warp * kStages * 2 * kTile;
    constexpr int kPieces = D / 8, kRows = 32 / kPieces;   // 16-byte pieces of a row, rows that the warp copies at once
    const int piece = lane % kPieces;
    auto fetch = [&](int i0, int stage) {
        const uint32_t to = ring_at + stage * 2 * kTile;
        // rows of the ring that follow one another, as most do
        const int64_t r0 = row_of(i0);
        const bool run = i0 >= ns && i0 + kStep < count && r0 >= (int64_t)p.sinks * D &&
                         r0 + (kStep - 1) * D < (int64_t)p.pool_rows * D;
#pragma unroll
        for (int j = 0; j < kStep / kRows; j++) {
            const int k = j * kRows + lane / kPieces;
            const int64_t r = run ? r0 + k * D : row_of(i0 + k);
            copy16(to + place<D>(k, piece), (r < 0 ? kn : kc + r) + 8 * piece);
            copy16(to + kTile + place<D>(k, piece), (r < 0 ? vn : vc + r) + 8 * piece);
        }
    };
    const int stride = ranks * kWarps * kStep;
    const int begin = (rank * kWarps + warp) * kStep;
#pragma unroll
    for (int s = 0; s < kStages - 1; s++) {
        if (begin + s * stride < count) fetch(begin + s * stride, s);
        copy_commit();
    }
    int stage = 0;
    for (int i0 = begin; i0 < count; i0 += stride) {
        {
            const int ahead = i0 + (kStages - 1) * stride;
            if (ahead < count) fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
            copy_commit();
        }
        copy_wait<kStages - 1>();
        __syncwarp();
        const uint32_t kt = ring_at + stage * 2 * kTile, vt = kt + kTile;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) {
                const uint4 kr = shared16(kt + place<D>(8 * j + g, 4 * kk + c));
                mma16816<E>(s[j], qa[kk].x, qb[kk].x, qa[kk].y, qb[kk].y, kr.x, kr.y);
                mma16816<E>(s[j], qa[kk].z, qb[kk].z, qa[kk].w, qb[kk].w, kr.z, kr.w);
            }
        }
        if (i0 + kStep > count) {
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int e = 0; e < 2; e++)
                    if (i0 + 8 * j + 2 * c + e >= count) s[j][e] = s[j][2 + e] = -INFINITY;
        }
        float a = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float b = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
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
            for (int i = 0; i < D / 64; i++)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    o[i][j][0] *= f0;
                    o[i][j][1] *= f0;
                    o[i][j][2] *= f1;
                    o[i][j][3] *= f1;
                }
            m0 = a;
            m1 = b;
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0 * p.scale_log2, z1 = m1 == -INFINITY ? 0.f : m1 * p.scale_log2;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            s[j][0] = ex2(fmaf(s[j][0], p.scale_log2, -z0));
            s[j][1] = ex2(fmaf(s[j][1], p.scale_log2, -z0));
            s[j][2] = ex2(fmaf(s[j][2], p.scale_log2, -z1));
            s[j][3] = ex2(fmaf(s[j][3], p.scale_log2, -z1));
            l0 += s[j][0] + s[j][1];
            l1 += s[j][2] + s[j][3];
        }
        // probabilities in 16 bits, as the tensor cores take them; their sum stays fp32
        const uint32_t p0 = Half2<E>::pack(s[0][0], s[0][1]), p1 = Half2<E>::pack(s[0][2], s[0][3]);
        const uint32_t p2 = Half2<E>::pack(s[1][0], s[1][1]), p3 = Half2<E>::pack(s[1][2], s[1][3]);
#pragma unroll
        for (int hh = 0; hh < D / 64; hh++) {
            const uint4 v0 = shared16(vt + place<D>(2 * c, 8 * hh + g)), v1 = shared16(vt + place<D>(2 * c + 1, 8 * hh + g));
            const uint4 v2 = shared16(vt + place<D>(2 * c + 8, 8 * hh + g)), v3 = shared16(vt + place<D>(2 * c + 9, 8 * hh + g));
            const uint32_t r0[4] = {v0.x, v0.y, v0.z, v0.w}, r1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t r2[4] = {v2.x, v2.y, v2.z, v2.w}, r3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
                mma16816<E>(o[hh][j], p0, p1, p2, p3, __byte_perm(r0[j / 2], r1[j / 2], sel),
                            __byte_perm(r2[j / 2], r3[j / 2], sel));
            }
        }
        __syncwarp();                // the stage may be filled again
    }
    copy_wait<0>();
    __syncthreads();                 // the rings become the join's buffers
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (c == 0) {
        sm.m[warp][g] = m0;
        sm.m[warp][g + 8] = m1;
        sm.l[warp][g] = l0;
        sm.l[warp][g + 8] = l1;
    }
    // column 2c (+1) of the tile (hh, j) is element 64 hh + 16 c (+ 8) + j
#pragma unroll
    for (int hh = 0; hh < D / 64; hh++)
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
            for (int q = 0; q < 2; q++) {
                float *to = &sm.o[warp][g + 8 * e][64 * hh + 16 * c + 8 * q];
                float4 x, y;
                x.x = o[hh][0][2 * e + q]; x.y = o[hh][1][2 * e + q]; x.z = o[hh][2][2 * e + q]; x.w = o[hh][3][2 * e + q];
                y.x = o[hh][4][2 * e + q]; y.y = o[hh][5][2 * e + q]; y.z = o[hh][6][2 * e + q]; y.w = o[hh][7][2 * e + q];
                reinterpret_cast<float4 *>(to)[0] = x;
                reinterpret_cast<float4 *>(to)[1] = y;
            }
    __syncthreads();
    // join the warps: this CTA's maximum, sum and O into part 0 (each element is
    // read and written by one thread; the factors are read before part 0's are replaced)
    constexpr int kQuads = D / 4;
    float mm[kHeads * kQuads / (kWarps * 32)], ll[kHeads * kQuads / (kWarps * 32)];
#pragma unroll
    for (int it = 0; it < kHeads * kQuads / (kWarps * 32); it++) {
        const int e = threadIdx.x + it * kWarps * 32, h = e / kQuads, d4 = e % kQuads;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) m = fmaxf(m, sm.m[w][h]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const float f = m == -INFINITY ? 0.f : ex2((sm.m[w][h] - m) * p.scale_log2);
            const float4 x = reinterpret_cast<const float4 *>(sm.o[w][h])[d4];
            l += sm.l[w][h] * f;
            acc.x += x.x * f;
            acc.y += x.y * f;
            acc.z += x.z * f;
            acc.w += x.w * f;
        }
        mm[it] = m;
        ll[it] = l;
        reinterpret_cast<float4 *>(sm.o[0][h])[d4] = acc;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kHeads * kQuads / (kWarps * 32); it++) {
        const int e = threadIdx.x + it * kWarps * 32;
        if (e % kQuads == 0) {
            sm.m[0][e / kQuads] = mm[it];
            sm.l[0][e / kQuads] = ll[it];
        }
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    // join the CTAs: the cluster's threads share the output's elements
    for (int e = rank * kWarps * 32 + threadIdx.x; e < heads * kQuads; e += ranks * kWarps * 32) {
        const int h = e / kQuads, d4 = e % kQuads;
        float m = -INFINITY, l = 0.f;
        for (int r = 0; r < ranks; r++) m = fmaxf(m, cluster.map_shared_rank(&sm.m[0][h], r)[0]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < ranks; r++) {
            const float f = m == -INFINITY ? 0.f : ex2((cluster.map_shared_rank(&sm.m[0][h], r)[0] - m) * p.scale_log2);
            const float4 x = *cluster.map_shared_rank(reinterpret_cast<float4 *>(sm.o[0][h]) + d4, r);
            l += cluster.map_shared_rank(&sm.l[0][h], r)[0] * f;
            acc.x += x.x * f;
            acc.y += x.y * f;
            acc.z += x.z * f;
            acc.w += x.w * f;
        }
        const float inv = 1.f / l;
        uint2 r2;
        r2.x = Half2<E>::pack(acc.x * inv, acc.y * inv);
        r2.y = Half2<E>::pack(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(p.out + ((int64_t)n * p.Hq + head0 + h) * D + 4 * d4) = r2;
    }
    if (ranks > 1) cluster.sync();      // nobody leaves while its shared memory is being read
}

template <typename E, int D>
cudaError_t launch(const WindowArgs &a, const DecodeWinParams &p)
{
    const int64_t units = (int64_t)p.N * p.Hk * p.groups;
    int64_t steps = ((int64_t)p.window + p.sinks + kStep - 1) / kStep;   // at most, of one unit
    if (steps > (p.pool_rows + kStep - 1) / kStep) steps = (p.pool_rows + kStep - 1) / kStep;
    int ranks = 1;
    while (ranks < 8 && units * ranks * 2 <= kCtasPerSm * a.num_sms && ranks * kWarps < steps) ranks *= 2;
    constexpr int kRing = kWarps * kStages * 2 * kStep * D * 2, kJoin = sizeof(DecodeSmem<D>);
    constexpr int smem = kRing > kJoin ? kRing : kJoin;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, a.device, [&]() {
        return cudaFuncSetAttribute(window_decode_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * ranks));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, window_decode_kernel<E, D>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_window_decode(const WindowArgs &a)
{
    DecodeWinParams p;
    p.q = (const uint16_t *)a.q; p.k = (const uint16_t *)a.k; p.v = (const uint16_t *)a.v;
    p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
    p.positions = a.starts; p.slots = a.slots;
    p.pool = (uint16_t *)a.pool; p.out = (uint16_t *)a.out;
    p.N = a.N; p.Hq = a.Hq; p.Hk = a.Hk; p.groups = (a.Hq / a.Hk + kHeads - 1) / kHeads;
    p.num_slots = a.num_slots; p.pool_rows = a.pool_rows; p.window = a.window; p.sinks = a.sinks;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err_word;
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
