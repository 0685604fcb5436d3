// kda_window_rows.cu -- window attention for few rows of a sequence: one new token
// each (decode; the token's key and value enter the cache) or a few (drafts, short
// prompts).
//
// For the query at position p, o = sum_j softmax_j(scale q . k_j) v_j over p's sinks
// and window.  A key head's cached rows are read once for 16 query rows (the G query
// heads that share it, of 16 / G tokens), 2 x 2 d bytes against 64 d operations, so
// HBM bounds it as long as enough loads are in flight.
//
// A CTA of four warps takes 16 query rows of one key head; a cluster of CTAs shares
// such a unit where there are too few units to fill the SMs.  The list of visible
// rows is dealt to all warps in steps of 16 keys, which each warp copies ahead
// (cp.async) into a ring of kStages steps of its own: the eight warps of an SM keep
// 128 KB on their way, several times what the latency of HBM asks for.  The query
// rows are the 16 rows of the warp MMA: S = Q K^T, then O += P V with a running
// maximum and sum per warp.  The order of the summed index is free, so a lane reads
// 16 contiguous bytes of a key row and uses them as the operands of two MMAs (q is
// held in the same order); the value rows come transposed by ldmatrix.  Warps, then
// CTAs of a cluster (through distributed shared memory), join their (maximum, sum,
// O) at the end.  In decode the new token's rows are taken from the call's arguments
// by everyone, so nobody reads the cache row being written.  On a GB300, 64 sequences
// of 32 query heads on 8 key heads of 128 over a window of 4096: 155 us, the copy
// bandwidth; 8 drafted tokens of each over a window of 1024: 67 us, bound by a warp's
// chain of products and exponentials.
#include <cooperative_groups.h>
#include <stdint.h>

#include "kda_warp_mma.cuh"
#include "kda_window.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 2;  // finer shares of an SM than one CTA of eight warps: 163 us instead of 174 (64 x 8 units)
constexpr int kRows = 16;       // query rows of a warp: the rows of the MMA
constexpr int kMaxRanks = 8;    // CTAs of a cluster
constexpr int kStep = 16;       // keys at a time
constexpr int kTiles = kStep / 8;   // score tiles of a step
constexpr int kStages = 3;      // steps in a ring, for each warp that shares it

// shared memory of a CTA: every warp's O, then maxima and sums; after the warps
// are joined, those of the CTA's 16 SHARE rows in the first SHARE parts
template <int D> struct JoinSmem {
    float o[kWarps][kRows][D + 8];   // rows 8 banks apart
    float m[kWarps][kRows], l[kWarps][kRows];
};

// MANY false: one new token of each sequence (decode), which also enters the cache;
// true: the rows of packed sequences.  SHARE: warps that share a ring and with it
// each key read from memory, with 16 query rows each; the CTA's other warps take
// other keys.
template <typename E, int D, bool MANY, int SHARE>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
window_rows_kernel(const __grid_constant__ WindowParams p)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    JoinSmem<D> &sm = *reinterpret_cast<JoinSmem<D> *>(smem_raw);
    constexpr int kParts = kWarps / SHARE, kRing = kStages * SHARE;   // shares of the keys; steps in a ring
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int part = warp / SHARE, sub = warp % SHARE;   // which keys, which rows

    if (MANY) grid_go_on();
    // In a divided batch this grid must not end before that of the tiles, which is why its
    // last cluster waits for it: the cache kernel waits for this one only.
    auto leave = [&]() {
        if (MANY && blockIdx.x + ranks >= gridDim.x) grid_wait();
    };
    int unit = blockIdx.x / ranks;
    const int group = unit % p.groups;
    unit /= p.groups;
    const int hk = unit % p.Hk;
    const int head0 = hk * p.G + group * kRows * SHARE, heads = min(kRows * SHARE, p.G - group * kRows * SHARE);   // of one token
    const bool reports = threadIdx.x < 32 && rank == 0 && hk == 0 && group == 0;
    // The unit's rows: `tokens` tokens from row t0 on, at positions first .. last; position
    // x of the sequence is row bos + x - start of the call from `start` on, before it
    // a row of the cache.  A padded sequence or a number without rows: the whole
    // cluster leaves.
    int entry, t0, bos, start, first, tokens = 1;
    if (MANY) {
        const Rows r = rows_of(p, p.tile_tokens, unit / p.Hk, lane, reports);
        if (!r.n || is_long(p, r.len)) {
            leave();
            return;
        }
        entry = r.entry;
        bos = r.bos;
        start = r.start;
        t0 = r.bos + r.from;
        first = r.start + r.from;
        tokens = r.n;
    } else {
        t0 = bos = unit / p.Hk;
        start = p.starts[t0];
        entry = entry_of(p.slots, t0, p.num_slots, p.err, reports && lane == 0);
        if (entry < 0) return;
        if (start < 0) {
            if (reports && lane == 0) atomicOr(p.err, kErrBadPosition);
            start = 0;
        }
        first = start;
    }
    const int last = first + tokens - 1, rows = tokens * heads;

    // list of the positions that any of the rows sees: sinks before the window, then
    // the window
    const int lo = max(0, first - p.window + 1), ns = min(p.sinks, lo), count = ns + last - lo + 1;
    const int ring = p.pool_rows - p.sinks, wrap0 = max(lo, p.sinks);
    const int ring0 = p.pool ? (wrap0 - p.sinks) % ring : 0;
    const int64_t head_rows = (int64_t)p.pool_rows * D;
    uint16_t *kc = p.pool ? p.pool + ((int64_t)entry * 2 * p.Hk + hk) * head_rows : nullptr;
    const int64_t v_behind = p.Hk * head_rows;           // from a key row to its value row
    const uint16_t *kn = p.k + bos * p.k_stride + hk * D, *vn = p.v + bos * p.v_stride + hk * D;
    // row in the cache of list item i (which is there)
    auto cache_row = [&](int i) {
        const int x = i < ns ? i : lo + i - ns;
        if (x < p.sinks) return x;
        const int at = ring0 + (x - wrap0);
        return p.sinks + (at >= ring ? at - ring : at);
    };
    if (!MANY && rank == 0 && group == 0 && threadIdx.x < D / 4) {   // the new rows enter the cache
        const int64_t at = (int64_t)ring_row(first, p.sinks, p.pool_rows) * D;
        const int e = (threadIdx.x & (D / 8 - 1)) * 8;
        if (threadIdx.x < D / 8) *reinterpret_cast<uint4 *>(kc + at + e) = *reinterpret_cast<const uint4 *>(kn + e);
        else *reinterpret_cast<uint4 *>(kc + v_behind + at + e) = *reinterpret_cast<const uint4 *>(vn + e);
    }

    // q in the order of the key loads: rows g and g + 8, elements 32 kk + 8c .. + 7
    uint4 qa[D / 32], qb[D / 32];
    const int row_a = kRows * sub + g, row_b = row_a + 8;
    const int tok_a = MANY ? row_a / heads : 0, tok_b = MANY ? row_b / heads : 0;
    const uint16_t *qp = p.q + t0 * p.q_stride + (int64_t)head0 * D + 8 * c;
    const uint16_t *qpa = qp + tok_a * p.q_stride + (row_a - tok_a * heads) * D;
    const uint16_t *qpb = qp + tok_b * p.q_stride + (row_b - tok_b * heads) * D;
#pragma unroll
    for (int kk = 0; kk < D / 32; kk++) {
        qa[kk] = row_a < rows ? *reinterpret_cast<const uint4 *>(qpa + 32 * kk) : make_uint4(0, 0, 0, 0);
        qb[kk] = row_b < rows ? *reinterpret_cast<const uint4 *>(qpb + 32 * kk) : make_uint4(0, 0, 0, 0);
    }

    float o[D / 8][4];               // tiles of 8 columns
#pragma unroll
    for (int j = 0; j < D / 8; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // the ring of these keys; a stage is 16 key rows, then 16 value rows, each copied by
    // the warps that share it
    constexpr int kTile = kStep * D * 2;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(smem_raw) + part * kRing * 2 * kTile;
    constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;   // 16-byte pieces of a row, rows that a warp copies at once
    const int piece = lane % kPieces;
    auto fetch = [&](int i0, int stage) {
        const uint32_t to = ring_at + stage * 2 * kTile;
        // mostly all 16 rows follow one another, in the ring or in the call
        const int x0 = lo + i0 - ns;                     // position of the first, from item ns on
        const bool old = i0 >= ns && x0 >= p.sinks && x0 <= start - kStep;
        const int r0 = old ? cache_row(i0) : 0;
        if (old && r0 + kStep <= p.pool_rows) {
            const int k0 = sub * kAtOnce + lane / kPieces;
            const uint16_t *ks = kc + (int64_t)(r0 + k0) * D + 8 * piece, *vs = ks + v_behind;
#pragma unroll
            for (int j = 0; j < kStep / kAtOnce / SHARE; j++) {
                const int k = j * SHARE * kAtOnce;
                copy16(to + place_key<D>(k0 + k, piece), ks + k * D);
                copy16(to + kTile + place_value<D>(k0 + k, piece), vs + k * D);
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < kStep / kAtOnce / SHARE; j++) {
                const int k = (j * SHARE + sub) * kAtOnce + lane / kPieces;
                const uint16_t *ks, *vs;
                const int i = min(i0 + k, count - 1);    // past the end: any row of the list will do
                const int x = i < ns ? i : lo + i - ns;
                if (x < start) {
                    ks = kc + (int64_t)cache_row(i) * D;
                    vs = ks + v_behind;
                } else {
                    ks = kn + (x - start) * p.k_stride;
                    vs = vn + (x - start) * p.v_stride;
                }
                copy16(to + place_key<D>(k, piece), ks + 8 * piece);
                copy16(to + kTile + place_value<D>(k, piece), vs + 8 * piece);
            }
        }
    };
    const int stride = ranks * kParts * kStep;
    const int begin = (rank * kParts + part) * kStep;
#pragma unroll
    for (int s = 0; s < kRing - 1; s++) {
        if (begin + s * stride < count) fetch(begin + s * stride, s);
        copy_commit();
    }
    int stage = 0;
    for (int i0 = begin; i0 < count; i0 += stride) {
        copy_wait<kRing - 2>();
        if (SHARE > 1) named_bar(1 + part, 32 * SHARE);  // everyone's copies of this stage, and done with the last one
        else __syncwarp();
        const int ahead = i0 + (kRing - 1) * stride;
        if (ahead < count) fetch(ahead, stage == 0 ? kRing - 1 : stage - 1);
        copy_commit();
        const uint32_t kt = ring_at + stage * 2 * kTile, vt = kt + kTile;
        stage = stage + 1 == kRing ? 0 : stage + 1;
        if (SHARE > 1 && kRows * sub >= rows) continue;  // no row of this warp's: it only copies
        float s[kTiles][4];
#pragma unroll
        for (int j = 0; j < kTiles; j++) {
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) {
                const uint4 kr = shared16(kt + place_key<D>(8 * j + g, 4 * kk + c));
                mma16816<E>(s[j], qa[kk].x, qb[kk].x, qa[kk].y, qb[kk].y, kr.x, kr.y);
                mma16816<E>(s[j], qa[kk].z, qb[kk].z, qa[kk].w, qb[kk].w, kr.z, kr.w);
            }
        }
        if (MANY) {
            // items after the sinks are tested where a row may not see them
            const int x0 = lo + i0 - ns;
            if (i0 + kStep > count || (i0 + kStep > ns && (x0 > first - (kStep - 1) || x0 <= last - p.window))) {
#pragma unroll
                for (int j = 0; j < kTiles; j++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int i = i0 + 8 * j + 2 * c + e, x = lo + i - ns;
                        const bool sink = i < ns || x < p.sinks;
                        if (i >= count || (i >= ns && (x > first + tok_a || (x <= first + tok_a - p.window && !sink))))
                            s[j][e] = -INFINITY;
                        if (i >= count || (i >= ns && (x > first + tok_b || (x <= first + tok_b - p.window && !sink))))
                            s[j][2 + e] = -INFINITY;
                    }
            }
        } else if (i0 + kStep > count) {
#pragma unroll
            for (int j = 0; j < kTiles; j++)
#pragma unroll
                for (int e = 0; e < 2; e++)
                    if (i0 + 8 * j + 2 * c + e >= count) s[j][e] = s[j][2 + e] = -INFINITY;
        }
        float a = fmaxf(s[0][0], s[0][1]), b = fmaxf(s[0][2], s[0][3]);
#pragma unroll
        for (int j = 1; j < kTiles; j++) {
            a = fmaxf(a, fmaxf(s[j][0], s[j][1]));
            b = fmaxf(b, fmaxf(s[j][2], s[j][3]));
        }
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
        for (int j = 0; j < kTiles; j++) {
            s[j][0] = ex2((s[j][0] - z0) * p.scale_log2);
            s[j][1] = ex2((s[j][1] - z0) * p.scale_log2);
            s[j][2] = ex2((s[j][2] - z1) * p.scale_log2);
            s[j][3] = ex2((s[j][3] - z1) * p.scale_log2);
            l0 += s[j][0] + s[j][1];
            l1 += s[j][2] + s[j][3];
        }
#pragma unroll
        for (int k = 0; k < kTiles / 2; k++) {
            // probabilities in 16 bits, as the tensor cores take them; their sum stays fp32
            const float(&x)[4] = s[2 * k], (&y)[4] = s[2 * k + 1];
            const uint32_t p0 = Half2<E>::pack(x[0], x[1]), p1 = Half2<E>::pack(x[2], x[3]);
            const uint32_t p2 = Half2<E>::pack(y[0], y[1]), p3 = Half2<E>::pack(y[2], y[3]);
            const int r = 16 * k + (lane & 15);
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
                uint32_t b[4];
                load_matrices_t(vt + place_value<D>(r, j + (lane >> 4)), b);
                mma16816<E>(o[j], p0, p1, p2, p3, b[0], b[1]);
                mma16816<E>(o[j + 1], p0, p1, p2, p3, b[2], b[3]);
            }
        }
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
#pragma unroll
    for (int j = 0; j < D / 8; j++) {
        *reinterpret_cast<float2 *>(&sm.o[warp][g][8 * j + 2 * c]) = make_float2(o[j][0], o[j][1]);
        *reinterpret_cast<float2 *>(&sm.o[warp][g + 8][8 * j + 2 * c]) = make_float2(o[j][2], o[j][3]);
    }
    __syncthreads();
    // join the warps of different keys: the CTA's maxima, sums and O into the first SHARE
    // parts (each element is read and written by one thread; the factors are read
    // before those parts' are replaced)
    constexpr int kQuads = D / 4, kEach = SHARE * kRows * kQuads / (kWarps * 32);
    float mm[kEach], ll[kEach];
#pragma unroll
    for (int it = 0; it < kEach; it++) {
        const int e = threadIdx.x + it * kWarps * 32, h = e / kQuads % kRows, who = e / kQuads / kRows, d4 = e % kQuads;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kParts; w++) m = fmaxf(m, sm.m[w * SHARE + who][h]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kParts; w++) {
            const float f = m == -INFINITY ? 0.f : ex2((sm.m[w * SHARE + who][h] - m) * p.scale_log2);
            const float4 x = reinterpret_cast<const float4 *>(sm.o[w * SHARE + who][h])[d4];
            l += sm.l[w * SHARE + who][h] * f;
            acc.x += x.x * f;
            acc.y += x.y * f;
            acc.z += x.z * f;
            acc.w += x.w * f;
        }
        mm[it] = m;
        ll[it] = l;
        reinterpret_cast<float4 *>(sm.o[who][h])[d4] = acc;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kEach; it++) {
        const int e = threadIdx.x + it * kWarps * 32;
        if (e % kQuads == 0) {
            sm.m[e / kQuads / kRows][e / kQuads % kRows] = mm[it];
            sm.l[e / kQuads / kRows][e / kQuads % kRows] = ll[it];
        }
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    // join the CTAs: the cluster's threads share the output's elements
    for (int e = rank * kWarps * 32 + threadIdx.x; e < rows * kQuads; e += ranks * kWarps * 32) {
        const int r = e / kQuads, d4 = e % kQuads;
        float *ms = &sm.m[r / kRows][r % kRows], *ls = &sm.l[r / kRows][r % kRows];
        float4 *os = reinterpret_cast<float4 *>(sm.o[r / kRows][r % kRows]) + d4;
        // all the ranks' parts are on their way together: a read of another CTA takes some
        // hundred nanoseconds
        float mk[kMaxRanks], lk[kMaxRanks], m = -INFINITY, l = 0.f;
        float4 ok[kMaxRanks];
#pragma unroll
        for (int k = 0; k < kMaxRanks; k++) {
            mk[k] = -INFINITY;
            lk[k] = 0.f;
            ok[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < ranks) {
                mk[k] = *cluster.map_shared_rank(ms, k);
                lk[k] = *cluster.map_shared_rank(ls, k);
                ok[k] = *cluster.map_shared_rank(os, k);
            }
        }
#pragma unroll
        for (int k = 0; k < kMaxRanks; k++) m = fmaxf(m, mk[k]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxRanks; k++) {
            const float f = mk[k] == -INFINITY ? 0.f : ex2((mk[k] - m) * p.scale_log2);
            l += lk[k] * f;
            acc.x += ok[k].x * f;
            acc.y += ok[k].y * f;
            acc.z += ok[k].z * f;
            acc.w += ok[k].w * f;
        }
        const float inv = 1.f / l;
        uint2 r2;
        r2.x = Half2<E>::pack(acc.x * inv, acc.y * inv);
        r2.y = Half2<E>::pack(acc.z * inv, acc.w * inv);
        const int tok = MANY ? r / heads : 0;
        *reinterpret_cast<uint2 *>(p.out + ((int64_t)(t0 + tok) * p.Hq + head0 + r - tok * heads) * D + 4 * d4) = r2;
    }
    if (ranks > 1) cluster.sync();      // nobody leaves while its shared memory is being read
    leave();
}

template <typename E, int D, bool MANY, int SHARE>
cudaError_t launch(const WindowArgs &a, WindowParams p)
{
    p.groups = (p.G + kRows * SHARE - 1) / (kRows * SHARE);
    p.tile_tokens = MANY && p.G < kRows * SHARE ? kRows * SHARE / p.G : 1;
    const int64_t units = (MANY ? (int64_t)p.T / p.tile_tokens + p.N : (int64_t)p.N) * p.Hk * p.groups;
    // the longest list of a unit: what its tokens see, and no more than there is
    int64_t steps = (int64_t)p.window + p.sinks + p.tile_tokens - 1, held = (int64_t)(p.pool ? p.pool_rows : 0) + p.T;
    steps = ((steps < held ? steps : held) + kStep - 1) / kStep;
    int ranks = 1;
    while (ranks < kMaxRanks && units * ranks * 2 <= kCtasPerSm * a.num_sms && ranks * (kWarps / SHARE) < steps) ranks *= 2;
    if (units * ranks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int kRings = kWarps * kStages * 2 * kStep * D * 2, kJoin = sizeof(JoinSmem<D>);
    constexpr int smem = kRings > kJoin ? kRings : kJoin;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, a.device, [&]() {
        return cudaFuncSetAttribute(window_rows_kernel<E, D, MANY, SHARE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * ranks));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.longer ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, window_rows_kernel<E, D, MANY, SHARE>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// as many warps to a key as the rows of a sequence fill (on average, for MANY)
template <typename E, int D, bool MANY>
cudaError_t launch_shared(const WindowArgs &a, const WindowParams &p)
{
    const int64_t rows = MANY ? ((int64_t)p.T * p.G + p.N - 1) / p.N : p.G;
    return rows <= kRows       ? launch<E, D, MANY, 1>(a, p)
           : rows <= 2 * kRows ? launch<E, D, MANY, 2>(a, p)
                               : launch<E, D, MANY, 4>(a, p);
}

template <bool MANY>
cudaError_t launch_rows(const WindowArgs &a, int longer)
{
    WindowParams p = window_params(a);
    p.longer = longer;
    if (a.d == 128) return a.f16 ? launch_shared<__half, 128, MANY>(a, p) : launch_shared<__nv_bfloat16, 128, MANY>(a, p);
    return a.f16 ? launch_shared<__half, 64, MANY>(a, p) : launch_shared<__nv_bfloat16, 64, MANY>(a, p);
}

}  // namespace

cudaError_t launch_window_decode(const WindowArgs &a) { return launch_rows<false>(a, 0); }
cudaError_t launch_window_rows(const WindowArgs &a, int longer) { return launch_rows<true>(a, longer); }

}  // namespace kda
