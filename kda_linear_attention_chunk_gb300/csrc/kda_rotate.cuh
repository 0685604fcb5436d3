// kda_rotate.cuh -- RMS norm of a head and the rotation of its position, as a group of
// d / 8 lanes does it.  Not installed.
//
//     y = w x / sqrt(mean(x^2) + eps);  (a, b) <- (a c_i - b s_i, b c_i + a s_i)
//
// over the pairs (y[i], y[i + r/2]) or (y[2i], y[2i+1]), i < r/2, in fp32 with one
// rounding at the end.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace kda {

template <typename E> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 up(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t down(float lo, float hi)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ float2 up(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
    static __device__ __forceinline__ uint32_t down(float lo, float hi)
    {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

// The lane's eight elements as pairs (a[i], b[i]) that turn together.  HALF: a are
// four consecutive elements and b those half the rotary width further on, so no
// lane needs another's; INTERLEAVED, and behind the rotary width: eight consecutive.
template <typename E, bool HALF>
__device__ __forceinline__ void unpack(const uint2 (&r)[2], float (&a)[4], float (&b)[4])
{
    const float2 w0 = Pair<E>::up(r[0].x), w1 = Pair<E>::up(r[0].y), w2 = Pair<E>::up(r[1].x), w3 = Pair<E>::up(r[1].y);
    if (HALF) {
        a[0] = w0.x; a[1] = w0.y; a[2] = w1.x; a[3] = w1.y;
        b[0] = w2.x; b[1] = w2.y; b[2] = w3.x; b[3] = w3.y;
    } else {
        a[0] = w0.x; b[0] = w0.y; a[1] = w1.x; b[1] = w1.y;
        a[2] = w2.x; b[2] = w2.y; a[3] = w3.x; b[3] = w3.y;
    }
}

template <typename E, bool HALF>
__device__ __forceinline__ void pack(const float (&a)[4], const float (&b)[4], uint2 (&r)[2])
{
    if (HALF) {
        r[0] = make_uint2(Pair<E>::down(a[0], a[1]), Pair<E>::down(a[2], a[3]));
        r[1] = make_uint2(Pair<E>::down(b[0], b[1]), Pair<E>::down(b[2], b[3]));
    } else {
        r[0] = make_uint2(Pair<E>::down(a[0], b[0]), Pair<E>::down(a[1], b[1]));
        r[1] = make_uint2(Pair<E>::down(a[2], b[2]), Pair<E>::down(a[3], b[3]));
    }
}

// What a lane does to its eight elements of any head of one token.  FULL: every element
// turns (rotary = D).
template <typename E, int D, bool HALF, bool FULL>
struct Turn {
    int half, ea, eb;                // half the rotary width; elements ea .. ea + 3 and eb .. eb + 3 of a head
    bool turns;                      // they are rotated
    // a' = rs (a ac - b bs),  b' = rs (b bc + a as): weights and angles folded once for
    // all heads
    float ac[4], as[4], bc[4], bs[4];

    // c: the lane's place in its head
    __device__ __forceinline__ Turn(int c, int rotary)
    {
        half = FULL ? D / 2 : rotary / 2;
        turns = FULL || 4 * c < half;
        ea = HALF && turns ? 4 * c : 8 * c;
        eb = HALF && turns ? 4 * c + half : 8 * c + 4;
    }
    __device__ __forceinline__ void load(const uint16_t *at, uint2 (&r)[2]) const
    {
        if (HALF) {
            r[0] = __ldcs(reinterpret_cast<const uint2 *>(at + ea));
            r[1] = __ldcs(reinterpret_cast<const uint2 *>(at + eb));
        } else {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(at + ea));
            r[0] = make_uint2(v.x, v.y);
            r[1] = make_uint2(v.z, v.w);
        }
    }
    __device__ __forceinline__ void store(uint16_t *at, const uint2 (&r)[2]) const
    {
        if (HALF) {
            __stcs(reinterpret_cast<uint2 *>(at + ea), r[0]);
            __stcs(reinterpret_cast<uint2 *>(at + eb), r[1]);
        } else {
            __stcs(reinterpret_cast<uint4 *>(at + ea), make_uint4(r[0].x, r[0].y, r[1].x, r[1].y));
        }
    }
    // row: the angles of this lane's pairs, cosines and, half further on, sines (read
    // where the lane turns any); weight: [D] or nullptr
    __device__ __forceinline__ void fold(const float *row, const float *weight)
    {
        float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turns && half) {
            cs = __ldg(reinterpret_cast<const float4 *>(row));
            sn = __ldg(reinterpret_cast<const float4 *>(row + half));
        }
        float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
        if (weight) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(weight + ea));
            const float4 w = __ldg(reinterpret_cast<const float4 *>(weight + eb));
            if (HALF) {
                wa[0] = v.x; wa[1] = v.y; wa[2] = v.z; wa[3] = v.w;
                wb[0] = w.x; wb[1] = w.y; wb[2] = w.z; wb[3] = w.w;
            } else {
                wa[0] = v.x; wb[0] = v.y; wa[1] = v.z; wb[1] = v.w;
                wa[2] = w.x; wb[2] = w.y; wa[3] = w.z; wb[3] = w.w;
            }
        }
        const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            ac[i] = wa[i] * cv[i];
            as[i] = wa[i] * sv[i];
            bc[i] = wb[i] * cv[i];
            bs[i] = wb[i] * sv[i];
        }
    }
    // the new elements of a head, by its whole group of lanes (of a converged warp)
    __device__ __forceinline__ void apply(uint2 (&r)[2], bool norm, float eps) const
    {
        constexpr int kLanes = D / 8;
        float a[4], b[4];
        unpack<E, HALF>(r, a, b);
        if (norm) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                s0 = fmaf(a[i], a[i], s0);
                s1 = fmaf(b[i], b[i], s1);
            }
            float ss = s0 + s1;
#pragma unroll
            for (int k = kLanes / 2; k > 0; k /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, k);
            const float rs = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                a[i] *= rs;
                b[i] *= rs;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float v = a[i], w = b[i];
            a[i] = v * ac[i];
            b[i] = w * bc[i];
            if (turns) {                                 // 0 times an infinity would not be 0
                a[i] = fmaf(-w, bs[i], a[i]);
                b[i] = fmaf(v, as[i], b[i]);
            }
        }
        pack<E, HALF>(a, b, r);
    }
};

}  // namespace kda
