// act8.cuh -- 8-bit activation checkpoints: quantize and dequantize.
//
// Blocks of 32 consecutive values of a row share one power-of-two scale 2^e,
// stored as the byte e + 127.  With the block's largest magnitude
// amax = 1.m 2^x (bf16: x and the 7 bits of m are bit fields),
//   int8   e = max(x - 6, -127): amax / 2^e in [64, 128), code = the nearest
//          integer (ties to even), 127.5 -> 127
//   E4M3   e = max(x - 8, -127), one more where 1.m > 1.75, so that
//          amax / 2^e <= 448, code = the nearest E4M3 value (ties to even)
// and the value is code * 2^e.  A power of two costs up to one bit of the
// code's range against the amax / 127 scale of the 8-bit optimizer states, and
// in exchange division, multiplication and the way back are exact: a code has
// at most 7 (int8) or 4 (E4M3) significant bits, so the restored value is a
// bf16 number and whatever reads the checkpoint computes with exactly the
// tensor that act8_dequant writes.  The only rounding is the code's own.
// A block that holds an infinity or a NaN gets the byte 255 and restores to
// NaN throughout, so that a broken step stays visible.
//
// Both directions are HBM streams (2 B in and 1 + 1/32 B out per value, or
// the reverse).  A warp takes segments of 4 x 256 values; per pass, lane l
// holds values 8l..8l+7, so loads and stores of every instruction are
// contiguous across the warp and the block maximum is two shuffles over 4
// lanes on packed 16-bit integers (the magnitude order of bf16 is the order
// of its bit patterns).  4096 x 28672 int8 (356 MB either way): 59 us to quantize,
// 53 us back, of 54 at the copy rate.  Launched programmatically: a kernel waits for the one
// before it before it reads anything.
#pragma once
#include "common.cuh"
#include "adamw8.cuh"

namespace qnf4 {
namespace act8 {

constexpr int kThreads = 256;
constexpr int kPasses = 4;                        // 16-byte loads in flight per lane
constexpr int kWarpChunks = 32 * kPasses;         // chunks of 8 values per warp

// CTAs for n8 chunks (n8 <= 2^37: the most that act8_sizes admits)
inline unsigned grid_of(int64_t n8) { return (unsigned)cdiv(n8, (int64_t)kWarpChunks * (kThreads / 32)); }

// fp32 value of the scale byte: 2^(b - 127), 2^-127 as a subnormal, 255 -> NaN
__device__ __forceinline__ float scale_of(uint32_t b) {
    uint32_t bits = b << 23;
    if (b == 0u) bits = 0x00400000u;
    if (b == 255u) bits = 0x7fc00000u;
    return __uint_as_float(bits);
}

// the values of four codes (one 32-bit word)
template <bool E4M3>
__device__ __forceinline__ void values4(uint32_t w, float (&v)[4]) {
    if (E4M3) {
        const float2 a = adam::e4m3x2_to_f32(w), b = adam::e4m3x2_to_f32(w >> 16);
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
        // two's complement byte c: bits of 2^23 + (c + 128), minus 2^23 + 128, is c
        const uint32_t u = w ^ 0x80808080u;
        constexpr float kBias = 8388608.f + 128.f;
        v[0] = __uint_as_float(prmt(u, 0x4b000000u, 0x7540u)) - kBias;
        v[1] = __uint_as_float(prmt(u, 0x4b000000u, 0x7541u)) - kBias;
        v[2] = __uint_as_float(prmt(u, 0x4b000000u, 0x7542u)) - kBias;
        v[3] = __uint_as_float(prmt(u, 0x4b000000u, 0x7543u)) - kBias;
    }
}

// four codes times s, as two packed bf16 pairs
template <bool E4M3>
__device__ __forceinline__ void restore4(uint32_t w, float s, uint32_t& lo, uint32_t& hi) {
    float v[4];
    values4<E4M3>(w, v);
    lo = pack_bf16x2(v[0] * s, v[1] * s);
    hi = pack_bf16x2(v[2] * s, v[3] * s);
}

// n8: chunks of 8 values (a multiple of 4: blocks of 32 are whole)
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) k_act8_quantize(const uint16_t* __restrict__ X, int64_t n8,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t c0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kWarpChunks + lane;
    uint4 x[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t c = c0 + 32 * p;
        x[p] = c < n8 ? ldg_nc_v4(X + 8 * c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t c = c0 + 32 * p;
        const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
        uint32_t a = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                              __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int amax = (int)max(a & 0xffffu, a >> 16);
        const bool bad = amax >= 0x7f80;
        int sb = E4M3 ? (amax >> 7) - 8 + ((amax & 0x7f) > 0x60 ? 1 : 0) : (amax >> 7) - 6;
        sb = bad ? 255 : max(sb, 0);
        // 2^-e = 2^(127 - sb); sb <= 249
        const float inv = bad ? 0.f : __uint_as_float((uint32_t)(254 - sb) << 23);
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float v0 = bf16lo_to_f32(w[2 * h]), v1 = bf16hi_to_f32(w[2 * h]);
            const float v2 = bf16lo_to_f32(w[2 * h + 1]), v3 = bf16hi_to_f32(w[2 * h + 1]);
            if (E4M3) {
                o[h] = adam::f32x2_to_e4m3(v0 * inv, v1 * inv) | (adam::f32x2_to_e4m3(v2 * inv, v3 * inv) << 16);
            } else {
                // v inv + 1.5 2^23 rounds v inv to an integer in the low bits, two's complement
                constexpr float kM = 12582912.f;
                auto enc = [&](float v) {
                    return __float_as_uint(fminf(fmaxf(__fmaf_rn(v, inv, kM), kM - 127.f), kM + 127.f));
                };
                o[h] = prmt(prmt(enc(v0), enc(v1), 0x0040u), prmt(enc(v2), enc(v3), 0x0040u), 0x5410u);
            }
        }
        if (bad) o[0] = o[1] = 0u;
        if (c < n8) {
            *reinterpret_cast<uint2*>(codes + 8 * c) = make_uint2(o[0], o[1]);
            if ((lane & 3) == 0) scales[c >> 2] = (uint8_t)sb;
        }
    }
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) k_act8_dequant(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t n8,
                                                           uint16_t* __restrict__ out) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t c0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kWarpChunks + lane;
    uint2 q[kPasses];
    uint32_t sb[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t c = c0 + 32 * p;
        q[p] = make_uint2(0, 0);
        sb[p] = 0;
        if (c < n8) {
            q[p] = __ldg(reinterpret_cast<const uint2*>(codes + 8 * c));
            sb[p] = __ldg(scales + (c >> 2));
        }
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t c = c0 + 32 * p;
        const float s = scale_of(sb[p]);
        uint4 o;
        restore4<E4M3>(q[p].x, s, o.x, o.y);
        restore4<E4M3>(q[p].y, s, o.z, o.w);
        if (c < n8) *reinterpret_cast<uint4*>(out + 8 * c) = o;
    }
}

}  // namespace act8
}  // namespace qnf4
