// Device helpers of the full-attention kernels: rotation angles, head rows of
// eight channels a lane, e8m0 scales, page lookups.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace gdn {
namespace attn {

// Waits for the previous grid on the stream, then lets the next one be
// scheduled: not before, as a kernel that reads constants ahead of its own wait
// (the delta-rule decode its convolution taps) would read them before a copy
// still running two launches back.
__device__ __forceinline__ void grid_dep_enter() {
    grid_dep_wait();
    grid_dep_launch();
}

// cos and sin of position * frequency.  freq is in turns per position as a
// 64-bit binary fraction, so the product mod 2^64 is the angle's exact
// fraction of a turn (the integer multiply drops whole turns).  Its upper 32
// bits, plus an eighth of a turn, give the quadrant (two bits) and the angle
// from the quadrant's middle, t within +-pi/4, rounded to f32; there the Taylor
// series to t^9 and t^8 are off by less than 2^-25 (t^11/11!, t^10/10!).
__device__ __forceinline__ void rope_angle(long long pos, uint64_t freq, float &c, float &s) {
    const uint32_t turns = (uint32_t)(((uint64_t)pos * freq) >> 32) + 0x20000000u;
    const float t = (float)((int32_t)(turns & 0x3fffffffu) - 0x20000000) * 1.4629180792671596e-9f;   // pi 2^-31
    const float t2 = t * t;
    const float sn = t * fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
    const float cs = fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const bool odd = turns & 0x40000000u, neg = turns & 0x80000000u;
    // quadrants 0..3: (cos, sin), (-sin, cos), (-cos, -sin), (sin, -cos)
    const float x = odd ? -sn : cs, y = odd ? cs : sn;
    c = neg ? -x : x;
    s = neg ? -y : y;
}

// Eight bf16 (16 bytes) to f32 and back.
__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// The value of an e8m0 byte, 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
}

// The e8m0 byte of the smallest power of two s >= 2^-127 with amax <= 448 s,
// from amax's bits (448 = 1.75 * 2^8); 255 for an infinity or NaN.
__device__ __forceinline__ uint32_t e8m0_for(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);
    if (e == 255) return 255u;
    const int byte = e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(byte < 0 ? 0 : byte);
}

// 1 / e8m0_value(byte), exact (byte <= 247 for a finite row); NaN for 255.
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
    return __uint_as_float(byte == 255 ? 0x7fffffffu : (254u - byte) << 23);
}

// Eight f32 to e4m3 codes, round to nearest even.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack8_e4m3(const uint2 &r, float (&x)[8]) {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The cache row (in units of D channels) of head h at position p of a row
// whose page-table line is `line`, or -1 without a valid page.
__device__ __forceinline__ long long cache_row(const PagedCache &c, int Hkv, const int32_t *line, long long p, int h) {
    if (p < 0 || (p >> c.shift) >= c.width) return -1;
    const int32_t page = line[p >> c.shift];
    if (page < 0 || page >= c.n_pages) return -1;
    return (((long long)page * Hkv + h) << c.shift) + (p & (c.page - 1));
}

__device__ __forceinline__ int clamp_new(const int32_t *n_new, int b, int T) {
    return n_new == nullptr ? T : min(max(n_new[b], 0), T);
}

}  // namespace attn
}  // namespace gdn
