// quant.cuh - MXFP8 (OCP MX: E4M3 elements, one E8M0 scale per 32) on the
// device: the block quantiser in its two forms (one thread per block of 32, or
// four neighbouring lanes with 8 elements each) and the way back. Both forms
// take the scale from the block's largest magnitude by e8m0_code and round by
// f32x2_to_e4m3x2, so they give the same bytes.
#pragma once

#include "common.cuh"

namespace mok {

// One 32-element MXFP8 block: E8M0 code of its amax, E4M3 bytes of x / scale.
// One thread holds the block; quantize8 below is the same rule over four lanes.
__device__ __forceinline__ uint32_t quantize32(const float (&f)[32], uint4& o0, uint4& o1) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(f[i]));
    const uint32_t code = e8m0_code(amax);
    const float inv = e8m0_inv_scale(code);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = f32x2_to_e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) |
               (f32x2_to_e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16);
    o0 = make_uint4(w[0], w[1], w[2], w[3]);
    o1 = make_uint4(w[4], w[5], w[6], w[7]);
    return code;
}

// 32 BF16 values (four 16-byte words) to fp32.
__device__ __forceinline__ void unpack32(const uint4 (&v)[4], float (&f)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[8 * i + 0] = bf16_lo(v[i].x); f[8 * i + 1] = bf16_hi(v[i].x);
        f[8 * i + 2] = bf16_lo(v[i].y); f[8 * i + 3] = bf16_hi(v[i].y);
        f[8 * i + 4] = bf16_lo(v[i].z); f[8 * i + 5] = bf16_hi(v[i].z);
        f[8 * i + 6] = bf16_lo(v[i].w); f[8 * i + 7] = bf16_hi(v[i].w);
    }
}

__device__ __forceinline__ uint32_t quantize_block32(const __nv_bfloat16* src, uint4& o0, uint4& o1) {
    const uint4* s4 = reinterpret_cast<const uint4*>(src);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldg(s4 + i);
    float f[32];
    unpack32(v, f);
    return quantize32(f, o0, o1);
}

// 8 of a block's 32 elements in each of four neighbouring lanes (lane % 4 =
// position in the block; all four call together): the E8M0 code (the same in
// the four lanes) and this lane's E4M3 bytes.
__device__ __forceinline__ uint32_t quantize8(const float (&f)[8], uint2& o) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = e8m0_code(amax);
    const float inv = e8m0_inv_scale(code);
    o.x = f32x2_to_e4m3x2(f[0] * inv, f[1] * inv) | (f32x2_to_e4m3x2(f[2] * inv, f[3] * inv) << 16);
    o.y = f32x2_to_e4m3x2(f[4] * inv, f[5] * inv) | (f32x2_to_e4m3x2(f[6] * inv, f[7] * inv) << 16);
    return code;
}

// The same from 8 BF16 values: the maximum is taken on packed pairs (it is one of
// the values, so no rounding is involved).
__device__ __forceinline__ uint32_t quantize8_bf16(const uint4& v, uint2& o) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    auto bf2 = [](uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); };
    __nv_bfloat162 m = __hmax2(__hmax2(bf2(w[0] & 0x7fff7fffu), bf2(w[1] & 0x7fff7fffu)),
                               __hmax2(bf2(w[2] & 0x7fff7fffu), bf2(w[3] & 0x7fff7fffu)));
    uint32_t b = *reinterpret_cast<uint32_t*>(&m);
    uint32_t a = max(b << 16, b & 0xffff0000u);   // non-negative fp32 patterns order like whole numbers
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t code = e8m0_code(__uint_as_float(a));
    const float inv = e8m0_inv_scale(code);
    const float2 inv2 = make_float2(inv, inv);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __fmul2_rn(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), inv2);
        q[i] = f32x2_to_e4m3x2(f.x, f.y);
    }
    o.x = q[0] | (q[1] << 16);
    o.y = q[2] | (q[3] << 16);
    return code;
}

// 8 BF16 values (one 16-byte word) to fp32 and back.
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// 2^(code - 127), exact for every code below 255 (code 0 is a subnormal).
__device__ __forceinline__ float e8m0_scale(uint32_t code) {
    return code ? __uint_as_float(code << 23) : __uint_as_float(1u << 22);
}

// Values 2i and 2i + 1 of 8 E4M3 bytes, without their block's scale. E4M3 converts
// exactly to FP16 and on to fp32.
__device__ __forceinline__ float2 e4m3_pair(const uint2& q, int i) {
    const __nv_fp8x2_storage_t pair = (__nv_fp8x2_storage_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1)));
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3)));
}

// The values that 8 E4M3 bytes and their block's scale code stand for. The scale is
// a power of two, so every value is exact (and, with 4 significant bits, a BF16
// number).
__device__ __forceinline__ void dequantize8(const uint2& q, uint32_t code, float (&f)[8]) {
    const float s = e8m0_scale(code);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = e4m3_pair(q, i);
        f[2 * i] = v.x * s;
        f[2 * i + 1] = v.y * s;
    }
}

}  // namespace mok
