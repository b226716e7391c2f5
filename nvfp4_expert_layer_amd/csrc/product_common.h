// Device helpers of the MXFP4 products: operand decoding, matrix instructions,
// group bounds, stores.
#pragma once
#include "device_common.h"
#include "ops.h"

typedef int i32x8_t __attribute__((ext_vector_type(8)));

namespace moe {

// Rows [rb, re) of group g, within [0, M].
__device__ __forceinline__ void group_rows(const ProductArgs& p, int g, int& rb, int& re) {
    if (!p.offsets) {
        rb = 0;
        re = p.M;
        return;
    }
    rb = min(max(p.offsets[g], 0), p.M);
    re = min(max(p.offsets[g + 1], rb), p.M);
}

// The i-th group that holds rows, or -1 (every wave finds it by itself).
__device__ __forceinline__ int nth_group(const ProductArgs& p, int i) {
    const int lane = threadIdx.x & 63;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
        int rb = 0, re = 0;
        if (g0 + lane < p.G) group_rows(p, g0 + lane, rb, re);
        uint64_t m = __ballot(re > rb);
        const int n = __popcll(m);
        if (i < n) {
            for (; i > 0; --i) m &= m - 1;
            return g0 + __ffsll((unsigned long long)m) - 1;
        }
        i -= n;
    }
    return -1;
}

// Eight E2M1 codes times 2^(exponent of sc) -> eight bf16 (exact).
__device__ __forceinline__ u32x4_t mx_decode8(uint32_t codes, float sc) {
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 3))};
}

// Eight rows' dwords of eight codes with their scale bytes -> op[c]: column c of the
// eight rows, as bf16.
__device__ __forceinline__ void mx_decode_columns(const uint32_t (&code)[8], const uint32_t (&sb)[8],
                                                  u32x4_t (&op)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const u32x4_t a = mx_decode8(code[j], __uint_as_float(sb[j] << 23));
        const u32x4_t b = mx_decode8(code[j + 1], __uint_as_float(sb[j + 1] << 23));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            op[2 * q][j / 2] = __builtin_amdgcn_perm(b[q], a[q], 0x05040100u);
            op[2 * q + 1][j / 2] = __builtin_amdgcn_perm(b[q], a[q], 0x07060302u);
        }
    }
}

__device__ __forceinline__ i32x8_t mx_operand(const u32x4_t& c) {
    return i32x8_t{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};       // fp4 uses the first four dwords
}

// 16 x 16 x 128, both operands MXFP4, scale in the low byte.
__device__ __forceinline__ f32x4_t mfma_mx16(const u32x4_t& a, uint32_t as, const u32x4_t& b, uint32_t bs,
                                             const f32x4_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, 0, (int)as, 0,
                                                            (int)bs);
}

__device__ __forceinline__ f32x4_t mfma_bf16_16(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}

// Eight bf16 from p (at any element), of which `left` exist (the others 0).
__device__ __forceinline__ u32x4_t load8_bf16(const uint16_t* p, int left) {
    if (left >= 8) return *reinterpret_cast<const u32x4_any_t*>(p);
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return v;
}

// Four outputs to two dwords of bf16 or f16.
__device__ __forceinline__ u32x2_t pack4(int dtype, float a, float b, float c, float d) {
    if (dtype == kBF16) return u32x2_t{f32x2_to_bf16x2(a, b), f32x2_to_bf16x2(c, d)};
    return u32x2_t{f32_to_f16_bits(a) | (f32_to_f16_bits(b) << 16), f32_to_f16_bits(c) | (f32_to_f16_bits(d) << 16)};
}

// Four consecutive outputs of a row, of which `left` exist, at element `el`.
__device__ __forceinline__ void store4(void* out, int dtype, int64_t el, const f32x4_t& f, int left) {
    if (dtype == kF32) {
        float* o = static_cast<float*>(out) + el;
        if (left >= 4) {
            *reinterpret_cast<u32x4_any_t*>(o) = __builtin_bit_cast(u32x4_t, f);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) o[i] = f[i];
        return;
    }
    const u32x2_t v = pack4(dtype, f[0], f[1], f[2], f[3]);
    uint16_t* o = static_cast<uint16_t*>(out) + el;
    if (left >= 4) {
        *reinterpret_cast<u32x2_any_t*>(o) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
}

// dout's rows lie in aligned 16-byte pieces that end with the row (direct loads to LDS).
inline bool dout_vector(const ProductArgs& p) {
    return p.N % 8 == 0 && (p.M <= 1 || p.as % 8 == 0) && (reinterpret_cast<uintptr_t>(p.a) & 15) == 0;
}

}  // namespace moe
