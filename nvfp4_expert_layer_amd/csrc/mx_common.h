// Device helpers of the microscaling formats (MXFP4, MXFP8): a block is 32 consecutive
// elements of a row, eight a thread, four neighbouring threads a block.
#pragma once
#include "device_common.h"
#include "ops.h"

namespace moe {

constexpr int kMx = 32;

// Maximum over a quad of lanes (lanes 4 i .. 4 i + 3).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);   // quad_perm 1,0,3,2
    v = v > a ? v : a;
    const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);   // quad_perm 2,3,0,1
    return v > b ? v : b;
}

// fp32 magnitude bits of eight loaded elements: the largest (integers order as the
// magnitudes do; Inf and NaN are above every finite value).
template <int DT>
__device__ __forceinline__ uint32_t top_bits(const uint32_t (&w)[DT == kF32 ? 8 : 4]) {
    uint32_t m = 0;
    if constexpr (DT == kF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    } else {
        uint32_t h = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = max(m, w[i] & 0x7FFFu);
            h = max(h, w[i] & 0x7FFF0000u);
        }
        if constexpr (DT == kBF16) return max(h, m << 16);
        m = max(m, h >> 16);
        return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)m));
    }
}

// ---------------------------------------------------------------------------
// MXFP8.  With E the biased fp32 exponent of the block's largest magnitude the scale byte
// is s = max(E - 8, 0): floor(log2 amax) - emax(E4M3) + 127, emax = 8; 255 where the block
// holds an Inf or NaN.  v_cvt_scalef32_pk_fp8_* divides by 2^(s - 127) and rounds to nearest,
// ties to even, for every scale byte, subnormal codes too (checked on the device on both sides
// of every midpoint); from 464 on it gives NaN, which is made 448.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t mx8_scale(uint32_t top) {
    const int field = (int)(top >> 23);
    return field == 255 ? 255u : (uint32_t)max(field - 8, 0);
}

// Four E4M3 bytes: NaN (only from an overflow) -> the largest magnitude, the sign kept.
__device__ __forceinline__ uint32_t mx8_saturate(uint32_t c) {
    return c - ((((c & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u);
}

// Eight loaded elements -> eight codes under scale byte sb.
template <int DT>
__device__ __forceinline__ u32x2_t mx8_encode8(const uint32_t (&w)[DT == kF32 ? 8 : 4], uint32_t sb) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float scale = __uint_as_float(sb << 23);
    s16x2 c[2] = {{0, 0}, {0, 0}};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if constexpr (DT == kF32) {
            c[q] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c[q], __uint_as_float(w[4 * q]), __uint_as_float(w[4 * q + 1]),
                                                            scale, false);
            c[q] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c[q], __uint_as_float(w[4 * q + 2]),
                                                            __uint_as_float(w[4 * q + 3]), scale, true);
        } else if constexpr (DT == kBF16) {
            c[q] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c[q], __builtin_bit_cast(bf16x2_t, w[2 * q]), scale, false);
            c[q] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c[q], __builtin_bit_cast(bf16x2_t, w[2 * q + 1]), scale, true);
        } else {
            c[q] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c[q], __builtin_bit_cast(f16x2_t, w[2 * q]), scale, false);
            c[q] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c[q], __builtin_bit_cast(f16x2_t, w[2 * q + 1]), scale, true);
        }
    }
    if (sb == 255u) return u32x2_t{0u, 0u};
    return u32x2_t{mx8_saturate(__builtin_bit_cast(uint32_t, c[0])), mx8_saturate(__builtin_bit_cast(uint32_t, c[1]))};
}

// The block's scale byte and this thread's eight codes, of eight fp32 values a thread and
// four threads (a quad of lanes) a block.
__device__ __forceinline__ u32x2_t mx8_quantize8(const float (&f)[8], uint32_t& sb) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
    sb = mx8_scale(quad_max(top_bits<kF32>(w)));
    return mx8_encode8<kF32>(w, sb);
}

// Eight codes under scale byte sb -> fp32 (exact; NaN where sb is 255).
__device__ __forceinline__ void mx8_decode8(const u32x2_t& c, uint32_t sb, float (&f)[8]) {
    const float scale = __uint_as_float(sb << 23);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[q], scale, false);
        const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[q], scale, true);
        f[4 * q] = a[0]; f[4 * q + 1] = a[1]; f[4 * q + 2] = b[0]; f[4 * q + 3] = b[1];
    }
}

}  // namespace moe
