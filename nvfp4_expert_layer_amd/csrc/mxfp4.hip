// MXFP4 quantizer and dequantizer (gfx950).
//
// A block is 32 consecutive elements of a row.  With E the biased fp32 exponent of
// its largest magnitude (bf16 and f16 convert to fp32 exactly), the scale byte is
//   s = max(E - 2, 0):  floor(log2 amax) - emax(E2M1) + 127, emax = 2,
// and the codes are E2M1(x 2^(127 - s)), to nearest, ties to even, saturating.
// gfx950 converts with the block scale in one instruction per pair
// (v_cvt_scalef32_pk_fp4_{f32,bf16,f16}, and _pk_{f32,bf16}_fp4 back), which was
// checked on the device for every scale byte and on both sides of every midpoint;
// s = 0 (a subnormal fp32 scale operand) counts as 2^-127 and s = 255 gives NaN,
// as the format says.
//
// Both kernels are bound by memory.  Eight elements a thread, four neighbouring
// threads a block: 16-byte loads and stores of consecutive lanes are consecutive,
// and the block maximum takes two exchanges within a quad of lanes.  65536 x 4096: from
// fp32 200 us (6.1 TB/s), from bf16 114 us (6.0 TB/s); back to fp32 164 us (222 when no
// cache holds any of it), to bf16 93 us.
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

// Eight elements times 2^-(exponent of scale) -> eight E2M1 codes.
template <int DT>
__device__ __forceinline__ uint32_t encode8(const uint32_t (&w)[DT == kF32 ? 8 : 4], float scale) {
    uint32_t c = 0;
    if constexpr (DT == kF32) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[0]), __uint_as_float(w[1]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[2]), __uint_as_float(w[3]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[4]), __uint_as_float(w[5]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[6]), __uint_as_float(w[7]), scale, 3);
    } else if constexpr (DT == kBF16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[3]), scale, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[3]), scale, 3);
    }
    return c;
}

// Piece i: eight elements.  per_row pieces a row; FLAT: rows follow each other
// without gaps (x is one long row).
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const void* __restrict__ x, int64_t pieces, int per_row,
                                                             int64_t xs, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
    constexpr int W = DT == kF32 ? 8 : 4;
    const int64_t stride = (int64_t)gridDim.x * 256;
    // a quad's four pieces are one block: pieces is a multiple of 4, so quads are whole
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += stride) {
        int64_t el = i * 8;
        if (!FLAT) {
            const int64_t r = i / per_row;
            el = r * xs + (i - r * per_row) * 8;
        }
        uint32_t w[W];
        const u32x4_any_t* src = reinterpret_cast<const u32x4_any_t*>(static_cast<const char*>(x) + el * (W / 2));
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
            const u32x4_t v = src[q];
            w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
        }
        const int field = (int)(quad_max(top_bits<DT>(w)) >> 23);
        const bool bad = field == 255;                     // Inf or NaN in the block
        const uint32_t sb = bad ? 255u : (uint32_t)max(field - 2, 0);
        const uint32_t c = encode8<DT>(w, __uint_as_float(sb << 23));
        __builtin_nontemporal_store(bad ? 0u : c, reinterpret_cast<uint32_t*>(codes + i * 4));
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)sb;
    }
}

// Piece i: 16 bytes of output (eight 16-bit or four fp32 values), per_row pieces a row.
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t pieces,
                                                               int per_row, void* __restrict__ out, int64_t os) {
    constexpr int N = DT == kF32 ? 4 : 8;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += stride) {
        int64_t el = i * N;
        if (!FLAT) {
            const int64_t r = i / per_row;
            el = r * os + (i - r * per_row) * N;
        }
        const float s = __uint_as_float((uint32_t)scales[i / (kMx / N)] << 23);
        uint32_t w[4];                                     // the piece's bits
        if constexpr (DT == kF32) {
            const uint32_t c = *reinterpret_cast<const uint16_t*>(codes + i * 2);
            const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
            const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
            w[0] = __float_as_uint(a[0]); w[1] = __float_as_uint(a[1]);
            w[2] = __float_as_uint(b[0]); w[3] = __float_as_uint(b[1]);
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + i * 4);
            if constexpr (DT == kBF16) {
                w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
                w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
                w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
                w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
            } else {
                // through fp32: rounded to f16 once
                const f32x2_t v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0),
                                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
                                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2),
                                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3)};
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = f32_to_f16_bits(v[q][0]) | (f32_to_f16_bits(v[q][1]) << 16);
            }
        }
        // streaming stores of consecutive lanes' consecutive 16 bytes
        __builtin_nontemporal_store(u32x4_t{w[0], w[1], w[2], w[3]},
                                    reinterpret_cast<u32x4_any_t*>(static_cast<char*>(out) + el * (16 / N)));
    }
}

// Blocks of 256 threads: one piece a thread, and a grid-stride loop beyond 2^22
// blocks (a grid holds fewer than 2^32 threads).
static unsigned piece_blocks(int64_t pieces) {
    const int64_t n = (pieces + 255) / 256;
    return (unsigned)(n < (1 << 22) ? n : (1 << 22));
}

template <int DT>
static void quantize_dt(const void* x, int64_t R, int C, int64_t xs, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const int64_t pieces = R * (C / 8);
    const dim3 grid(piece_blocks(pieces));
    const bool flat = R == 1 || xs == C;
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, x, pieces, C / 8, xs, codes, scales);
    };
    flat ? run(mxfp4_quantize_kernel<DT, true>) : run(mxfp4_quantize_kernel<DT, false>);
}

template <int DT>
static void dequantize_dt(const uint8_t* codes, const uint8_t* scales, int64_t R, int C, void* out, int64_t os,
                          hipStream_t s) {
    constexpr int n = DT == kF32 ? 4 : 8;
    const int64_t pieces = R * (C / n);
    const dim3 grid(piece_blocks(pieces));
    const bool flat = R == 1 || os == C;
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, codes, scales, pieces, C / n, out, os);
    };
    flat ? run(mxfp4_dequantize_kernel<DT, true>) : run(mxfp4_dequantize_kernel<DT, false>);
}

hipError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t R, int C, int64_t xs, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
    if (dtype == kBF16) quantize_dt<kBF16>(x, R, C, xs, codes, scales, s);
    else if (dtype == kF16) quantize_dt<kF16>(x, R, C, xs, codes, scales, s);
    else quantize_dt<kF32>(x, R, C, xs, codes, scales, s);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int C, int dtype,
                                   void* out, int64_t os, hipStream_t s) {
    if (dtype == kBF16) dequantize_dt<kBF16>(codes, scales, R, C, out, os, s);
    else if (dtype == kF16) dequantize_dt<kF16>(codes, scales, R, C, out, os, s);
    else dequantize_dt<kF32>(codes, scales, R, C, out, os, s);
    return hipGetLastError();
}

}  // namespace moe
