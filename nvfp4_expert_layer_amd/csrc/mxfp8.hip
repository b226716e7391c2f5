// MXFP8 quantizer and dequantizer (gfx950): E4M3 codes, one E8M0 scale per 32 elements.
//
// Both are bound by memory and laid out as MXFP4's: eight elements a thread, four
// neighbouring threads a block.  65536 x 4096 from bf16 135 us (6.0 TB/s), back 124 us (6.5).
#include "block.h"
#include "eights.h"
#include "mx_common.h"

namespace moe {

// Piece i: eight elements.  per_row pieces a row; FLAT: rows follow each other without gaps
// (x is one long row).
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void mxfp8_quantize_kernel(const void* __restrict__ x, int64_t pieces, int per_row,
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
        const uint32_t sb = mx8_scale(quad_max(top_bits<DT>(w)));
        __builtin_nontemporal_store(mx8_encode8<DT>(w, sb), reinterpret_cast<u32x2_t*>(codes + i * 8));
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)sb;
    }
}

// Piece i: eight codes, 16 or 32 bytes of output; per_row pieces a row.
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void mxfp8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t pieces,
                                                               int per_row, void* __restrict__ out, int64_t os) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += stride) {
        int64_t el = i * 8;
        if (!FLAT) {
            const int64_t r = i / per_row;
            el = r * os + (i - r * per_row) * 8;
        }
        float f[8];
        mx8_decode8(*reinterpret_cast<const u32x2_t*>(codes + i * 8), scales[i >> 2], f);
        store8<DT>(out, el, f);
    }
}

// Blocks of 256 threads: one piece a thread, and a grid-stride loop beyond 2^22 blocks (a
// grid holds fewer than 2^32 threads).
static unsigned piece_blocks(int64_t pieces) {
    const int64_t n = (pieces + 255) / 256;
    return (unsigned)(n < (1 << 22) ? n : (1 << 22));
}

template <int DT>
static void quantize_dt(const void* x, int64_t R, int C, int64_t xs, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const int64_t pieces = R * (C / 8);
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(piece_blocks(pieces)), dim3(256), 0, s, x, pieces, C / 8, xs, codes, scales);
    };
    R == 1 || xs == C ? run(mxfp8_quantize_kernel<DT, true>) : run(mxfp8_quantize_kernel<DT, false>);
}

template <int DT>
static void dequantize_dt(const uint8_t* codes, const uint8_t* scales, int64_t R, int C, void* out, int64_t os,
                          hipStream_t s) {
    const int64_t pieces = R * (C / 8);
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(piece_blocks(pieces)), dim3(256), 0, s, codes, scales, pieces, C / 8, out, os);
    };
    R == 1 || os == C ? run(mxfp8_dequantize_kernel<DT, true>) : run(mxfp8_dequantize_kernel<DT, false>);
}

hipError_t launch_mxfp8_quantize(const void* x, int dtype, int64_t R, int C, int64_t xs, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
    if (dtype == kBF16) quantize_dt<kBF16>(x, R, C, xs, codes, scales, s);
    else if (dtype == kF16) quantize_dt<kF16>(x, R, C, xs, codes, scales, s);
    else quantize_dt<kF32>(x, R, C, xs, codes, scales, s);
    return hipGetLastError();
}

hipError_t launch_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int C, int dtype,
                                   void* out, int64_t os, hipStream_t s) {
    if (dtype == kBF16) dequantize_dt<kBF16>(codes, scales, R, C, out, os, s);
    else if (dtype == kF16) dequantize_dt<kF16>(codes, scales, R, C, out, os, s);
    else dequantize_dt<kF32>(codes, scales, R, C, out, os, s);
    return hipGetLastError();
}

}  // namespace moe
