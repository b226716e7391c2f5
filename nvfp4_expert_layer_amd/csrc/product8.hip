// Products of MXFP8 rows with MXFP4 weights (W4A8, gfx950), rows sorted by group:
//   out[r][n] = sum_k a[r][k] w[g(r)][n][k]
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both formats as they lie in memory.  Operand
// layouts (checked on the device): of the 128 k of a step, lane l of the FP4 operand holds the
// 32 codes of block l / 16 of row l % 16; of the FP8 operand the 16 codes from 16 (l / 16) and
// the 16 from 64 + 16 (l / 16) of column l % 16; both give the scale of block l / 16.  The
// accumulator's element v sits at row 4 (l / 16) + v, column l % 16.  The weight is the row
// operand, tokens are columns, so a lane ends with four consecutive outputs of one token.
//
// The unit adds the products of eight neighbouring k aligned to the largest, without the bits
// below 2^-13 of it (checked on the device); everything beyond is fp32.
#include "block.h"
#include "product_common.h"

namespace moe {

__device__ __forceinline__ f32x4_t mfma_w4a8_16(const u32x4_t& w, uint32_t ws, const u32x4_t& lo, const u32x4_t& hi,
                                                uint32_t as, const f32x4_t& c) {
    const i32x8_t a = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(w), a, c, 4, 0, 0, (int)ws, 0, (int)as);
}

constexpr int kSWaves = 4;

// One pass over 16 weight rows' K for NT tiles of 16 tokens from row r0; the waves take units
// of 256 k in turn and join their sums in LDS in wave order.
template <int NT>
__device__ __forceinline__ void stream8_tiles(const ProductArgs& p, int g, int r0, int re, int n0, f32x4_t* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, lg = lane >> 4;
    const int KB = p.K / 32;
    const int64_t n = (int64_t)g * p.N + min(n0 + col, p.N - 1);                     // rows past N: any valid row
    const uint8_t* wrow = p.w + n * (p.K / 2);
    const uint8_t* srow = p.w_s + n * KB;
    const uint8_t* a = static_cast<const uint8_t*>(p.a);
    f32x4_t acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int u = wave; u * 8 < KB; u += kSWaves) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k0 = (u * 8 + s * 4) * 32, kb = u * 8 + s * 4 + lg;            // the step's first k, this lane's block
            const bool kv = kb < KB;
            u32x4_t wc = {0u, 0u, 0u, 0u};
            uint32_t ws = 0u;
            if (kv) {
                wc = *reinterpret_cast<const u32x4_t*>(wrow + (int64_t)kb * 16);
                ws = srow[kb];
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int64_t r = r0 + 16 * t + col;
                const int ka = k0 + 16 * lg;
                u32x4_t lo = {0u, 0u, 0u, 0u}, hi = {0u, 0u, 0u, 0u};
                uint32_t as = 0u;
                if (r < re) {
                    if (ka < p.K) lo = *reinterpret_cast<const u32x4_t*>(a + r * p.K + ka);
                    if (ka + 64 < p.K) hi = *reinterpret_cast<const u32x4_t*>(a + r * p.K + ka + 64);
                    if (kv) as = p.a_s[r * KB + kb];
                }
                acc[t] = mfma_w4a8_16(wc, ws, lo, hi, as, acc[t]);
            }
        }
    }
    __syncthreads();                                            // red's previous readers are done
#pragma unroll
    for (int t = 0; t < NT; ++t) red[(wave * NT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int x = threadIdx.x; x < NT * 64; x += 64 * kSWaves) {
        f32x4_t s = red[x];
#pragma unroll
        for (int w = 1; w < kSWaves; ++w) s += red[w * NT * 64 + x];
        const int l = x & 63, r = r0 + 16 * (x >> 6) + (l & 15), o = n0 + 4 * (l >> 4);
        if (r < re) store4(p.out, p.out_dtype, r * p.os + o, s, p.N - o);
    }
}

__global__ __launch_bounds__(64 * kSWaves) void product8_stream_kernel(ProductArgs p, int by_rank) {
    __shared__ f32x4_t red[kSWaves * 4 * 64];
    const int g = by_rank ? nth_group(p, blockIdx.y) : (int)blockIdx.y;
    if (g < 0) return;
    int rb, re;
    group_rows(p, g, rb, re);
    for (int r0 = rb; r0 < re;) {
        const int left = re - r0;
        if (left > 32) { stream8_tiles<4>(p, g, r0, re, blockIdx.x * 16, red); r0 += 64; }
        else if (left > 16) { stream8_tiles<2>(p, g, r0, re, blockIdx.x * 16, red); r0 += 32; }
        else { stream8_tiles<1>(p, g, r0, re, blockIdx.x * 16, red); r0 += 16; }
    }
}

hipError_t launch_product8(const ProductArgs& p, int cus, hipStream_t s) {
    const int groups = min(p.G, p.M);                           // at most so many hold rows
    hipLaunchKernelGGL(product8_stream_kernel, dim3((p.N + 15) / 16, groups), dim3(64 * kSWaves), 0, s, p,
                       p.M < p.G ? 1 : 0);
    return hipGetLastError();
}

}  // namespace moe
