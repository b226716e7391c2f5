// Products with MXFP4 weights over rows sorted by group, few rows a group (gfx950):
//   forward   out[r][n]   = sum_k a[r][k] w[g(r)][n][k]
//   backward  drows[r][k] = sum_n dout[r][n] w[g(r)][n][k]
// With few rows the weight's bytes are the whole cost: each group's weight is read once
// from memory per 16 to 64 of its rows, straight into registers in matrix-core operand
// order; a workgroup's waves split the reduction and join their sums in LDS in wave
// order, so nothing depends on timing.
//
//   product_resident_kernel  forward, K up to 4096 (MXFP4, MXFP8 rows: 8192).  512 rows over
//       160 experts of 2048 x 4096: W4A16 131 us, 5.4 TB/s, W4A4 122 us, 5.8 TB/s, W4A8 125 us
//       (a large copy: 4.95); one row of 2048 x 4096: 4.9 us.  The form below it, which loads tokens
//       again for each weight tile, took 216 us for the 512 rows.
//   product_stream_kernel    forward, longer K.
//   product_grad_stream_kernel  512 rows over 160 experts: 236 us, 3.0 TB/s (268 before
//       neighbouring column blocks met on one XCD); one row 8 us.  Bound by its 4-byte
//       loads (eight weight rows a lane) and their latency: without the next step's loads
//       in flight 603 us.
//
// Operand layouts (v_mfma_*_16x16x*): lane l holds row (or column) l % 16 and the K
// slice of lane group l / 16; the accumulator's element v sits at row 4 (l/16) + v,
// column l % 16.  The weight is the row operand, tokens are columns, so a lane ends with
// four consecutive outputs of one token.
//   W4A4: v_mfma_scale_f32_16x16x128_f8f6f4 takes 32 codes (16 bytes) and one E8M0
//     scale a lane: one 32-element block as it lies in memory, no decoding.
//   W4A8: the same instruction with FP8 columns (two pieces of 16 k a lane).
//   W4A16: 16 bytes of codes are four operands of v_mfma_f32_16x16x32_bf16;
//     v_cvt_scalef32_pk_bf16_fp4 decodes a pair with its block scale, exactly.
#include "device_common.h"
#include "ops.h"
#include "product_common.h"

namespace moe {

constexpr int kSWaves = 4;

// How the rows are held.
enum RowFormat { kRowsBf16, kRowsMx4, kRowsMx8 };

// A lane's tokens of block kb of row r (bf16, MXFP4), or its two pieces of 16 k of the step of 128
// that the block is in (MXFP8: the FP8 operand's lane group lg holds k 16 lg .. + 16 and 64 + 16 lg
// .. + 16), 16 bytes a load, and the block's scale; 0 where they pass K or the row is not `valid`.
// (MXFP4: codes and scale under one condition, rows of 32 bits.  With the scale's load apart and rows of
// 64 bits three rows of 2048 x 8224 took W4A4 6.2 us, now 5.7, W4A8 8.2, now 7.0.)
template <int FMT> constexpr int kTokenLoads = FMT == kRowsMx4 ? 1 : (FMT == kRowsMx8 ? 2 : 4);
template <int FMT>
__device__ __forceinline__ void load_token(const ProductArgs& p, int r, int kb, int lg, bool valid,
                                           u32x4_t (&v)[kTokenLoads<FMT>], uint32_t& scale) {
    const int KB = p.K / 32;
    const bool in = kb < KB && valid;
    scale = 0u;
    if constexpr (FMT == kRowsMx4) {
        v[0] = u32x4_t{0u, 0u, 0u, 0u};
        if (in) {
            v[0] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(p.a) + (int64_t)r * (p.K / 2) +
                                                     (int64_t)kb * 16);
            scale = p.a_s[(int64_t)r * KB + kb];
        }
    } else {
#pragma unroll
        for (int q = 0; q < kTokenLoads<FMT>; ++q) {
            v[q] = u32x4_t{0u, 0u, 0u, 0u};
            if constexpr (FMT == kRowsMx8) {
                const int k = (kb - lg) * 32 + 64 * q + 16 * lg;
                if (valid && k < p.K)
                    v[q] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(p.a) + (int64_t)r * p.K + k);
            } else if (in) {
                v[q] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p.a) + (int64_t)r * p.as +
                                                         (int64_t)kb * 32 + 8 * q);
            }
        }
        if (FMT == kRowsMx8 && in) scale = p.a_s[(int64_t)r * KB + kb];
    }
}

// One step of 128 k: 16 weight rows' codes and scale byte, 16 tokens.
template <int FMT>
__device__ __forceinline__ f32x4_t mfma_mx(const u32x4_t& w, uint32_t ws, const u32x4_t (&a)[kTokenLoads<FMT>],
                                           uint32_t as, const f32x4_t& c) {
    if constexpr (FMT == kRowsMx4) return mfma_mx16(w, ws, a[0], as, c);
    else return mfma_w4a8_16(w, ws, a[0], a[1], as, c);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// One pass over the weight tile's K for NT tiles of 16 tokens from row r0.
template <int FMT, int NR, int NT>
__device__ __forceinline__ void stream_tiles(const ProductArgs& p, int g, int r0, int re, int n0, f32x4_t* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, lg = lane >> 4;
    const int KB = p.K / 32;
    const uint8_t* wrow[NR];
    const uint8_t* srow[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int64_t n = (int64_t)g * p.N + min(n0 + 16 * i + col, p.N - 1);      // rows past N: any valid row
        wrow[i] = p.w + n * (p.K / 2);
        srow[i] = p.w_s + n * KB;
    }
    f32x4_t acc[NR][NT];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // units of 256 k (a full 128-byte line of a row's codes), wave-interleaved
    for (int u = wave; u * 8 < KB; u += kSWaves) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int kb = u * 8 + s * 4 + lg;                  // this lane's block
            const bool kv = kb < KB;
            u32x4_t wc[NR];
            uint32_t ws[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                wc[i] = u32x4_t{0u, 0u, 0u, 0u};
                ws[i] = 0u;
                if (kv) {
                    wc[i] = *reinterpret_cast<const u32x4_t*>(wrow[i] + (int64_t)kb * 16);
                    ws[i] = srow[i][kb];
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int r = r0 + 16 * t + col;
                u32x4_t av[kTokenLoads<FMT>];
                uint32_t as;
                load_token<FMT>(p, r, kb, lg, r < re, av, as);
                if constexpr (FMT != kRowsBf16) {
#pragma unroll
                    for (int i = 0; i < NR; ++i) acc[i][t] = mfma_mx<FMT>(wc[i], ws[i], av, as, acc[i][t]);
                } else {
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        const float sc = __uint_as_float(ws[i] << 23);
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            acc[i][t] = mfma_bf16_16(mx_decode8(wc[i][m], sc), av[m], acc[i][t]);
                    }
                }
            }
        }
    }
    // join the waves' sums in wave order
    __syncthreads();                                            // red's previous readers are done
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[((wave * NR + i) * NT + t) * 64 + lane] = acc[i][t];
    __syncthreads();
    for (int x = threadIdx.x; x < NR * NT * 64; x += 64 * kSWaves) {
        f32x4_t s = red[x];
#pragma unroll
        for (int w = 1; w < kSWaves; ++w) s += red[w * NR * NT * 64 + x];
        const int l = x & 63, t = (x >> 6) % NT, i = (x >> 6) / NT;
        const int r = r0 + 16 * t + (l & 15), n = n0 + 16 * i + 4 * (l >> 4);
        if (r < re) store4(p.out, p.out_dtype, r * p.os + n, s, p.N - n);
    }
}

template <int FMT, int NR>
__global__ __launch_bounds__(64 * kSWaves) void product_stream_kernel(ProductArgs p, int by_rank) {
    __shared__ f32x4_t red[kSWaves * NR * 4 * 64];
    const int g = by_rank ? nth_group(p, blockIdx.y) : (int)blockIdx.y;
    if (g < 0) return;
    int rb, re;
    group_rows(p, g, rb, re);
    const int n0 = blockIdx.x * 16 * NR;
    for (int r0 = rb; r0 < re;) {
        const int left = re - r0;
        if (left > 32) { stream_tiles<FMT, NR, 4>(p, g, r0, re, n0, red); r0 += 64; }
        else if (left > 16) { stream_tiles<FMT, NR, 2>(p, g, r0, re, n0, red); r0 += 32; }
        else { stream_tiles<FMT, NR, 1>(p, g, r0, re, n0, red); r0 += 16; }
    }
}

// ---------------------------------------------------------------------------
// forward, K up to 4096 (MXFP4, MXFP8 rows: 8192): eight waves split K into contiguous parts of KS steps (128 k),
// each keeps its part of the tokens in registers and walks the workgroup's weight
// tiles (16 rows) with the codes of the next two in flight, so that only weights
// stream; one barrier a tile joins the waves' sums.
// ---------------------------------------------------------------------------
constexpr int kRWaves = 8;

template <int FMT, int KS, int NT, bool S16>
__device__ __forceinline__ void resident_tiles(const ProductArgs& p, int g, int r0, int re, int t0, int t1,
                                               f32x4_t* red) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, lg = lane >> 4, KB = p.K / 32;
    const int kb0 = wave * KS * 4 + lg;                         // this lane's block of step s: kb0 + 4 s
    u32x4_t tok[KS][NT][kTokenLoads<FMT>];
    uint32_t ts[KS][NT];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + col;
            load_token<FMT>(p, r, kb0 + 4 * s, lg, r < re, tok[s][t], ts[s][t]);
        }
    struct Weight {
        u32x4_t c[KS];
        uint32_t s[KS];
    };
    const uint8_t* wbase = p.w + (int64_t)g * p.N * (p.K / 2);
    const uint8_t* sbase = p.w_s + (int64_t)g * p.N * KB;
    // blocks past K: any valid block's codes (the tokens there are 0) under scale 2^0, for
    // 0 times a NaN scale would not be 0
    auto load = [&](int t, Weight& w) {
        const int64_t n = min(t * 16 + col, p.N - 1);           // rows past N: any valid row
#pragma unroll
        for (int s = 0; s < KS; ++s)
            w.c[s] = *reinterpret_cast<const u32x4_t*>(wbase + n * (p.K / 2) + min(kb0 + 4 * s, KB - 1) * 16);
        if constexpr (S16) {                                    // KS dwords of the row: byte lg of dword s
            const uint8_t* sr = sbase + n * KB + min(wave * KS * 4, KB - KS * 4);
            if constexpr (KS >= 4) {
#pragma unroll
                for (int s = 0; s < KS; s += 4) {
                    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(sr + 4 * s);
                    w.s[s] = v.x; w.s[s + 1] = v.y; w.s[s + 2] = v.z; w.s[s + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int s = 0; s < KS; ++s) w.s[s] = *reinterpret_cast<const uint32_t*>(sr + 4 * s);
            }
        } else {
#pragma unroll
            for (int s = 0; s < KS; ++s) w.s[s] = sbase[n * KB + min(kb0 + 4 * s, KB - 1)];
        }
    };
    auto tile = [&](int t, Weight& w) {
        f32x4_t acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint32_t sb = S16 ? (w.s[s] >> (8 * lg)) & 0xFFu : w.s[s];
            if (kb0 + 4 * s >= KB) sb = 127u;
            if constexpr (FMT != kRowsBf16) {
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i] = mfma_mx<FMT>(w.c[s], sb, tok[s][i], ts[s][i], acc[i]);
            } else {
                const float sc = __uint_as_float(sb << 23);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const u32x4_t wv = mx_decode8(w.c[s][q], sc);
#pragma unroll
                    for (int i = 0; i < NT; ++i) acc[i] = mfma_bf16_16(wv, tok[s][i][q], acc[i]);
                }
            }
        }
        if (t + 2 < t1) load(t + 2, w);
        f32x4_t* buf = red + (t & 1) * kRWaves * NT * 64;
#pragma unroll
        for (int i = 0; i < NT; ++i) buf[(wave * NT + i) * 64 + lane] = acc[i];
        // (a plain barrier would wait for the loads in flight.)  Two buffers: the tile after
        // the next writes this one again only after the next tile's barrier
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (((t * NT + i) & (kRWaves - 1)) != wave) continue;
            f32x4_t sum = buf[i * 64 + lane];
#pragma unroll
            for (int v = 1; v < kRWaves; ++v) sum += buf[(v * NT + i) * 64 + lane];
            const int r = r0 + 16 * i + col, n = t * 16 + 4 * lg;
            if (r < re) store4(p.out, p.out_dtype, r * p.os + n, sum, p.N - n);
        }
    };
    Weight w0, w1;
    load(t0, w0);
    if (t0 + 1 < t1) load(t0 + 1, w1);
    for (int t = t0; t < t1; t += 2) {
        tile(t, w0);
        if (t + 1 < t1) tile(t + 1, w1);
    }
    // both buffers are free before the next rows' tiles write them
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int FMT, int KS, int MAXT, bool S16>
__global__ __launch_bounds__(64 * kRWaves) void product_resident_kernel(ProductArgs p, int by_rank, int per_block) {
    __shared__ f32x4_t red[2 * kRWaves * MAXT * 64];
    const int g = by_rank ? nth_group(p, blockIdx.y) : (int)blockIdx.y;
    if (g < 0) return;
    int rb, re;
    group_rows(p, g, rb, re);
    const int t0 = blockIdx.x * per_block, t1 = min(t0 + per_block, (p.N + 15) / 16);
    for (int r0 = rb; r0 < re;) {
        if (MAXT > 1 && re - r0 > 16) {
            resident_tiles<FMT, KS, MAXT, S16>(p, g, r0, re, t0, t1, red);
            r0 += 16 * MAXT;
        } else {
            resident_tiles<FMT, KS, 1, S16>(p, g, r0, re, t0, t1, red);
            r0 += 16;
        }
    }
}

template <int FMT, int KS, int MAXT>
static void launch_resident(const ProductArgs& p, int cus, int groups, int by_rank, hipStream_t s) {
    // tiles a workgroup: as many as leave one workgroup a CU, 16 at most. Experts of 2048 x
    // 4096: 8 rows over 320 take 11.4 us, with two workgroups a CU 14.0; 512 rows over 160
    // take 131 us, with at most 8 or 32 tiles 141 and 140.
    const int tiles = (p.N + 15) / 16;
    const int per = max(1, min(16, (int)((int64_t)tiles * groups / cus)));
    const dim3 grid((tiles + per - 1) / per, groups);
    // a wave's part of a scale row is one aligned load (per 16 bytes)
    constexpr int part = KS >= 4 ? 16 : 4 * KS;
    const bool s16 = p.K % (128 * KS) == 0 && (p.K / 32) % part == 0 &&
                     (reinterpret_cast<uintptr_t>(p.w_s) & (part - 1)) == 0;
    if (s16)
        hipLaunchKernelGGL((product_resident_kernel<FMT, KS, MAXT, true>), grid, dim3(64 * kRWaves), 0, s, p, by_rank,
                           per);
    else
        hipLaunchKernelGGL((product_resident_kernel<FMT, KS, MAXT, false>), grid, dim3(64 * kRWaves), 0, s, p, by_rank,
                           per);
}

template <int FMT>
static hipError_t launch_stream(const ProductArgs& p, int cus, hipStream_t s) {
    const int groups = min(p.G, p.M);                           // at most so many hold rows
    const int by_rank = p.M < p.G ? 1 : 0;
    // (a variant for 16 tokens alone, with fewer registers, was no faster at any row count)
    if (p.K <= 1024) launch_resident<FMT, 1, 2>(p, cus, groups, by_rank, s);
    else if (p.K <= 2048) launch_resident<FMT, 2, 2>(p, cus, groups, by_rank, s);
    else if (p.K <= 4096) launch_resident<FMT, 4, 2>(p, cus, groups, by_rank, s);
    else if (FMT != kRowsBf16 && p.K <= 8192) launch_resident<FMT == kRowsBf16 ? kRowsMx4 : FMT, 8, 1>(p, cus, groups, by_rank, s);
    else
        hipLaunchKernelGGL((product_stream_kernel<FMT, 1>), dim3((p.N + 15) / 16, groups), dim3(64 * kSWaves), 0, s, p,
                           by_rank);
    return hipGetLastError();
}

hipError_t launch_product_stream(const ProductArgs& p, int cus, hipStream_t s) {
    if (p.a8) return launch_stream<kRowsMx8>(p, cus, s);
    return p.a_s ? launch_stream<kRowsMx4>(p, cus, s) : launch_stream<kRowsBf16>(p, cus, s);
}

// ---------------------------------------------------------------------------
// backward.  The reduction runs over the weight's rows, so an operand needs eight
// rows' codes of one column.  A lane takes eight neighbouring columns (one dword of
// codes) of eight rows, decodes pairs along a row with that row's block scale and
// regroups them by column (v_perm); operand c of the eight then holds columns
// 8 i + c for operand row i, and a lane ends with eight consecutive outputs.
// ---------------------------------------------------------------------------
constexpr int kGWaves = 8;

template <int NT>
__device__ __forceinline__ void grad_tiles(const ProductArgs& p, int g, int r0, int re, int k0, float* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, lg = lane >> 4;
    const int KB = p.K / 32, kc = k0 + 8 * col;                 // this lane's columns kc .. kc + 7
    const bool kv = kc < p.K;                                   // K is a multiple of 32: all eight or none
    const uint8_t* wbase = p.w + (int64_t)g * p.N * (p.K / 2) + (kv ? kc / 2 : 0);
    const uint8_t* sbase = p.w_s + (int64_t)g * p.N * KB + (kv ? kc / 32 : 0);
    const uint16_t* dout = static_cast<const uint16_t*>(p.a);
    f32x4_t acc[8][NT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[c][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // a step: 32 weight rows, eight a lane group; loaded one step ahead
    struct Step {
        uint32_t code[8], sb[8];
        u32x4_t dv[NT];
    };
    auto load = [&](int ns, Step& st) {
        const int n = ns + 8 * lg;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // rows past N: the last one, against zeros of dout; its scale is masked below
            const int64_t row = min(n + j, p.N - 1);
            st.code[j] = *reinterpret_cast<const uint32_t*>(wbase + row * (p.K / 2));
            st.sb[j] = sbase[row * KB];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + col;
            st.dv[t] = r < re ? load8_bf16(dout + r * p.as + n, p.N - n) : u32x4_t{0u, 0u, 0u, 0u};
        }
    };
    auto multiply = [&](int ns, Step& st) {
        if (ns + 32 > p.N) {                                    // (0 times a NaN scale would not be 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (ns + 8 * lg + j >= p.N) st.sb[j] = 127u;
        }
        u32x4_t op[8];
        mx_decode_columns(st.code, st.sb, op);
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[c][t] = mfma_bf16_16(op[c], st.dv[t], acc[c][t]);
    };
    constexpr int STRIDE = 32 * kGWaves;
    Step s0, s1;
    int ns = wave * 32;
    if (ns < p.N) load(ns, s0);
    for (; ns < p.N; ns += 2 * STRIDE) {
        if (ns + STRIDE < p.N) load(ns + STRIDE, s1);
        multiply(ns, s0);
        if (ns + STRIDE >= p.N) break;
        if (ns + 2 * STRIDE < p.N) load(ns + 2 * STRIDE, s0);
        multiply(ns + STRIDE, s1);
    }
    // join the waves' sums, 16 tokens at a time: red [wave][v][c][lane]
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        __syncthreads();                                        // red's previous readers are done
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[((wave * 4 + v) * 8 + c) * 64 + lane] = acc[c][t][v];
        __syncthreads();
        // thread: lane l, value v, half q of its eight columns
        const int l = threadIdx.x & 63, v = (threadIdx.x >> 6) & 3, q = threadIdx.x >> 8;
        f32x4_t f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            f[c] = red[(v * 8 + 4 * q + c) * 64 + l];
#pragma unroll
            for (int w = 1; w < kGWaves; ++w) f[c] += red[((w * 4 + v) * 8 + 4 * q + c) * 64 + l];
        }
        const int r = r0 + 16 * t + (l & 15), k = k0 + 8 * (4 * (l >> 4) + v) + 4 * q;
        if (r < re && k < p.K) store4(p.out, p.out_dtype, r * p.os + k, f, 4);
    }
}

// Two neighbouring column blocks share the weight's 128-byte lines: they run on one XCD
// (workgroup b runs on XCD b % 8), one after the other, so that its L2 fetches a line once.
// Whole groups go around the XCDs, or, with fewer than eight, ranges of columns.
__global__ __launch_bounds__(64 * kGWaves) void product_grad_stream_kernel(ProductArgs p, int by_rank) {
    __shared__ float red[kGWaves * 32 * 64];
    const int nx = gridDim.x, lin = blockIdx.y * nx + blockIdx.x;
    int x = blockIdx.x, y = blockIdx.y;
    if ((gridDim.y & 7) == 0) {
        x = (lin >> 3) % nx;
        y = (lin >> 3) / nx * 8 + (lin & 7);
    } else if ((nx & 7) == 0) {
        x = (x & 7) * (nx >> 3) + (x >> 3);
    }
    const int g = by_rank ? nth_group(p, y) : y;
    if (g < 0 || g >= p.G) return;
    int rb, re;
    group_rows(p, g, rb, re);
    const int k0 = x * 128;
    for (int r0 = rb; r0 < re;) {
        if (re - r0 > 16) { grad_tiles<2>(p, g, r0, re, k0, red); r0 += 32; }
        else { grad_tiles<1>(p, g, r0, re, k0, red); r0 += 16; }
    }
}

hipError_t launch_product_grad_stream(const ProductArgs& p, hipStream_t s) {
    const int groups = min(p.G, p.M);
    const dim3 grid((p.K + 127) / 128, groups < 8 ? groups : (groups + 7) & ~7);
    const int by_rank = p.M < p.G ? 1 : 0;
    hipLaunchKernelGGL(product_grad_stream_kernel, grid, dim3(64 * kGWaves), 0, s, p, by_rank);
    return hipGetLastError();
}

// The tiles address 256 rows by 32-bit offsets.
static bool tiles_reach(const ProductArgs& p) { return p.as <= (1 << 22); }

// Rows a group (M / G, an upper bound of their mean) up to which the weight is streamed
// past the tokens instead of multiplied in 256 x 256 tiles.  Measured on 64 groups of
// 2048 x 4096, us streamed against tiled: W4A16 77 / 110 at 16 rows, 124 / 119 at 32;
// W4A4 59 / 72 and 96 / 75.  Tiles that leave most of the card idle lose for longer (one
// group of 4096 x 4096: W4A16 38 / 54 at 128 rows, 74 / 85 at 256; W4A4 24 / 27 at 128;
// eight groups of 2048 x 4096 cross at about 32 again): the bound grows with the CUs that
// the tiles of one row block leave four times over, up to `most` times.  There the card is
// idle either way and the streaming kernels' passes over 32 rows, one after another, cost
// as much as a tile (one group, K = 4096, 16, 256 and 512 outputs alike): W4A16 73 / 84 at
// 256 rows, 150 / 83 at 512, 450 / 84 at 1536; W4A4 23 / 27 at 128, 45 / 33 at 256, 172 / 33
// at 1024 (K = 1024: W4A16 24 / 28 at 256, 47 / 28 at 512; W4A4 18 / 13 at 256).
// M is the buffer's: where few of its rows are kept or one group holds many of them the rule
// can pick the slower kernel (W4A16, 160 experts of 2048 x 4096: 3500 rows 198 / 236 spread
// evenly, 572 / 324 after a Zipf law; 40 of 320 experts, an eighth of 2048 rows kept, 47 / 71).
//
// MXFP8 rows, streamed / tiled us; `one`: the tiles of one row block of every group.
// Scales in dwords, K up to 4096 (short tiles).  Two cards of tiles or more: 320 groups of 2048 x 4096
// 274 / 263 at 8 rows a group, 333 / 284 at 24; of 4096 x 1024 174 / 156 at 8; 64 groups of 2048 x 4096
// 48 / 50 at 8, 53 / 52 at 14, 73 / 57 at 24.  A third of a card to two: 16 groups 17.8 / 20.2 at 19, 28.8 /
// 24.3 at 20; 32 groups 23 / 23 at 4, 28 / 24 at 20, 47 / 28 at 28; 20 groups of 4096 x 2048 22 / 23 at 8,
// 26 / 23 at 20; where the streams' workgroups fill the card unevenly tiles win at every count: 24 groups
// 30 / 21 at 4, 36 / 21 at 20, 48 groups 43 / 40 and 50 / 41, 12 of 4096 x 1024 14 / 8 and 15 / 9.  A quarter
// (8 groups) 24 / 24 at 48, 31 / 25 at 56; a sixteenth (one group of 4096 x 4096) 24 / 24 at 96, 31 / 24 at 128.
// Scales that are no whole dwords, K up to 4096 (tall tiles, of which one alone takes longer: 43 us at
// K = 4064): 160 groups of 2048 x 4064 233 / 267 at 32, 283 / 274 at 40; 64 groups 103 / 111 at 40, 122 / 113
// at 48; half a card (16 groups) 30 / 45 at 40, 44 / 46 at 64; a quarter (8 groups) 37 / 47 at 110, 45 / 52 at
// 128; a sixteenth (one group of 4096 x 4064) 36 / 54 at 200, 41 / 53 at 256.
// The bounds are those of K up to 4096.  Beyond, the resident tokens are 16 at a time (beyond 8192 none)
// and the bounds are too high, by up to four times: 160 groups of 2048 x 4128 242 / 258 at 8, 267 / 259 at 12,
// 503 / 280 at 32; 16 groups 22 / 43 at 8, 59 / 47 at 20; 8 groups 46 / 47 at 48, 90 / 50 at 96; one of 4096 x
// 4128 47 / 51 at 160, 57 / 55 at 192; in dwords 64 groups of 2048 x 8192 112 / 133 at 8, 16 groups 26 / 36 at
// 8, 47 / 36 at 12; of 2048 x 8320 201 / 125 and 40 / 39 at 8, one of 4096 x 8320 28 / 44 at 64, 45 / 47 at 96.
static bool streamed(const ProductArgs& p, int cus) {
    if (p.a8) {
        const int64_t one = (int64_t)p.G * ((p.N + 255) / 256);
        if (product8_dwords(p))
            return p.M <= (int64_t)p.G * (one >= 2 * cus ? 8 : (one * 3 >= cus ? 20 : (one * 8 >= cus ? 48 : 96)));
        return p.M <= (int64_t)p.G * (one * 12 <= cus ? 200 : (one * 4 <= cus ? 110 : 40));
    }
    const int rows = p.a_s ? 20 : 24;
    const int64_t most = p.a_s ? 8 : 12, tiles = (int64_t)p.G * ((p.N + 255) / 256);
    const int64_t idle = min(most, cus / (4 * tiles));
    return p.M <= p.G * rows * (idle > 1 ? idle : 1) || !tiles_reach(p);
}
// The gradient's crossings, us streamed against tiled: 64 groups of 2048 x 4096 154 / 171
// at 32 rows a group, 197 / 175 at 47 (16 groups: 47 / 50 at 40, 64 / 52 at 64); with the
// tiles of one row block on half the card (eight groups) 43 / 49 at 90, on a quarter
// or less 39 / 47 at 100 and 58 / 54 at 150 (four groups), 65 / 86 at 128 (one of 4096 x
// 4096).
static bool grad_streamed(const ProductArgs& p, int cus) {
    const int64_t tiles = (int64_t)p.G * ((p.K + 255) / 256), idle = min((int64_t)4, cus / tiles);
    return p.M <= p.G * 36 * (idle > 1 ? idle : 1) || !tiles_reach(p);
}

hipError_t launch_product(const ProductArgs& p, int cus, hipStream_t s) {
    if (streamed(p, cus)) return launch_product_stream(p, cus, s);
    return p.a8 ? launch_product8_tiles(p, cus, s) : launch_product_tiles(p, cus, s);
}
hipError_t launch_product_grad(const ProductArgs& p, int cus, hipStream_t s) {
    return grad_streamed(p, cus) ? launch_product_grad_stream(p, s) : launch_product_grad_tiles(p, cus, s);
}

}  // namespace moe

int moe_internal_product_streams(int M, int N, int K, int G, int64_t stride, int mx, int backward, int cus) {
    moe::ProductArgs p{};
    alignas(16) const uint8_t scales = 0;
    p.M = M; p.N = N; p.K = K; p.G = G; p.as = stride;
    p.a_s = mx ? &scales : nullptr;
    p.a8 = mx == 2;
    return backward ? moe::grad_streamed(p, cus) : moe::streamed(p, cus);
}
