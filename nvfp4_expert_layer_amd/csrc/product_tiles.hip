// MXFP4 products in tiles, for many rows a group (gfx950).  A tile is 256 rows of
// one group x 256 outputs; eight waves; the operands come through LDS rings filled
// straight from global memory (global_load_lds), two or three stages ahead; one
// workgroup a CU.  The weight is the matrix cores' row operand and tokens are their
// columns, so that a lane ends with groups of four consecutive outputs of one token
// (packed stores into the output's staging).
//
//   mx_tile_kernel     W4A4: 32x32x64 scaled MFMAs on the codes as they lie in
//                      memory; 128 k a stage, four stages.
//   a16_tile_kernel    W4A16: bf16 rows, 64 k a stage, three stages; each wave
//                      decodes its weight operand in registers (one conversion a
//                      pair, the block scale within it), then 32x32x16 bf16 MFMAs.
//   grad_tile_kernel   backward: the reduction runs over the weight's rows, 64 a
//                      stage; a lane takes four neighbouring columns of eight rows,
//                      decodes them and regroups the pairs by column.
//
// Lane layout of the 32x32 MFMAs: lane l holds row (column) l % 32 and the K slice of
// lane half l / 32; accumulator value v sits at row 8 (v/4) + 4 (l/32) + v % 4, column
// l % 32.  K runs in any order as long as both operands use the same one.
//
// Past a row's end (K, N not multiples of a stage) lanes load from a block of zeros.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "ops.h"
#include "product_common.h"

namespace moe {

constexpr int kTM = 256, kTN = 256, kTWaves = 8, kTThreads = 64 * kTWaves;

typedef __attribute__((address_space(3))) void lds_void_t;

static __device__ __align__(16) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ void to_lds16(const void* src, void* dst) {
    __builtin_amdgcn_global_load_lds(src, (lds_void_t*)dst, 16, 0, 0);
}
__device__ __forceinline__ void to_lds4(const void* src, void* dst) {
    __builtin_amdgcn_global_load_lds(src, (lds_void_t*)dst, 4, 0, 0);
}
// one byte a lane, each to a dword of its own
__device__ __forceinline__ void to_lds1(const void* src, void* dst) {
    __builtin_amdgcn_global_load_lds(src, (lds_void_t*)dst, 1, 0, 0);
}
// A wave-uniform pointer, in scalar registers and opaque: loads then take it with a
// 32-bit lane offset (else each load keeps and advances a 64-bit pointer a lane).
template <typename T>
__device__ __forceinline__ T* scalar(T* p) {
    asm("" : "+s"(p));
    return p;
}
// Operand reads stay before the MFMAs that follow them in the source (the scheduler
// would sink each read to its use and wait for it there).
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}

// p, or the zeros where `in` is false, without a branch (the compiler waits for every
// outstanding load around one).
__device__ __forceinline__ const void* within(bool in, const void* p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), z = reinterpret_cast<uintptr_t>(kZeros);
    return reinterpret_cast<const void*>(z ^ ((a ^ z) & (uintptr_t)-(intptr_t)in));
}

// Byte offset of 16-byte unit u of row r in a tile of 128-byte rows: eight
// consecutive rows put a unit in eight different slots, rows r and r + 8 differ too.
__device__ __forceinline__ int swz8(int r, int u) { return r * 128 + ((u ^ (r & 7) ^ ((r >> 3) & 1)) << 4); }
// The same for 64-byte rows of four units.
__device__ __forceinline__ int swz4(int r, int u) { return r * 64 + ((u ^ (((r >> 1) ^ (r >> 3)) & 3)) << 4); }

struct Tile {
    int g, rb, re, nt;            // group, its rows [rb, re) of this tile, column block
};

// Tile of this workgroup, or g = -1.  Tiles are numbered group by group, the NT
// column blocks of 256 rows together; the eight XCDs (workgroup b runs on XCD b % 8)
// take contiguous ranges, so that the rows of a tile and the weight of a group are
// shared within an XCD's L2.  s: 1024 + 16 words of LDS.
__device__ __forceinline__ Tile find_tile(const ProductArgs& p, int NT, int* s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int n[2], first[2], rows[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int g = 2 * tid + i;
        int rb = 0, re = 0;
        if (g < p.G) group_rows(p, g, rb, re);
        first[i] = rb;
        rows[i] = re;
        n[i] = (re - rb + kTM - 1) / kTM;
    }
    const int sum = n[0] + n[1];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(inc, o, 64);
        if (lane >= o) inc += y;
    }
    if (lane == 63) s[wave] = inc;
    __syncthreads();
    int at = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kTWaves; ++w) {
        if (w < wave) at += s[w];
        total += s[w];
    }
    const int64_t all = (int64_t)total * NT, per = (all + 7) >> 3;
    const int64_t b = blockIdx.x, logical = (b & 7) * per + (b >> 3);
    const bool live = (b >> 3) < per && logical < all;
    const int tile = live ? (int)(logical / NT) : -1;
    if (live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (tile >= at && tile < at + n[i]) {
                s[8] = 2 * tid + i;
                s[9] = first[i] + (tile - at) * kTM;
                s[10] = min(s[9] + kTM, rows[i]);
            }
            at += n[i];
        }
    }
    __syncthreads();
    Tile t{-1, 0, 0, 0};
    // scalar registers: the addresses below are a scalar base and a 32-bit lane offset
    if (live)
        t = Tile{__builtin_amdgcn_readfirstlane(s[8]), __builtin_amdgcn_readfirstlane(s[9]),
                 __builtin_amdgcn_readfirstlane(s[10]), (int)(logical - (int64_t)tile * NT)};
    __syncthreads();                                     // s is free again
    return t;
}

static int64_t tile_grid(const ProductArgs& p, int NT) {
    // groups' partial tiles: at most one each
    const int64_t tiles = p.M / kTM + min(p.G, p.M);
    return (tiles * NT + 7) / 8 * 8;
}

// ---------------------------------------------------------------------------
// Output staging: bf16 / f16 [256 tokens][264] in LDS (the row pitch spreads 32 rows'
// 8-byte pieces over all banks), then 16-byte row pieces to memory; fp32 goes straight
// from the accumulators, 16 bytes a lane.
// ---------------------------------------------------------------------------
constexpr int kYS = 264;

__device__ __forceinline__ void stage4(const ProductArgs& p, uint8_t* smem, const Tile& t, int row, int col, int width,
                                       float a, float b, float c, float d) {
    if (p.out_dtype == kF32) {
        if (t.rb + row < t.re)
            store4(p.out, kF32, (t.rb + row) * p.os + t.nt * kTN + col, f32x4_t{a, b, c, d},
                   width - t.nt * kTN - col, p.out_vec);
        return;
    }
    u32x2_t v;
    if (p.out_dtype == kBF16) v = u32x2_t{f32x2_to_bf16x2(a, b), f32x2_to_bf16x2(c, d)};
    else v = u32x2_t{f32_to_f16_bits(a) | (f32_to_f16_bits(b) << 16), f32_to_f16_bits(c) | (f32_to_f16_bits(d) << 16)};
    *reinterpret_cast<u32x2_t*>(smem + (row * kYS + col) * 2) = v;
}

__device__ __forceinline__ void store_staged(const ProductArgs& p, const uint8_t* smem, const Tile& t, int width) {
    if (p.out_dtype == kF32) return;
    __syncthreads();
    const int nrow = t.re - t.rb, ncol = min(kTN, width - t.nt * kTN);
    uint16_t* out = static_cast<uint16_t*>(p.out) + t.rb * p.os + t.nt * kTN;
    const bool vec = p.os % 8 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
    for (int x = threadIdx.x; x < kTM * (kTN / 8); x += kTThreads) {
        const int row = x >> 5, c = (x & 31) * 8;
        if (row >= nrow) break;                          // rows grow with x
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + (row * kYS + c) * 2);
        if (vec && c + 8 <= ncol) {
            *reinterpret_cast<u32x4_t*>(out + row * p.os + c) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < ncol) out[row * p.os + c + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        }
    }
}

// ---------------------------------------------------------------------------
// W4A4
// ---------------------------------------------------------------------------
constexpr int kMxStages = 4;
constexpr int kMxCodes = 256 * 64;                          // an operand's 128 k of a stage
// its scales: a row's four bytes in one dword, or (rows not aligned to dwords) each in
// one of its own, [4 blocks][256 rows]
constexpr int mx_scales(bool aligned) { return aligned ? 256 * 4 : 256 * 16; }
constexpr int mx_slot(bool aligned) { return 2 * kMxCodes + 2 * mx_scales(aligned); }   // codes: weight | rows; scales
constexpr int mx_lds(bool aligned) { return kMxStages * mx_slot(aligned); }             // 136 or 160 KB

template <int OPSEL>
__device__ __forceinline__ f32x16_t mfma_mx32(const u32x4_t& a, uint32_t as, const u32x4_t& b, uint32_t bs,
                                              const f32x16_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, OPSEL, (int)as,
                                                           OPSEL, (int)bs);
}

// ALIGNED: scale rows can be read in dwords (K % 128 == 0, 4-byte aligned scales).
template <bool ALIGNED>
__global__ __launch_bounds__(kTThreads) void mx_tile_kernel(ProductArgs p) {
    constexpr int kMxScales = mx_scales(ALIGNED), kMxSlot = mx_slot(ALIGNED);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const Tile t = find_tile(p, (p.N + kTN - 1) / kTN, reinterpret_cast<int*>(smem));
    if (t.g < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int wm = wave >> 2, wn = wave & 3;             // rows 128 wm .. +128, outputs 64 wn .. +64
    const int KB = p.K / 32, nc = (KB + 3) / 4, n0 = t.nt * kTN;
    const int64_t w0 = (int64_t)t.g * p.N + n0;
    const uint8_t* wbase = p.w + w0 * (p.K / 2);
    const uint8_t* abase = static_cast<const uint8_t*>(p.a) + (int64_t)t.rb * (p.K / 2);
    // rows and outputs past the tile's end: any valid row (their results are not stored)
    auto arow = [&](int r) { return (uint32_t)min(r, t.re - 1 - t.rb); };
    auto wrow = [&](int r) { return (uint32_t)min(r, p.N - 1 - n0); };

    // loads of a stage: per operand 16 KB of codes, two of 1 KB a wave: load q of wave w
    // fills rows 16 (2 w + q) .. +16, lane i row i / 4, slot i % 4, which holds unit
    // (i % 4) ^ f(row) of the stage (swz4); scales: 256 bytes a wave, waves 0-3 the
    // weight's rows 64 w .. +64, waves 4-7 the rows'
    uint32_t coff[2], aoff[2];
    int cu[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = (wave * 2 + q) * 16 + (lane >> 2);
        cu[q] = (lane & 3) ^ (((r >> 1) ^ (r >> 3)) & 3);
        coff[q] = wrow(r) * (uint32_t)(p.K / 2) + cu[q] * 16;
        aoff[q] = arow(r) * (uint32_t)(p.K / 2) + cu[q] * 16;
    }
    const int srow = (wave & 3) * 64 + lane;
    const uint8_t* sbase = wave < 4 ? p.w_s + w0 * KB : p.a_s + (int64_t)t.rb * KB;
    const uint32_t soff = (wave < 4 ? wrow(srow) : arow(srow)) * (uint32_t)KB;
    const int sdst = 2 * kMxCodes + (wave < 4 ? 0 : kMxScales) + (wave & 3) * 256;

    // part 0, 1: the wave's weight codes; 2, 3: the rows' codes; 4: the scales
    auto issue = [&](int c, int slot, int part) {
        uint8_t* base = smem + slot * kMxSlot;
        if (part < 4) {
            const int q = part & 1;
            const uint8_t* src = scalar((part < 2 ? wbase : abase) + (int64_t)c * 64) + (part < 2 ? coff[q] : aoff[q]);
            if (!ALIGNED) src = static_cast<const uint8_t*>(within(c * 4 + cu[q] < KB, src));
            to_lds16(src, base + (part < 2 ? 0 : kMxCodes) + (wave * 2 + q) * 1024);
        } else if (ALIGNED) {
            to_lds4(scalar(sbase + (int64_t)c * 4) + soff, base + sdst);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to_lds1(within(c * 4 + i < KB, scalar(sbase + (int64_t)c * 4 + i) + soff), base + sdst + i * 1024);
        }
    };

    f32x16_t acc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
    const int nvi = max(0, min(4, (t.re - t.rb - wm * 128 + 31) >> 5));      // 32-row blocks with rows
    const bool cols = n0 + wn * 64 < p.N;
    const int r32 = lane & 31;

    // Stage c sits in slot c % 4.  Lane half h of its MFMA m (0, 1) takes block 2 h + m of
    // the stage's four.  A step's second operands are read before its first MFMAs, the
    // next stage's first ones before its second MFMAs, so that the matrix cores do not
    // wait for LDS; the barrier stands between the two, where the step's slot has been
    // read and stage c + 4 may take it.  Past the end valid stages are loaded again, so
    // that each step issues as many loads and the wait leaves the two newer stages in flight.
    auto kloop = [&](auto nv_c) {
        constexpr int NV = decltype(nv_c)::value;
        u32x4_t wv[2][2], av[2][4];
        uint32_t ws[2][2], as[2][4];                      // scales by parity of the stage
        auto operands = [&](int c, auto m_c) {
            constexpr int m = decltype(m_c)::value;
            const uint8_t* S = smem + (c & 3) * kMxSlot;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                wv[m][j] = *reinterpret_cast<const u32x4_t*>(S + swz4(wn * 64 + j * 32 + r32, 2 * h + m));
#pragma unroll
            for (int i = 0; i < NV; ++i)
                av[m][i] = *reinterpret_cast<const u32x4_t*>(S + kMxCodes + swz4(wm * 128 + i * 32 + r32, 2 * h + m));
        };
        auto scale_pair = [&](const uint8_t* S, int r) {       // blocks 2 h and 2 h + 1 of row r
            if (ALIGNED) return (uint32_t)*reinterpret_cast<const uint16_t*>(S + r * 4 + 2 * h);
            return *reinterpret_cast<const uint32_t*>(S + 2048 * h + r * 4) |
                   (*reinterpret_cast<const uint32_t*>(S + 2048 * h + 1024 + r * 4) << 8);
        };
        auto scales = [&](int c, auto f_c) {
            constexpr int f = decltype(f_c)::value;
            const uint8_t* S = smem + (c & 3) * kMxSlot + 2 * kMxCodes;
#pragma unroll
            for (int j = 0; j < 2; ++j) ws[f][j] = scale_pair(S, wn * 64 + j * 32 + r32);
#pragma unroll
            for (int i = 0; i < NV; ++i) as[f][i] = scale_pair(S + kMxScales, wm * 128 + i * 32 + r32);
        };
        const std::integral_constant<int, 0> c0;
        const std::integral_constant<int, 1> c1;
        auto stage = [&](int c, auto f_c, auto g_c) {
            constexpr int f = decltype(f_c)::value;
            if constexpr (NV > 0) {
                operands(c, c1);
                keep_order();
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[j][i] = mfma_mx32<0>(wv[0][j], ws[f][j], av[0][i], as[f][i], acc[j][i]);
            }
            keep_order();
            if (ALIGNED) asm volatile("s_waitcnt vmcnt(10) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const int ahead = min(c + 4, nc - 1);
            if constexpr (NV > 0) {
                operands(c + 1, c0);
                scales(c + 1, g_c);
                keep_order();
            }
            // the loads one by one between the MFMAs: in a row they would hold up the wave
            // (and with it the matrix core) until the address unit has taken them all
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (NV > 0) {
                    if (i < NV) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[j][i] = mfma_mx32<1>(wv[1][j], ws[f][j], av[1][i], as[f][i], acc[j][i]);
                        keep_order();
                    }
                }
                issue(ahead, c & 3, i);
                keep_order();
            }
            issue(ahead, c & 3, 4);
        };
        if constexpr (NV > 0) {
            operands(0, c0);
            scales(0, c0);
        }
        int c = 0;
        for (; c + 1 < nc; c += 2) {
            stage(c, c0, c1);
            stage(c + 1, c1, c0);
        }
        if (c < nc) stage(c, c0, c1);
    };
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int part = 0; part < 5; ++part) issue(min(c, nc - 1), c, part);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    switch (cols ? nvi : 0) {
        case 4: kloop(std::integral_constant<int, 4>{}); break;
        case 3: kloop(std::integral_constant<int, 3>{}); break;
        case 2: kloop(std::integral_constant<int, 2>{}); break;
        case 1: kloop(std::integral_constant<int, 1>{}); break;
        default: kloop(std::integral_constant<int, 0>{}); break;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // all loads landed, all reads done
    if (cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= nvi) break;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; v += 4)
                    stage4(p, smem, t, wm * 128 + i * 32 + r32, wn * 64 + j * 32 + 2 * v + 4 * h, p.N, acc[j][i][v],
                           acc[j][i][v + 1], acc[j][i][v + 2], acc[j][i][v + 3]);
        }
    }
    store_staged(p, smem, t, p.N);
}

// ---------------------------------------------------------------------------
// W4A16
// ---------------------------------------------------------------------------
constexpr int kARows = 256 * 128;                        // 64 k of the tile's bf16 rows (32 KB)
constexpr int a16_chunk(bool aligned) { return kMxCodes + mx_scales(aligned); }   // 128 k of the weight
constexpr int kAOffW = 3 * kARows;                       // LDS: rows [3] | weight [3]
constexpr int a16_lds(bool aligned) { return kAOffW + 3 * a16_chunk(aligned); }   // 147 or 156 KB

__device__ __forceinline__ f32x16_t mfma_bf16_32(const u32x4_t& a, const u32x4_t& b, const f32x16_t& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}

template <bool ALIGNED>
__global__ __launch_bounds__(kTThreads) void a16_tile_kernel(ProductArgs p) {
    constexpr int kAChunk = a16_chunk(ALIGNED);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const Tile t = find_tile(p, (p.N + kTN - 1) / kTN, reinterpret_cast<int*>(smem));
    if (t.g < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int wm = wave >> 2, wn = wave & 3;
    // steps of 64 k, two to a weight chunk: an even number of them (the last may be
    // all zeros)
    const int KB = p.K / 32, nc = (KB + 3) / 4, nk = 2 * nc, n0 = t.nt * kTN;
    const int64_t w0 = (int64_t)t.g * p.N + n0;
    const uint8_t* wbase = p.w + w0 * (p.K / 2);
    const uint8_t* sbase = p.w_s + w0 * KB;
    const uint16_t* abase = static_cast<const uint16_t*>(p.a) + (int64_t)t.rb * p.as;
    auto wrow = [&](int r) { return (uint32_t)min(r, p.N - 1 - n0); };

    // rows: four loads of 1 KB (8 rows of 128 bytes) a wave and step; weight codes: two
    // of 1 KB (16 rows of 64 bytes) a wave and chunk; scales: 64 rows' dwords, each
    // quarter by two waves (the same bytes), or two of a row's four bytes a wave
    uint32_t aoff[4];
    int au[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = (wave * 4 + q) * 8 + (lane >> 3);
        au[q] = (lane & 7) ^ (lane >> 3) ^ (q & 1);
        aoff[q] = (uint32_t)(min(r, t.re - 1 - t.rb) * p.as + au[q] * 8);
    }
    uint32_t coff[2];
    int cu[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = (wave * 2 + q) * 16 + (lane >> 2);
        cu[q] = (lane & 3) ^ (((r >> 1) ^ (r >> 3)) & 3);
        coff[q] = wrow(r) * (uint32_t)(p.K / 2) + cu[q] * 16;
    }
    const uint32_t soff = wrow((wave & 3) * 64 + lane) * (uint32_t)KB;

    auto issue_rows = [&](int ks, int slot, int q) {
        const uint16_t* src = scalar(abase + (int64_t)ks * 64) + aoff[q];
        to_lds16(ALIGNED ? src : within(ks * 8 + au[q] < KB * 4, src), smem + slot * kARows + (wave * 4 + q) * 1024);
    };
    // part 0, 1: the wave's codes; 2 (and 3 when not ALIGNED): its scales
    constexpr int kParts = ALIGNED ? 3 : 4;
    auto issue_weight = [&](int c, int slot, int part) {
        uint8_t* base = smem + kAOffW + slot * kAChunk;
        if (part < 2) {
            const uint8_t* src = scalar(wbase + (int64_t)c * 64) + coff[part];
            to_lds16(ALIGNED ? src : within(c * 4 + cu[part] < KB, src), base + (wave * 2 + part) * 1024);
        } else if (ALIGNED) {
            to_lds4(scalar(sbase + (int64_t)c * 4) + soff, base + kMxCodes + (wave & 3) * 256);
        } else {
            const int b = (wave >> 2) * 2 + part - 2;
            to_lds1(within(c * 4 + b < KB, scalar(sbase + (int64_t)c * 4 + b) + soff),
                    base + kMxCodes + b * 1024 + (wave & 3) * 256);
        }
    };

    f32x16_t acc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
    const int nvi = max(0, min(4, (t.re - t.rb - wm * 128 + 31) >> 5));
    const bool cols = n0 + wn * 64 < p.N;
    const int r32 = lane & 31;

    // Step ks: rows in slot ks % 3, chunk ks / 2 in weight slot (ks / 2) % 3.  Lane half h
    // of MFMA kk (0 .. 3) takes k = 32 h + 8 kk .. + 8 of the step: dword kk of the weight
    // row's unit 2 (ks % 2) + h, and the row's unit 4 h + kk.  Operands are read one MFMA
    // ahead, a step's first ones before the last MFMAs of the step before.  The barrier
    // stands there: the step's rows have been read (slot free for step ks + 3), after an
    // odd step its chunk too (for chunk + 3), and the wait leaves in flight only what was
    // issued since the next step's rows (past the end valid data again).
    auto kloop = [&](auto nv_c) {
        constexpr int NV = decltype(nv_c)::value;
        u32x4_t wc[2][2], av[2][4];                       // codes by parity of the step; rows by parity of kk
        float sc[2][2];
        int as = 0, ws = 0;
        auto rows = [&](int slot, int kk, auto f_c) {
            constexpr int f = decltype(f_c)::value;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                av[f][i] = *reinterpret_cast<const u32x4_t*>(smem + slot * kARows +
                                                             swz8(wm * 128 + i * 32 + r32, 4 * h + kk));
        };
        auto codes = [&](int slot, auto st_c) {
            constexpr int ST = decltype(st_c)::value;
            const uint8_t* W = smem + kAOffW + slot * kAChunk;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = wn * 64 + j * 32 + r32, b = 2 * ST + h;
                wc[ST][j] = *reinterpret_cast<const u32x4_t*>(W + swz4(r, b));
                const uint32_t sb = W[kMxCodes + (ALIGNED ? r * 4 + b : b * 1024 + r * 4)];
                sc[ST][j] = __uint_as_float(sb << 23);
            }
        };
        auto mfmas = [&](auto st_c, int kk, auto f_c, auto between) {
            if constexpr (NV > 0) {
                constexpr int ST = decltype(st_c)::value, f = decltype(f_c)::value;
                u32x4_t wv[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) wv[j] = mx_decode8(wc[ST][j][kk], sc[ST][j]);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[j][i] = mfma_bf16_32(wv[j], av[f][i], acc[j][i]);
                    between(i);
                }
            }
#pragma unroll
            for (int i = NV; i < 4; ++i) between(i);
        };
        auto nothing = [](int) {};
        const std::integral_constant<int, 0> c0;
        const std::integral_constant<int, 1> c1;
        auto step = [&](int ks, auto st_c, auto next_c) {
            constexpr int ST = decltype(st_c)::value;
            const int an = as == 2 ? 0 : as + 1, wnx = ws == 2 ? 0 : ws + 1;
            if constexpr (NV > 0) {
                rows(as, 1, c1);
                keep_order();
                mfmas(st_c, 0, c0, nothing);
                rows(as, 2, c0);
                keep_order();
                mfmas(st_c, 1, c1, nothing);
                rows(as, 3, c1);
                keep_order();
                mfmas(st_c, 2, c0, nothing);
            }
            keep_order();
            // only the step before issued anything after the next step's rows: four loads, an
            // odd one the chunk's too
            if (ST == 1) asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else if (ALIGNED) asm volatile("s_waitcnt vmcnt(7) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if constexpr (NV > 0) {
                codes(ST == 1 ? wnx : ws, next_c);
                rows(an, 0, c0);
                keep_order();
            }
            // the loads one by one between the MFMAs: in a row they would hold up the wave
            // (and with it the matrix core) until the address unit has taken them all
            const int ra = min(ks + 3, nk - 1), ca = min(ks / 2 + 3, nc - 1);
            mfmas(st_c, 3, c1, [&](int i) {
                keep_order();
                issue_rows(ra, as, i);
                if (ST == 1 && i < kParts) issue_weight(ca, ws, i);
                keep_order();
            });
            as = an;
            if (ST == 1) ws = wnx;
        };
        if constexpr (NV > 0) {
            codes(0, c0);
            rows(0, 0, c0);
        }
        for (int ks = 0; ks < nk; ks += 2) {
            step(ks, c0, c1);
            step(ks + 1, c1, c0);
        }
    };
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) issue_rows(min(i, nk - 1), i, q);
#pragma unroll
        for (int q = 0; q < kParts; ++q) issue_weight(min(i, nc - 1), i, q);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    switch (cols ? nvi : 0) {
        case 4: kloop(std::integral_constant<int, 4>{}); break;
        case 3: kloop(std::integral_constant<int, 3>{}); break;
        case 2: kloop(std::integral_constant<int, 2>{}); break;
        case 1: kloop(std::integral_constant<int, 1>{}); break;
        default: kloop(std::integral_constant<int, 0>{}); break;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= nvi) break;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; v += 4)
                    stage4(p, smem, t, wm * 128 + i * 32 + r32, wn * 64 + j * 32 + 2 * v + 4 * h, p.N, acc[j][i][v],
                           acc[j][i][v + 1], acc[j][i][v + 2], acc[j][i][v + 3]);
        }
    }
    store_staged(p, smem, t, p.N);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
constexpr int kGDout = 256 * 128;                        // 64 n of the tile's bf16 gradient rows (32 KB)
constexpr int kGCodes = 64 * 128;                        // 64 weight rows, 256 k (8 KB)
constexpr int kGPitch = 144;                             // scales: [8 blocks][64 rows] as the upper halves of
constexpr int kGScales = 8 * kGPitch;                    //   fp32 powers of two; the pitch spreads the banks
constexpr int kGSlot = kGDout + kGCodes + kGScales;
constexpr int kGOffRaw = 3 * kGSlot, kGRaw = 512 * 4;    // scale bytes as loaded, a dword each, three stages
constexpr int kGLds = kGOffRaw + 3 * kGRaw;              // 130 KB (the output's staging: 132 KB)
constexpr int kGLdsAll = kGLds > kTM * kYS * 2 ? kGLds : kTM * kYS * 2;

// VECTOR: dout's rows in 16-byte units (dout_vector), else element by element
// through registers.
template <bool VECTOR>
__global__ __launch_bounds__(kTThreads) void grad_tile_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const Tile t = find_tile(p, (p.K + kTN - 1) / kTN, reinterpret_cast<int*>(smem));
    if (t.g < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int r32 = lane & 31;
    const int wt = wave >> 1, wk = wave & 1;             // rows 64 wt .. +64, columns 128 wk .. +128
    const int KB = p.K / 32, kb0 = t.nt * 8, nn = (p.N + 63) / 64;

    // dout: four loads of 8 rows a wave and stage; codes: one of 8 weight rows x 128
    // bytes, whose two 64-byte halves trade places in every other group of 8 rows (the
    // two lane halves read rows 8 apart: different banks); scales: one byte a thread
    const uint16_t* dbase = static_cast<const uint16_t*>(p.a) + (int64_t)t.rb * p.as;
    uint32_t doff[4];
    int du[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = (wave * 4 + q) * 8 + (lane >> 3);
        du[q] = (lane & 7) ^ (lane >> 3) ^ (q & 1);
        doff[q] = (uint32_t)(min(r, t.re - 1 - t.rb) * p.as + du[q] * 8);
    }
    // (columns past K: zeros at every stage)
    const int crow = wave * 8 + (lane >> 3), cunit = (lane & 7) ^ ((wave & 1) << 2);
    const bool cin = kb0 + cunit < KB;
    const uint8_t* cbase = p.w + (int64_t)t.g * p.N * (p.K / 2) + kb0 * 16;
    const uint32_t coff = crow * (uint32_t)(p.K / 2) + cunit * 16;
    const int srow = tid >> 3, sblk = tid & 7;
    const bool sin = kb0 + sblk < KB;
    const uint8_t* sbase = p.w_s + (int64_t)t.g * p.N * KB + kb0;
    const uint32_t soff = srow * (uint32_t)KB + sblk;

    // part 0 .. 3: the wave's gradient rows; 4: its weight rows' codes
    auto issue = [&](int s, int slot, int part) {
        uint8_t* base = smem + slot * kGSlot;
        if (part < 4) {
            const uint16_t* src = scalar(dbase + s * 64) + doff[part];
            uint8_t* dst = base + (wave * 4 + part) * 1024;
            const int left = p.N - s * 64 - du[part] * 8;
            if (VECTOR) to_lds16(within(left > 0, src), dst);
            else *reinterpret_cast<u32x4_t*>(dst + lane * 16) = load8_bf16<false>(src, left);
        } else {
            to_lds16(within(cin && s * 64 + crow < p.N, scalar(cbase + (int64_t)s * 64 * (p.K / 2)) + coff),
                     base + kGDout + wave * 1024);
        }
    };
    // scales: byte tid of a stage (row tid / 8, block tid % 8) to a dword of its own
    auto issue_scales = [&](int s, int slot) {
        to_lds1(within(sin && s * 64 + srow < p.N, scalar(sbase + (int64_t)s * 64 * KB) + soff),
                smem + kGOffRaw + slot * kGRaw + wave * 256);
    };
    // and from there to where the operands are decoded
    auto put_scales = [&](int slot) {
        const uint32_t b = smem[kGOffRaw + slot * kGRaw + tid * 4];
        const uint32_t at = lds_offset(smem) + slot * kGSlot + kGDout + kGCodes + sblk * kGPitch + srow * 2;
        // written out: before an ordinary LDS store the compiler waits for every direct
        // load in flight (they write LDS too).  The step's own wait covers it.
        asm volatile("ds_write_b16 %0, %1" ::"v"(at), "v"(b << 7) : "memory");
    };

    f32x16_t acc[4][2];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[c][i][v] = 0.f;
    const int nvi = max(0, min(2, (t.re - t.rb - wt * 64 + 31) >> 5));
    const bool cols = kb0 * 32 + wk * 128 < p.K;

    // Stage s in slot s % 3.  Lane half h of substep q (16 n) takes rows 16 q + 8 h .. + 8.
    // Operands are read one substep ahead, a stage's first ones before the last MFMAs of
    // the stage before; the barrier stands there, after which the stage's slot is free for
    // stage s + 3 and the wait has left only the last step's loads in flight.  A stage's
    // scales are loaded one step earlier than its rest and rearranged in the step before
    // its own, ahead of that step's barrier.
    auto nloop = [&](auto nv_c) {
        constexpr int NV = decltype(nv_c)::value;
        uint32_t code[2][8];
        u32x4_t sc[2], dv[2][2];                          // by parity of the substep
        int slot = 0;
        auto operands = [&](int sl, int q, auto f_c) {
            constexpr int f = decltype(f_c)::value;
            const uint8_t* D = smem + sl * kGSlot;
            const uint8_t* C = D + kGDout + ((wk ^ h) * 64) + 2 * r32 + (16 * q + 8 * h) * 128;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                dv[f][i] = *reinterpret_cast<const u32x4_t*>(D + swz8(wt * 64 + i * 32 + r32, 2 * q + h));
            sc[f] = *reinterpret_cast<const u32x4_t*>(D + kGDout + kGCodes + (wk * 4 + (r32 >> 3)) * kGPitch +
                                                      (16 * q + 8 * h) * 2);
#pragma unroll
            for (int j = 0; j < 8; ++j) code[f][j] = *reinterpret_cast<const uint16_t*>(C + j * 128);
        };
        auto mfmas = [&](auto f_c, auto between) {
            constexpr int f = decltype(f_c)::value;
            u32x4_t op[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float s0 = __uint_as_float(sc[f][j / 2] << 16), s1 = __uint_as_float(sc[f][j / 2] & 0xFFFF0000u);
                const uint32_t c0 = code[f][j], c1 = code[f][j + 1];
                const uint32_t a0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c0, s0, 0));
                const uint32_t a1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c0, s0, 1));
                const uint32_t b0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c1, s1, 0));
                const uint32_t b1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c1, s1, 1));
                op[0][j / 2] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
                op[1][j / 2] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
                op[2][j / 2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
                op[3][j / 2] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    acc[c][i] = mfma_bf16_32(op[c], dv[f][i], acc[c][i]);
                    if (i == NV - 1) between(c);
                }
        };
        auto nothing = [](int) {};
        const std::integral_constant<int, 0> c0;
        const std::integral_constant<int, 1> c1;
        if constexpr (NV > 0) operands(0, 0, c0);
        for (int s = 0; s < nn; ++s) {
            const int next = slot == 2 ? 0 : slot + 1;
            put_scales(next);
            if constexpr (NV > 0) {
                operands(slot, 1, c1);
                keep_order();
                mfmas(c0, nothing);
                operands(slot, 2, c0);
                keep_order();
                mfmas(c1, nothing);
                operands(slot, 3, c1);
                keep_order();
                mfmas(c0, nothing);
            }
            keep_order();
            if (VECTOR) asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(2) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            // the loads one by one between the MFMAs (in a row they would hold up the wave
            // until the address unit has taken them all)
            auto ahead = [&](int i) {
                keep_order();
                issue(min(s + 3, nn - 1), slot, i);
                if (i == 3) {
                    issue(min(s + 3, nn - 1), slot, 4);
                    issue_scales(min(s + 4, nn - 1), next);
                }
                keep_order();
            };
            if constexpr (NV > 0) {
                operands(next, 0, c0);
                keep_order();
                mfmas(c1, ahead);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) ahead(i);
            }
            slot = next;
        }
    };
#pragma unroll
    for (int s = 0; s < 3; ++s) {
#pragma unroll
        for (int part = 0; part < 5; ++part) issue(min(s, nn - 1), s, part);
        issue_scales(min(s, nn - 1), s);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    put_scales(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    issue_scales(min(3, nn - 1), 0);
    switch (cols ? nvi : 0) {
        case 2: nloop(std::integral_constant<int, 2>{}); break;
        case 1: nloop(std::integral_constant<int, 1>{}); break;
        default: nloop(std::integral_constant<int, 0>{}); break;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // operand row i of MFMA c holds column 4 i + c: value v of the four c are four
    // consecutive columns
    if (cols) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= nvi) break;
#pragma unroll
            for (int v = 0; v < 16; ++v)
                stage4(p, smem, t, wt * 64 + i * 32 + r32, wk * 128 + 4 * (8 * (v >> 2) + 4 * h + (v & 3)), p.K,
                       acc[0][i][v], acc[1][i][v], acc[2][i][v], acc[3][i][v]);
        }
    }
    store_staged(p, smem, t, p.K);
}

template <auto Kern, int LDS>
static hipError_t launch_tiles(const ProductArgs& p, int width, hipStream_t s) {
    const hipError_t e = allow_dynamic_lds<Kern>(LDS);
    if (e != hipSuccess) return e;
    const int64_t grid = tile_grid(p, (width + kTN - 1) / kTN);
    hipLaunchKernelGGL(Kern, dim3((unsigned)grid), dim3(kTThreads), LDS, s, p);
    return hipGetLastError();
}

hipError_t launch_product_tiles(const ProductArgs& p, hipStream_t s) {
    const bool aligned =
        p.K % 128 == 0 && ((reinterpret_cast<uintptr_t>(p.w_s) | reinterpret_cast<uintptr_t>(p.a_s)) & 3) == 0;
    if (p.a_s)
        return aligned ? launch_tiles<mx_tile_kernel<true>, mx_lds(true)>(p, p.N, s)
                       : launch_tiles<mx_tile_kernel<false>, mx_lds(false)>(p, p.N, s);
    return aligned ? launch_tiles<a16_tile_kernel<true>, a16_lds(true)>(p, p.N, s)
                   : launch_tiles<a16_tile_kernel<false>, a16_lds(false)>(p, p.N, s);
}

hipError_t launch_product_grad_tiles(const ProductArgs& p, hipStream_t s) {
    return dout_vector(p) ? launch_tiles<grad_tile_kernel<true>, kGLdsAll>(p, p.K, s)
                          : launch_tiles<grad_tile_kernel<false>, kGLdsAll>(p, p.K, s);
}

}  // namespace moe
