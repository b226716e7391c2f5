// Shared by the kernels of products in tiles of 256 rows of one group x 256 outputs: direct
// loads to LDS, the tiles of a launch, outputs on their way out.
#pragma once
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "ops.h"
#include "product_common.h"

namespace moe {

constexpr int kTM = 256, kTN = 256, kTWaves = 8, kTThreads = 64 * kTWaves;

typedef __attribute__((address_space(3))) void lds_void_t;
typedef int i32x2_t __attribute__((ext_vector_type(2)));

static __device__ __align__(16) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}

// A direct load of BYTES a lane from a scalar base and a 32-bit lane offset to LDS
// (lane i at dst + i * max(BYTES, 4); dst is the same for the wave).  Written out: the
// compiler adds 64-bit addresses a lane for each load inside a loop.  M0 holds the LDS
// address (one wait state before its use); nothing comes back to registers, and the
// kernels' own waits cover the loads (before a transposing LDS read the compiler waits
// for every load of its own builtin).
template <int BYTES>
__device__ __forceinline__ void load_lds(const void* base, uint32_t off, const void* dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_offset(dst));
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                     ::"v"(off), "s"(base), "s"(at) : "memory", "m0");
    else if constexpr (BYTES == 4)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                     ::"v"(off), "s"(base), "s"(at) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1"
                     ::"v"(off), "s"(base), "s"(at) : "memory", "m0");
}
// The same from an address a lane.
template <int BYTES>
__device__ __forceinline__ void load_lds(const void* src, const void* dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_offset(dst));
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                     ::"v"(src), "s"(at) : "memory", "m0");
    else if constexpr (BYTES == 4)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                     ::"v"(src), "s"(at) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off"
                     ::"v"(src), "s"(at) : "memory", "m0");
}
// Operand reads stay before the MFMAs that follow them in the source (the scheduler
// would sink each read to its use and wait for it there).
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

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

template <int TM = kTM>
static int64_t tile_grid(const ProductArgs& p, int NT) {
    // groups' partial tiles: at most one each
    const int64_t tiles = p.M / TM + min(p.G, p.M);
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
                   width - t.nt * kTN - col);
        return;
    }
    *reinterpret_cast<u32x2_t*>(smem + (row * kYS + col) * 2) = pack4(p.out_dtype, a, b, c, d);
}

__device__ __forceinline__ void store_staged(const ProductArgs& p, const uint8_t* smem, const Tile& t, int width) {
    if (p.out_dtype == kF32) return;
    __syncthreads();
    const int nrow = t.re - t.rb, ncol = min(kTN, width - t.nt * kTN);
    uint16_t* out = static_cast<uint16_t*>(p.out) + t.rb * p.os + t.nt * kTN;
    for (int x = threadIdx.x; x < kTM * (kTN / 8); x += kTThreads) {
        const int row = x >> 5, c = (x & 31) * 8;
        if (row >= nrow) break;                          // rows grow with x
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + (row * kYS + c) * 2);
        if (c + 8 <= ncol) {
            *reinterpret_cast<u32x4_any_t*>(out + row * p.os + c) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < ncol) out[row * p.os + c + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        }
    }
}

// Scales of 256 rows and `blocks` blocks in LDS: a row's bytes together, or (rows that
// are not aligned to dwords) each byte in a dword of its own, [blocks][256 rows].
constexpr int scale_bytes(bool aligned, int blocks) { return 256 * blocks * (aligned ? 1 : 4); }
constexpr int kWaveStage = 2048;                            // a wave's 32 x 32 outputs on their way out
constexpr int kTable = (1024 + 1) * 4;

// table[g] = tiles (of TM rows) of the groups before g, g = 0 .. G; returns their total.  512
// threads; ends with a barrier.
template <int TM = kTM>
__device__ __forceinline__ int tile_table(const ProductArgs& p, int* table) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int rb = 0, re = 0;
        if (2 * tid + i < p.G) group_rows(p, 2 * tid + i, rb, re);
        n[i] = (re - rb + TM - 1) / TM;
    }
    const int sum = n[0] + n[1];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(inc, o, 64);
        if (lane >= o) inc += y;
    }
    if (lane == 63) table[wave] = inc;
    __syncthreads();
    int at = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kTWaves; ++w) {
        if (w < wave) at += table[w];
        total += table[w];
    }
    __syncthreads();
    if (2 * tid <= p.G) table[2 * tid] = at;
    if (2 * tid + 1 <= p.G) table[2 * tid + 1] = at + n[0];
    if (tid == 0 && p.G == 1024) table[1024] = total;
    __syncthreads();
    // (offsets that decrease could claim more tiles than the rows hold)
    return __builtin_amdgcn_readfirstlane(min(total, p.M / TM + p.G));
}

// Tile `logical` (tile-major, NT column blocks a tile) by search in the table.
template <int TM = kTM>
__device__ __forceinline__ Tile table_tile(const ProductArgs& p, const int* table, int logical, int NT) {
    const int tile = logical / NT;
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__builtin_amdgcn_readfirstlane(table[mid]) <= tile) lo = mid;
        else hi = mid;
    }
    int rb, re;
    group_rows(p, lo, rb, re);
    rb += (tile - __builtin_amdgcn_readfirstlane(table[lo])) * TM;
    return Tile{lo, __builtin_amdgcn_readfirstlane(rb), __builtin_amdgcn_readfirstlane(min(rb + TM, re)),
                logical - tile * NT};
}

// A wave's 32 tokens x 32 outputs to memory through 2 KB of LDS of its own, without a
// barrier: tokens' 64-byte rows, whose 16-byte units trade places by row so that both the
// 8-byte stores and the 16-byte loads spread over all banks.  The lane's four values 4 g
// .. + 4 are outputs 8 g + 4 h .. + 4 (an accumulator), or, PAIRED, 16 (g / 2) + 8 h + 4 (g
// % 2) .. + 4 (the backward's column pairs).
template <bool PAIRED>
__device__ __forceinline__ void wave_store(const ProductArgs& p, uint8_t* stage, const Tile& t, int row0, int col0,
                                           int width, const f32x16_t& acc) {
    const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5;
    const int left = width - t.nt * kTN - col0;
    if (p.out_dtype == kF32) {
        if (t.rb + row0 + r32 < t.re) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = PAIRED ? 16 * (g >> 1) + 8 * h + 4 * (g & 1) : 8 * g + 4 * h;
                store4(p.out, kF32, (t.rb + row0 + r32) * p.os + t.nt * kTN + col0 + c,
                       f32x4_t{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]}, left - c);
            }
        }
        return;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const u32x2_t v = pack4(p.out_dtype, acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
        const int unit = PAIRED ? 2 * (g >> 1) + h : g, half = PAIRED ? g & 1 : h;
        const uint32_t at = lds_offset(stage) + r32 * 64 + ((unit ^ (r32 >> 2)) & 3) * 16 + half * 8;
        // written out: before an ordinary LDS store the compiler waits for every direct
        // load in flight.  LDS serves a wave in order: the loads below come after.
        asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(v) : "memory");
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = x * 16 + (lane >> 2), u = lane & 3;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stage + r * 64 + ((u ^ (r >> 2)) & 3) * 16);
        if (t.rb + row0 + r >= t.re) continue;
        uint16_t* o = static_cast<uint16_t*>(p.out) + (t.rb + row0 + r) * p.os + t.nt * kTN + col0 + 8 * u;
        if (8 * u + 8 <= left) {
            *reinterpret_cast<u32x4_any_t*>(o) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (8 * u + i < left) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        }
    }
}

// An accumulator through 1 KB, 16 outputs (tokens' 32-byte rows) at a time.
__device__ __forceinline__ void wave_store_halves(const ProductArgs& p, uint8_t* stage, const Tile& t, int row0,
                                                  int col0, int width, const f32x16_t& acc) {
    const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5;
    const int left = width - t.nt * kTN - col0;
    if (p.out_dtype == kF32) {
        wave_store<false>(p, stage, t, row0, col0, width, acc);
        return;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int v0 = 8 * x + 4 * g;
            const u32x2_t v = pack4(p.out_dtype, acc[v0], acc[v0 + 1], acc[v0 + 2], acc[v0 + 3]);
            const uint32_t at = lds_offset(stage) + r32 * 32 + ((g ^ (r32 >> 3)) & 1) * 16 + h * 8;
            asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(v) : "memory");
        }
        const int r = lane >> 1, u = lane & 1, c = 16 * x + 8 * u;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stage + r * 32 + ((u ^ (r >> 3)) & 1) * 16);
        if (t.rb + row0 + r >= t.re) continue;
        uint16_t* o = static_cast<uint16_t*>(p.out) + (t.rb + row0 + r) * p.os + t.nt * kTN + col0 + c;
        if (c + 8 <= left) {
            *reinterpret_cast<u32x4_any_t*>(o) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < left) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        }
    }
}

template <auto Kern, int LDS>
static hipError_t launch_tiles(const ProductArgs& p, int64_t grid, hipStream_t s) {
    const hipError_t e = allow_dynamic_lds<Kern>(LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(Kern, dim3((unsigned)grid), dim3(kTThreads), LDS, s, p);
    return hipGetLastError();
}

}  // namespace moe
