// MXFP4 products in tiles, for many rows a group (gfx950).  A tile is 256 rows of
// one group x 256 outputs; eight waves, one workgroup a CU (the operands' rings fill the
// LDS); the operands come straight from global memory to LDS (global_load_lds).  The
// weight is the matrix cores' row operand and tokens are their columns, so that a lane
// ends with groups of four consecutive outputs of one token (packed stores).  An
// operand is read from LDS one group of MFMAs ahead of its use, across the stage's
// barrier too, so that the matrix cores do not wait for LDS.
//
//   mx_tile_kernel     W4A4: 32x32x64 scaled MFMAs on the codes as they lie in memory;
//                      256 k (a full line a row) a stage, two stages; a workgroup takes
//                      tile after tile, the next one's stages loading while the last
//                      one's outputs leave.  65536 rows over 320 experts of 2048 x 4096:
//                      472 us, 2.33 PFLOP/s, 3.9 TB/s (its loads alone, without LDS reads
//                      and MFMAs: 417 us); 16384 x 8192 x 8192: 638 us, 3.45 PFLOP/s (loads
//                      alone 539 us).  Bound by the loads' line accesses and depth: 128 k a
//                      stage in four stages (64-byte pieces) took 844 us, scales every stage
//                      instead of every other 682 us, touching lines two stages early 716 us.
//                      Groups' tiles of even height instead of 256 rows and a rest: within 1%.
//   a16_tile_kernel    W4A16: bf16 rows, 64 k a stage, three stages; each wave decodes
//                      its weight operand in registers (one conversion a pair, the block
//                      scale within it), then 32x32x16 bf16 MFMAs.  32768 rows over 64
//                      experts of 2048 x 4096: 515 us, 1.07 PFLOP/s; 16384 x 8192 x 8192:
//                      1.67 ms, 1.31 PFLOP/s, as a large bf16 product of the library (1.28).
//                      The clock falls to 2.05 GHz under it; the matrix cores are busy half of
//                      the former's cycles (a fifth of its tiles hold a few rows only).
//   grad_tile_kernel   backward: the reduction runs over the weight's rows, 64 a stage,
//                      three stages; a lane takes two neighbouring columns of eight rows
//                      with one transposing LDS read, decodes them between the MFMAs and
//                      regroups the pairs by column.  32768 rows over 64 experts of 2048 x
//                      4096: 604 us, 0.91 PFLOP/s (617 with a read a row); 16384 x 8192 x
//                      8192: 1.92 ms, 1.14 PFLOP/s.  No one resource bounds it: timing-only
//                      variants of the former took 525 us without the row operands' LDS
//                      reads, 523 without the decoding, 481 without the loads, and as long
//                      without the scales' LDS reads.  64 x 128 wave tiles were as fast with
//                      16-bit LDS reads and took 677 us with eight rows' dwords side by side;
//                      four waves of 256 x 64 (half the decoding, one wave a SIMD) took 2.08 ms
//                      on the latter product; tiles of even height 642 us on the former.
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

// ---------------------------------------------------------------------------
// W4A4
// ---------------------------------------------------------------------------
// Scales of 256 rows and `blocks` blocks in LDS: a row's bytes together, or (rows that
// are not aligned to dwords) each byte in a dword of its own, [blocks][256 rows].
constexpr int scale_bytes(bool aligned, int blocks) { return 256 * blocks * (aligned ? 1 : 4); }
constexpr int kMxCodes = 256 * 128;                         // an operand's 256 k of a stage
// weight | rows; with them the stage's scales, or (aligned) those of two stages apart, for
// a row's few bytes cost a line access however many they are
constexpr int mx_slot(bool aligned) { return 2 * kMxCodes + (aligned ? 0 : 2 * scale_bytes(false, 8)); }
constexpr int kMxPair = 2 * scale_bytes(true, 16);          // two stages' scales of both operands
constexpr int kWaveStage = 2048;                            // a wave's 32 x 32 outputs on their way out
constexpr int kTable = (1024 + 1) * 4;
// LDS: stages [2] | scales [2] | waves' staging [8] (half a block each) | table.  Without
// aligned scales the stages take all 160 KB: one tile a workgroup, staged and looked up in
// the stages' place.
constexpr int kMxOffS = 2 * mx_slot(true), kMxOffStage = kMxOffS + 2 * kMxPair;
constexpr int kMxOffTable = kMxOffStage + kTWaves * kWaveStage / 2;
constexpr int mx_lds(bool aligned) { return aligned ? kMxOffTable + kTable : 2 * mx_slot(false); }

template <int OPSEL>
__device__ __forceinline__ f32x16_t mfma_mx32(const u32x4_t& a, uint32_t as, const u32x4_t& b, uint32_t bs,
                                              const f32x16_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, OPSEL, (int)as,
                                                           OPSEL, (int)bs);
}

// table[g] = tiles of the groups before g, g = 0 .. G; returns their total.  512
// threads; ends with a barrier.
__device__ __forceinline__ int tile_table(const ProductArgs& p, int* table) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int rb = 0, re = 0;
        if (2 * tid + i < p.G) group_rows(p, 2 * tid + i, rb, re);
        n[i] = (re - rb + kTM - 1) / kTM;
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
    return __builtin_amdgcn_readfirstlane(min(total, p.M / kTM + p.G));
}

// Tile `logical` (tile-major, NT column blocks a tile) by search in the table.
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
    rb += (tile - __builtin_amdgcn_readfirstlane(table[lo])) * kTM;
    return Tile{lo, __builtin_amdgcn_readfirstlane(rb), __builtin_amdgcn_readfirstlane(min(rb + kTM, re)),
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

// A workgroup takes tiles one after another: while a tile's last stages are multiplied
// the next tile's first ones are loaded, and its outputs leave while those land.
// ALIGNED: scale rows can be read in dwords (K % 128 == 0, 4-byte aligned scales).
template <bool ALIGNED>
__global__ __launch_bounds__(kTThreads) void mx_tile_kernel(ProductArgs p) {
    constexpr int kScales = scale_bytes(ALIGNED, ALIGNED ? 16 : 8), kSlot = mx_slot(ALIGNED);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int wm = wave >> 2, wn = wave & 3;             // rows 128 wm .. +128, outputs 64 wn .. +64
    const int NT = (p.N + kTN - 1) / kTN, KB = p.K / 32, nc = (KB + 7) / 8, r32 = lane & 31;

    // This workgroup's tiles: workgroup b runs on XCD b % 8, each XCD takes a contiguous
    // range (it shares the tile's rows and the group's weight in its L2), its workgroups
    // tiles next to each other.
    int* table = reinterpret_cast<int*>(smem + (ALIGNED ? kMxOffTable : 0));
    const int all = tile_table(p, table) * NT, per = (all + 7) >> 3, stride = gridDim.x >> 3;
    const int end = min(((int)blockIdx.x & 7) * per + per, all);
    int mine = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (mine >= end) return;
    Tile t = table_tile(p, table, mine, NT);
    if (!ALIGNED) __syncthreads();                       // the table's place is a stage's

    // ---- loads, two stages ahead of the multiplication ----
    // codes of a stage: per operand 32 KB, four loads of 1 KB a wave: load q of wave w
    // fills rows 8 (4 w + q) .. +8 (a full 128-byte line each), lane i row i / 8, slot
    // i % 8, which holds unit (i & 7) ^ (i >> 3) ^ (q & 1) (swz8); scales: waves 0-3 the
    // weight's rows 64 w .. +64, waves 4-7 the rows'.  Rows and outputs past the tile's
    // end: any valid row (their results are not stored).
    const uint8_t *wbase, *abase, *sbase;
    uint32_t coff[4], aoff[4], soff[ALIGNED ? 4 : 1];
    const int cu = (lane & 7) ^ (lane >> 3), srow = (wave & 3) * 64;
    const int sdst = (ALIGNED ? kMxOffS : 2 * kMxCodes) + (wave < 4 ? 0 : kScales);
    constexpr int kSLoads = ALIGNED ? 4 : 1;             // loads of 16 rows x four dwords, or (bytes) of 64 rows
    auto load_from = [&](const Tile& n) {
        const int n0 = n.nt * kTN;
        const int64_t w0 = (int64_t)n.g * p.N + n0;
        wbase = p.w + w0 * (p.K / 2);
        abase = static_cast<const uint8_t*>(p.a) + (int64_t)n.rb * (p.K / 2);
        sbase = wave < 4 ? p.w_s + w0 * KB : p.a_s + (int64_t)n.rb * KB;
        const int wmax = p.N - 1 - n0, amax = n.re - 1 - n.rb;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = (wave * 4 + q) * 8 + (lane >> 3), u = cu ^ (q & 1);
            coff[q] = min(r, wmax) * (uint32_t)(p.K / 2) + u * 16;
            aoff[q] = min(r, amax) * (uint32_t)(p.K / 2) + u * 16;
        }
#pragma unroll
        for (int q = 0; q < kSLoads; ++q) {
            const int r = srow + (ALIGNED ? q * 16 + (lane >> 2) : lane);
            soff[q] = min(r, wave < 4 ? wmax : amax) * (uint32_t)KB + (ALIGNED ? (lane & 3) * 4 : 0);
        }
    };
    // part 0 .. 3: the wave's codes of both operands; 4: its scales (ALIGNED: at even stages
    // this one's and the next's)
    int spair = 0;                                       // their slot
    auto issue = [&](int c, int slot, int part) {
        uint8_t* base = smem + slot * kSlot;
        const bool whole = c * 8 + 8 <= KB;
        if (part < 4) {
            const uint8_t *wb = wbase + (int64_t)c * 128, *ab = abase + (int64_t)c * 128;
            uint8_t *wd = base + (wave * 4 + part) * 1024, *ad = wd + kMxCodes;
            if (whole) {
                load_lds<16>(wb, coff[part], wd);
                load_lds<16>(ab, aoff[part], ad);
            } else {
                const bool in = c * 8 + (cu ^ (part & 1)) < KB;
                load_lds<16>(within(in, wb + coff[part]), wd);
                load_lds<16>(within(in, ab + aoff[part]), ad);
            }
        } else {
            const uint8_t* sb = sbase + (int64_t)c * 8;
            if (ALIGNED) {
                if (c & 1) return;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint8_t* sd = smem + spair * kMxPair + sdst + srow * 16 + q * 256;
                    if (c * 8 + 16 <= KB) load_lds<4>(sb, soff[q], sd);
                    else load_lds<4>(within(c * 8 + (lane & 3) * 4 < KB, sb + soff[q]), sd);
                }
                spair ^= 1;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint8_t* sd = base + sdst + i * 1024 + srow * 4;
                    if (whole) load_lds<1>(sb + i, soff[0], sd);
                    else load_lds<1>(within(c * 8 + i < KB, sb + i + soff[0]), sd);
                }
            }
        }
    };
    int next = mine, ic = 0;                             // tile and stage of the next loads
    bool more = true;
    auto advance = [&]() {
        if (++ic < nc) return;
        ic = 0;
        next += stride;
        more = ALIGNED && next < end;
        if (more) load_from(table_tile(p, table, next, NT));
    };

    // ---- the multiplication ----
    f32x16_t acc[2][4];
    u32x4_t wv[2][2], av[2][4];                          // operands by parity of the MFMA group
    uint32_t ws[2], as[4], wsn[2], asn[4];               // four blocks' scales; the next stage's
    auto operands = [&](int slot, auto m_c) {
        constexpr int m = decltype(m_c)::value, f = m & 1;
        const uint8_t* S = smem + slot * kSlot;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            wv[f][j] = *reinterpret_cast<const u32x4_t*>(S + swz8(wn * 64 + j * 32 + r32, 4 * h + m));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            av[f][i] = *reinterpret_cast<const u32x4_t*>(S + kMxCodes + swz8(wm * 128 + i * 32 + r32, 4 * h + m));
    };
    auto row_scales = [&](const uint8_t* S, int r) {     // blocks 4 h .. 4 h + 3 of row r
        if (ALIGNED) return *reinterpret_cast<const uint32_t*>(S + r * 16 + 4 * h);
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) v |= *reinterpret_cast<const uint32_t*>(S + (4 * h + i) * 1024 + r * 4) << (8 * i);
        return v;
    };
    int rpair = 1;                                       // slot of the scales being read
    auto scales = [&](int slot, int c) {                 // of stage c of its tile
        if (!(c & 1)) rpair ^= 1;
        const uint8_t* S = ALIGNED ? smem + kMxOffS + rpair * kMxPair + (c & 1) * 8 : smem + slot * kSlot + 2 * kMxCodes;
#pragma unroll
        for (int j = 0; j < 2; ++j) wsn[j] = row_scales(S, wn * 64 + j * 32 + r32);
#pragma unroll
        for (int i = 0; i < 4; ++i) asn[i] = row_scales(S + kScales, wm * 128 + i * 32 + r32);
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int j = 0; j < 2; ++j) ws[j] = wsn[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) as[i] = asn[i];
    };
    auto mfmas = [&](auto m_c, int i) {
        constexpr int m = decltype(m_c)::value, f = m & 1;
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j][i] = mfma_mx32<m>(wv[f][j], ws[j], av[f][i], as[i], acc[j][i]);
    };

    // A tile's stages; the running stage sits in `slot`.  Lane half h of MFMA group m
    // (0 .. 3) takes block 4 h + m of the stage's eight.  A group's operands are read before
    // the MFMAs of the group before it, so that the matrix cores do not wait for LDS; the
    // barrier stands before a stage's last MFMAs, where its slot has been read and the
    // stage after the next may take it.
    int slot = 0;
    auto stages = [&](int nv) {                          // nv: 32-row blocks of this wave with rows
        auto group = [&](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            operands(slot, std::integral_constant<int, m + 1>{});
            keep_order();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < nv) mfmas(m_c, i);
            keep_order();
        };
        for (int c = 0; c < nc; ++c) {
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            group(std::integral_constant<int, 2>{});
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            operands(slot ^ 1, std::integral_constant<int, 0>{});
            scales(slot ^ 1, c + 1 < nc ? c + 1 : 0);
            keep_order();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < nv) mfmas(std::integral_constant<int, 3>{}, i);
                keep_order();
                if (more) issue(ic, slot, i);
                keep_order();
            }
            if (more) {
                issue(ic, slot, 4);
                advance();
            }
            take_scales();
            slot ^= 1;
        }
    };

    load_from(t);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (!more) continue;
#pragma unroll
        for (int part = 0; part < 5; ++part) issue(ic, c, part);
        advance();
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    operands(0, std::integral_constant<int, 0>{});
    scales(0, 0);
    take_scales();
    for (;;) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
        const bool cols = t.nt * kTN + wn * 64 < p.N;
        const int nvi = cols ? max(0, min(4, (t.re - t.rb - wm * 128 + 31) >> 5)) : 0;   // 32-row blocks with rows
        stages(nvi);
        if (!ALIGNED) __syncthreads();                   // staged in the stages' place
        uint8_t* stage = smem + (ALIGNED ? kMxOffStage : 0) + wave * kWaveStage / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= nvi) break;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                wave_store_halves(p, stage, t, wm * 128 + i * 32, wn * 64 + j * 32, p.N, acc[j][i]);
        }
        mine += stride;
        if (!ALIGNED || mine >= end) break;
        t = table_tile(p, table, mine, NT);
    }
}

// ---------------------------------------------------------------------------
// W4A16
// ---------------------------------------------------------------------------
constexpr int kARows = 256 * 128;                        // 64 k of the tile's bf16 rows (32 KB)
constexpr int kAWeight = 256 * 64;                        // 128 k of the weight's codes
// LDS: rows [3] | codes [3] | scales [2], each 256 k of them: loading them 128 k at a time
// took as many line accesses as the rows (a row's few bytes are a line of their own)
constexpr int kAOffW = 3 * kARows, kAOffS = kAOffW + 3 * kAWeight;
constexpr int a16_lds(bool aligned) { return kAOffS + 2 * scale_bytes(aligned, 8); }   // 148 or 160 KB

__device__ __forceinline__ f32x16_t mfma_bf16_32(const u32x4_t& a, const u32x4_t& b, const f32x16_t& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}

template <bool ALIGNED>
__global__ __launch_bounds__(kTThreads) void a16_tile_kernel(ProductArgs p) {
    constexpr int kScales = scale_bytes(ALIGNED, 8);
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

    // rows: four loads of 1 KB (8 rows of 128 bytes) a wave and step; codes: two of 1 KB
    // (16 rows of 64 bytes) a wave and chunk of 128 k; scales, every 256 k: 32 rows' two
    // dwords a wave, or (not ALIGNED) each of their eight bytes to a dword
    uint32_t aoff[4];
    int au[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = (wave * 4 + q) * 8 + (lane >> 3);
        au[q] = (lane & 7) ^ (lane >> 3) ^ (q & 1);
        aoff[q] = (uint32_t)(min(r, t.re - 1 - t.rb) * p.as + au[q] * 8) * 2;
    }
    uint32_t coff[2];
    int cu[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = (wave * 2 + q) * 16 + (lane >> 2);
        cu[q] = (lane & 3) ^ (((r >> 1) ^ (r >> 3)) & 3);
        coff[q] = wrow(r) * (uint32_t)(p.K / 2) + cu[q] * 16;
    }
    constexpr int kSLoads = ALIGNED ? 1 : 4, kSLanes = ALIGNED ? 2 : 8;      // lanes a row
    uint32_t soff[kSLoads];
    const int sb = (lane & (kSLanes - 1)) * (8 / kSLanes);
#pragma unroll
    for (int q = 0; q < kSLoads; ++q) soff[q] = wrow(wave * 32 + q * 8 + lane / kSLanes) * (uint32_t)KB + sb;

    auto issue_rows = [&](int ks, int slot) {
        uint8_t* base = smem + slot * kARows + wave * 4096;
        const uint16_t* ab = abase + (int64_t)ks * 64;
        if (ALIGNED || ks * 2 + 2 <= KB) {
#pragma unroll
            for (int q = 0; q < 4; ++q) load_lds<16>(ab, aoff[q], base + q * 1024);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                load_lds<16>(within(ks * 8 + au[q] < KB * 4, reinterpret_cast<const uint8_t*>(ab) + aoff[q]),
                         base + q * 1024);
        }
    };
    auto issue_codes = [&](int c, int slot) {
        uint8_t* base = smem + kAOffW + slot * kAWeight;
        const uint8_t* wb = wbase + (int64_t)c * 64;
        if (ALIGNED || c * 4 + 4 <= KB) {
#pragma unroll
            for (int q = 0; q < 2; ++q) load_lds<16>(wb, coff[q], base + (wave * 2 + q) * 1024);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                load_lds<16>(within(c * 4 + cu[q] < KB, wb + coff[q]), base + (wave * 2 + q) * 1024);
        }
    };
    auto issue_scales = [&](int c, int slot) {            // c: of 256 k
        uint8_t* base = smem + kAOffS + slot * kScales + wave * (kScales / kTWaves);
        const uint8_t* src = sbase + (int64_t)c * 8;
        const bool whole = c * 8 + 8 <= KB;
#pragma unroll
        for (int q = 0; q < kSLoads; ++q) {
            if (whole) {
                load_lds<ALIGNED ? 4 : 1>(src, soff[q], base + q * 256);
            } else {
                const void* from = within(c * 8 + sb < KB, src + soff[q]);
                if (ALIGNED) load_lds<4>(from, base);
                else load_lds<1>(from, base + q * 256);
            }
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

    // Step ks: rows in slot ks % 3, codes of chunk ks / 2 in slot (ks / 2) % 3, scales in
    // slot (ks / 4) % 2.  Lane half h of MFMA kk (0 .. 3) takes k = 32 h + 8 kk .. + 8 of the
    // step: dword kk of the weight row's unit 2 (ks % 2) + h, and the row's unit 4 h + kk.
    // Operands are read one MFMA ahead, a step's first ones before the last MFMAs of the
    // step before.  The barrier stands there: the step's rows have been read (slot free for
    // step ks + 3), after an odd step its codes (for chunk + 3), after every fourth its
    // scales.  The wait leaves in flight only what was issued since the next step's rows:
    // six loads or more (past the end valid data again).
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
        auto codes = [&](int ks, int slot, auto st_c) {
            constexpr int ST = decltype(st_c)::value;
            const uint8_t* W = smem + kAOffW + slot * kAWeight;
            const uint8_t* S = smem + kAOffS + ((ks >> 2) & 1) * kScales + (2 * (ks & 3) + h) * (ALIGNED ? 1 : 4);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = wn * 64 + j * 32 + r32;
                wc[ST][j] = *reinterpret_cast<const u32x4_t*>(W + swz4(r, 2 * ST + h));
                sc[ST][j] = __uint_as_float((uint32_t)S[r * (kScales / 256)] << 23);
            }
        };
        auto mfmas = [&](auto st_c, int kk, auto f_c) {
            constexpr int ST = decltype(st_c)::value, f = decltype(f_c)::value;
            u32x4_t wv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) wv[j] = mx_decode8(wc[ST][j][kk], sc[ST][j]);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j][i] = mfma_bf16_32(wv[j], av[f][i], acc[j][i]);
        };
        const std::integral_constant<int, 0> c0;
        const std::integral_constant<int, 1> c1;
        auto step = [&](int ks, auto st_c, auto next_c) {
            constexpr int ST = decltype(st_c)::value;
            const int an = as == 2 ? 0 : as + 1, wnx = ws == 2 ? 0 : ws + 1;
            if constexpr (NV > 0) {
                rows(as, 1, c1);
                keep_order();
                mfmas(st_c, 0, c0);
                rows(as, 2, c0);
                keep_order();
                mfmas(st_c, 1, c1);
                rows(as, 3, c1);
                keep_order();
                mfmas(st_c, 2, c0);
            }
            keep_order();
            asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            issue_rows(min(ks + 3, nk - 1), as);
            if (ST == 1) issue_codes(min(ks / 2 + 3, nc - 1), ws);
            if (ST == 1 && (ks & 3) == 3) issue_scales(min(ks / 4 + 2, (nc - 1) / 2), (ks >> 2) & 1);
            if constexpr (NV > 0) {
                codes(ks + 1, ST == 1 ? wnx : ws, next_c);
                rows(an, 0, c0);
                keep_order();
                mfmas(st_c, 3, c1);
            }
            as = an;
            if (ST == 1) ws = wnx;
        };
        if constexpr (NV > 0) {
            codes(0, 0, c0);
            rows(0, 0, c0);
        }
        for (int ks = 0; ks < nk; ks += 2) {
            step(ks, c0, c1);
            step(ks + 1, c1, c0);
        }
    };
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        issue_rows(min(i, nk - 1), i);
        issue_codes(min(i, nc - 1), i);
        if (i < 2) issue_scales(min(i, (nc - 1) / 2), i);
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
constexpr int kGScales = 64 * 8 * 4;                     // their scales, a byte in a dword each
constexpr int kGSlot = kGDout + kGCodes + kGScales;
constexpr int kGOffStage = 3 * kGSlot, kGOffTable = kGOffStage + kTWaves * kWaveStage;
constexpr int kGLds = kGOffTable + kTable;               // stages [3] | waves' staging [8] | table: 147 KB

// Tiles one after another, as in mx_tile_kernel.  VECTOR: dout's rows in 16-byte units
// (dout_vector), else element by element through registers.
template <bool VECTOR>
__global__ __launch_bounds__(kTThreads) void grad_tile_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int r32 = lane & 31, wt = wave >> 2, wk = wave & 3;    // rows 128 wt .. +128, columns 64 wk .. +64
    const int NT = (p.K + kTN - 1) / kTN, KB = p.K / 32, nn = (p.N + 63) / 64;
    int* table = reinterpret_cast<int*>(smem + kGOffTable);
    const int all = tile_table(p, table) * NT, per = (all + 7) >> 3, stride = gridDim.x >> 3;
    const int end = min(((int)blockIdx.x & 7) * per + per, all);
    int mine = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (mine >= end) return;
    Tile t = table_tile(p, table, mine, NT);

    // ---- loads, three stages ahead ----
    // dout: four loads of 8 rows a wave and stage; codes: one of 8 weight rows x 128
    // bytes, unit u of a row in slot u ^ (row & 7) (a transposing read takes a unit of
    // eight rows: different banks); scales: wave w's rows 8 w .. +8,
    // lane i block i / 8 of row i % 8, so that eight rows' scales of a block follow each
    // other.  Columns past K, rows past N: zeros.
    const uint16_t* dbase;
    const uint8_t *cbase, *sbase;
    uint32_t doff[4];
    bool cin, sin, whole;                                // columns of this lane's, of the whole tile
    const int crow = wave * 8 + (lane >> 3), cunit = (lane & 7) ^ (lane >> 3), srow = wave * 8 + (lane & 7);
    const uint32_t coff = crow * (uint32_t)(p.K / 2) + cunit * 16, soff = srow * (uint32_t)KB + (lane >> 3);
    const int du = cunit;
    auto load_from = [&](const Tile& n) {
        dbase = static_cast<const uint16_t*>(p.a) + (int64_t)n.rb * p.as;
        cbase = p.w + (int64_t)n.g * p.N * (p.K / 2) + n.nt * 128;
        sbase = p.w_s + (int64_t)n.g * p.N * KB + n.nt * 8;
        cin = n.nt * 8 + cunit < KB;
        sin = n.nt * 8 + (lane >> 3) < KB;
        whole = n.nt * 8 + 8 <= KB;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = (wave * 4 + q) * 8 + (lane >> 3);
            doff[q] = (uint32_t)(min(r, n.re - 1 - n.rb) * p.as + (du ^ (q & 1)) * 8) * 2;
        }
    };
    auto issue = [&](int s, int slot) {
        uint8_t* base = smem + slot * kGSlot;
        const uint16_t* db = dbase + s * 64;
        const uint8_t* cs = cbase + (int64_t)s * 64 * (p.K / 2);
        const uint8_t* ss = sbase + (int64_t)s * 64 * KB;
        uint8_t *cd = base + kGDout + wave * 1024, *sd = base + kGDout + kGCodes + wave * 256;
        if (VECTOR && whole && s * 64 + 64 <= p.N) {
#pragma unroll
            for (int q = 0; q < 4; ++q) load_lds<16>(db, doff[q], base + (wave * 4 + q) * 1024);
            load_lds<16>(cs, coff, cd);
            load_lds<1>(ss, soff, sd);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint8_t* dst = base + (wave * 4 + q) * 1024;
                const uint16_t* src = reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(db) + doff[q]);
                const int left = p.N - s * 64 - (du ^ (q & 1)) * 8;
                if (VECTOR) load_lds<16>(within(left > 0, src), dst);
                else *reinterpret_cast<u32x4_t*>(dst + lane * 16) = load8_bf16(src, left);
            }
            load_lds<16>(within(cin && s * 64 + crow < p.N, cs + coff), cd);
            load_lds<1>(within(sin && s * 64 + srow < p.N, ss + soff), sd);
        }
    };
    int next = mine, is = 0;                             // tile and stage of the next loads
    bool more = true;
    auto advance = [&]() {
        if (++is < nn) return;
        is = 0;
        next += stride;
        more = next < end;
        if (more) load_from(table_tile(p, table, next, NT));
    };

    // ---- the multiplication ----
    // Lane half h of substep q (16 n) takes weight rows 16 q + 8 h .. + 8 of the stage, two
    // neighbouring columns (a byte) of each: MFMA c's operand row i is column 2 i + c.  One
    // transposing read brings the eight rows' bytes: 16 lanes read 8 rows x 16 bytes, lane i
    // of them gets byte column i.  Substep q + 1 is read from LDS before the MFMAs of substep
    // q and decoded between them.
    f32x16_t acc[2][4];
    u32x4_t op[2][2], dv[2][4];                          // operands by parity of the substep
    i32x2_t code;                                        // the next substep's codes and scales
    u32x4_t sc[2];
    const int erow = (lane & 15) >> 1;                   // of the eight rows, and where in it
    const int coded = erow * 128 + (((2 * wk + ((lane >> 4) & 1)) ^ erow) << 4) + (lane & 1) * 8;
    auto read = [&](int sl, int q, auto f_c) {
        constexpr int f = decltype(f_c)::value;
        const uint8_t* D = smem + sl * kGSlot;
        const uint8_t* C = D + kGDout + (16 * q + 8 * h) * 128 + coded;
        const uint8_t* S = D + kGDout + kGCodes + (2 * q + h) * 256 + (wk * 2 + (r32 >> 4)) * 32;
        code = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)C);
#pragma unroll
        for (int i = 0; i < 2; ++i) sc[i] = *reinterpret_cast<const u32x4_t*>(S + 16 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dv[f][i] = *reinterpret_cast<const u32x4_t*>(D + swz8(wt * 128 + i * 32 + r32, 2 * q + h));
    };
    auto decode = [&](auto j_c, auto f_c) {              // weight rows j and j + 1 of the eight
        constexpr int j = decltype(j_c)::value, f = decltype(f_c)::value;
        const float s0 = __uint_as_float(sc[j / 4][j & 3] << 23);
        const float s1 = __uint_as_float(sc[j / 4][(j & 3) + 1] << 23);
        const uint32_t a =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)code[j / 4], s0, j & 3));
        const uint32_t b = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)code[j / 4], s1, (j & 3) + 1));
        op[f][0][j / 2] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        op[f][1][j / 2] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    };
    const std::integral_constant<int, 0> c0;
    const std::integral_constant<int, 1> c1;
    const std::integral_constant<int, 2> c2;
    const std::integral_constant<int, 4> c4;
    const std::integral_constant<int, 6> c6;
    // MFMAs of parity f, the other parity's decoding between them; FULL: four row blocks
    auto mfmas = [&](auto full_c, int nv, auto f_c, auto g_c) {
        constexpr bool FULL = decltype(full_c)::value;
        constexpr int f = decltype(f_c)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (FULL || i < nv) {
#pragma unroll
                for (int c = 0; c < 2; ++c) acc[c][i] = mfma_bf16_32(op[f][c], dv[f][i], acc[c][i]);
            }
            keep_order();
            if (i == 1) decode(c0, g_c);
            if (i == 2) decode(c2, g_c);
            if (i == 3) decode(c4, g_c);
            if (i == 3) decode(c6, g_c);
            keep_order();
        }
    };
    // The barrier stands before a stage's last MFMAs: its slot has been read (free for the
    // stage three on), and the wait has left only the last step's loads in flight.
    int slot = 0;
    auto stages = [&](auto full_c, int nv) {             // nv: 32-row blocks of this wave with rows
        for (int s = 0; s < nn; ++s) {
            const int following = slot == 2 ? 0 : slot + 1;
            read(slot, 1, c1);
            keep_order();
            mfmas(full_c, nv, c0, c1);
            read(slot, 2, c0);
            keep_order();
            mfmas(full_c, nv, c1, c0);
            read(slot, 3, c1);
            keep_order();
            mfmas(full_c, nv, c0, c1);
            // (a workgroup's last stages issue nothing: then every load is waited for)
            if (!more) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else if (VECTOR) asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(2) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (more) {
                issue(is, slot);
                advance();
            }
            read(following, 0, c0);
            keep_order();
            mfmas(full_c, nv, c1, c0);
            slot = following;
        }
    };
    load_from(t);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        if (!more) continue;
        issue(is, s);
        advance();
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    read(0, 0, c0);
    decode(c0, c0);
    decode(c2, c0);
    decode(c4, c0);
    decode(c6, c0);
    for (;;) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[c][i][v] = 0.f;
        const bool cols = t.nt * kTN + wk * 64 < p.K;
        const int nvi = cols ? max(0, min(4, (t.re - t.rb - wt * 128 + 31) >> 5)) : 0;
        if (nvi == 4) stages(std::true_type{}, 4);
        else stages(std::false_type{}, nvi);
        // values v, v + 1 of both operands are four consecutive columns: 64 columns by 32
        // rows as two staged blocks of 32
        uint8_t* stage = smem + kGOffStage + wave * kWaveStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= nvi) break;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // operand rows 16 b .. + 16 (values 8 b .. + 8): columns 32 b .. + 32
                f32x16_t o;
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    o[2 * v] = acc[0][i][8 * b + v];
                    o[2 * v + 1] = acc[1][i][8 * b + v];
                }
                wave_store<true>(p, stage, t, wt * 128 + i * 32, wk * 64 + b * 32, p.K, o);
            }
        }
        mine += stride;
        if (mine >= end) break;
        t = table_tile(p, table, mine, NT);
    }
}

template <auto Kern, int LDS>
static hipError_t launch_tiles(const ProductArgs& p, int64_t grid, hipStream_t s) {
    const hipError_t e = allow_dynamic_lds<Kern>(LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(Kern, dim3((unsigned)grid), dim3(kTThreads), LDS, s, p);
    return hipGetLastError();
}

hipError_t launch_product_tiles(const ProductArgs& p, int cus, hipStream_t s) {
    const bool aligned =
        p.K % 128 == 0 && ((reinterpret_cast<uintptr_t>(p.w_s) | reinterpret_cast<uintptr_t>(p.a_s)) & 3) == 0;
    const int64_t tiles = tile_grid(p, (p.N + kTN - 1) / kTN);
    // one workgroup a CU, each for several tiles, or (tiles: a multiple of 8) one a tile
    const int64_t one_each = min(tiles, (int64_t)max(cus / 8 * 8, 8));
    if (p.a_s)
        return aligned ? launch_tiles<mx_tile_kernel<true>, mx_lds(true)>(p, one_each, s)
                       : launch_tiles<mx_tile_kernel<false>, mx_lds(false)>(p, tiles, s);
    return aligned ? launch_tiles<a16_tile_kernel<true>, a16_lds(true)>(p, tiles, s)
                   : launch_tiles<a16_tile_kernel<false>, a16_lds(false)>(p, tiles, s);
}

hipError_t launch_product_grad_tiles(const ProductArgs& p, int cus, hipStream_t s) {
    const int64_t grid = min(tile_grid(p, (p.K + kTN - 1) / kTN), (int64_t)max(cus / 8 * 8, 8));
    return dout_vector(p) ? launch_tiles<grad_tile_kernel<true>, kGLds>(p, grid, s)
                          : launch_tiles<grad_tile_kernel<false>, kGLds>(p, grid, s);
}

}  // namespace moe
