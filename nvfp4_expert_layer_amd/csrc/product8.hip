// Products of MXFP8 rows with MXFP4 weights (W4A8) in tiles, for more rows a group than are worth
// streaming for (gfx950).  A tile is 256 rows of one group x 256 outputs; eight waves of 64 rows x 128 outputs, one
// workgroup a CU; the operands come straight from global memory to LDS.
//
//   32x32x64 scaled MFMAs take both formats as they lie in memory (half the rate of FP4 x FP4,
//   twice bf16's).  The rows' ring holds two stages of 128 k, the weight's two of 256 k: a full
//   128-byte line of a row each.  The matrix cores need 2 x 512 cycles a SIMD and stage; LDS
//   gives 128 KB a stage to the waves, which the 64 x 128 wave tiles keep under their time
//   (128 x 64: 160 KB).
//
// The unit adds the products of eight neighbouring k aligned to the largest, without the bits
// below 2^-13 of it (checked on the device: rows spread over E4M3's whole range lose up to
// 2^-11 of their largest product); everything beyond is fp32.
#include "product_tiles_common.h"

namespace moe {

constexpr int k8Part = 256 * 128;                          // a slot: 128 k of the rows, 256 k of the weight
constexpr int k8OffW = 2 * k8Part, k8OffS = 4 * k8Part;    // rows [2] | weight [2] | scales [2] | ...
// Scales of both operands, 16 bytes a row: of 512 k, or (rows of scales that are not aligned to
// dwords) of 256 k, the aligned dwords that hold them.
constexpr int k8Scales = scale_bytes(true, 16);
// ... | waves' staging [8] | table
constexpr int k8OffStage = k8OffS + 4 * k8Scales, k8OffTable = k8OffStage + kTWaves * kWaveStage / 2;
constexpr int k8Lds = k8OffTable + kTable;

template <int OPSEL>
__device__ __forceinline__ f32x16_t mfma_w4a8_32(const u32x4_t& w, uint32_t ws, const u32x4_t& lo, const u32x4_t& hi,
                                                 uint32_t as, const f32x16_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(w), mx8_operand(lo, hi), c, 4, 0, OPSEL, (int)ws,
                                                           OPSEL, (int)as);
}

// Tile `logical` of this kernel: within a group, bands of eight column blocks, row tile by row
// tile, so that the 32 workgroups of an XCD meet on about four row tiles and eight column blocks:
// per k, 4 x 256 bytes of rows and 8 x 128 of weight feed 32 tiles (one row tile and 32 column
// blocks: 256 and 4096).  16384 x 8192 x 8192: 924 -> 866 us.
__device__ __forceinline__ Tile band_tile(const ProductArgs& p, const int* table, int logical, int NT) {
    Tile t = table_tile(p, table, logical, NT);
    if (NT <= 8) return t;
    const int first = __builtin_amdgcn_readfirstlane(table[t.g]), tiles = __builtin_amdgcn_readfirstlane(table[t.g + 1]) - first;
    const int at = logical - first * NT, band = at / (tiles * 8), rest = at - band * tiles * 8;
    const int width = min(8, NT - 8 * band), row = rest / width;
    int rb, re;
    group_rows(p, t.g, rb, re);
    rb += row * kTM;
    return Tile{t.g, __builtin_amdgcn_readfirstlane(rb), __builtin_amdgcn_readfirstlane(min(rb + kTM, re)),
                8 * band + rest - row * width};
}

// A workgroup takes tiles one after another: while a tile's last stages are multiplied the next
// tile's first ones are loaded, and its outputs leave while those land.
// ALIGNED: scale rows can be read in dwords (K % 128 == 0, 4-byte aligned scales), two chunks at a
// time.  Otherwise each chunk's eight bytes come with the dwords that hold them and are shifted
// into place (12004 rows over 24 experts of 1000 x 2080: 47 us byte by byte, 41 so).
template <bool ALIGNED>
__global__ __launch_bounds__(kTThreads) void w4a8_tile_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int wm = wave >> 1, wn = wave & 1;             // rows 64 wm .. +64, outputs 128 wn .. +128
    const int NT = (p.N + kTN - 1) / kTN, KB = p.K / 32, nc = (KB + 7) / 8, r32 = lane & 31;

    // This workgroup's tiles: workgroup b runs on XCD b % 8, each XCD takes a contiguous range.
    int* table = reinterpret_cast<int*>(smem + k8OffTable);
    const int all = tile_table(p, table) * NT, per = (all + 7) >> 3, stride = gridDim.x >> 3;
    const int end = min(((int)blockIdx.x & 7) * per + per, all);
    int mine = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (mine >= end) return;
    Tile t = band_tile(p, table, mine, NT);

    // ---- loads: rows one chunk (256 k) ahead of the multiplication, half a chunk a slot; the
    // weight and both operands' scales two chunks ahead.  Load q of wave w fills rows 8 (4 w + q)
    // .. +8 of a slot (a full 128-byte line each), lane i row i / 8, slot i % 8, which holds unit
    // (i & 7) ^ (i >> 3) ^ (q & 1) (swz8).  Scales: waves 0-3 the weight's rows 64 w .. +64, waves
    // 4-7 the rows'.  Rows and outputs past the tile's end: any valid row (their results are not
    // stored), but whole blocks of 32 rows are left out, as their multiplications are (320 experts
    // of 2048 x 4096, 48 rows each: 464 -> 445 us).
    // (Lane offsets are formed at each load: kept, they would not leave the registers for the
    // accumulators and operands.)
    const uint8_t *abase, *wbase, *sbase;
    int amax, wmax, smax;                                // last rows of the operands' parts
    const int cu = (lane & 7) ^ (lane >> 3), lrow = wave * 32 + (lane >> 3), srow = (wave & 3) * 64;
    const int sdst = k8OffS + (wave < 4 ? 0 : k8Scales);
    Tile wt;                                             // the tile of the next weight loads
    uint32_t wshift = 0, ashift = 0;                     // !ALIGNED: the lane's scale rows' first byte in a dword
    auto scales_from = [&](const Tile& n) {
        if (ALIGNED) return;
        const uintptr_t w = reinterpret_cast<uintptr_t>(p.w_s) + ((int64_t)n.g * p.N + n.nt * kTN) * KB;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p.a_s) + (int64_t)n.rb * KB;
        wshift = ((uint32_t)w + r32 * KB) & 3;
        ashift = ((uint32_t)a + r32 * KB) & 3;
    };
    auto rows_from = [&](const Tile& n) {
        abase = static_cast<const uint8_t*>(p.a) + (int64_t)n.rb * p.K;
        amax = n.re - 1 - n.rb;
        scales_from(n);                                  // (the rows' loads are one chunk ahead, as are the scales read)
    };
    auto weight_from = [&](const Tile& n) {
        wt = n;
        const int n0 = n.nt * kTN;
        const int64_t w0 = (int64_t)n.g * p.N + n0;
        wbase = p.w + w0 * (p.K / 2);
        wmax = p.N - 1 - n0;
        sbase = wave < 4 ? p.w_s + w0 * KB : p.a_s + (int64_t)n.rb * KB;
        smax = wave < 4 ? wmax : n.re - 1 - n.rb;
    };
    // the wave's part q of the rows' next half chunk (k 128 s ..)
    auto issue_rows = [&](int s, int q) {
        if (wave * 32 > amax) return;                    // (the waits count the weight loads alone)
        const uint32_t off = min(lrow + 8 * q, amax) * (uint32_t)p.K + (cu ^ (q & 1)) * 16;
        const uint8_t* ab = abase + (int64_t)s * 128;
        uint8_t* ad = smem + (s & 1) * k8Part + (wave * 4 + q) * 1024;
        if (s * 4 + 4 <= KB) load_lds<16>(ab, off, ad);
        else load_lds<16>(within(s * 128 + (cu ^ (q & 1)) * 16 < p.K, ab + off), ad);
    };
    auto issue_weight = [&](int c, int slot, int q) {
        const uint32_t off = min(lrow + 8 * q, wmax) * (uint32_t)(p.K / 2) + (cu ^ (q & 1)) * 16;
        const uint8_t* wb = wbase + (int64_t)c * 128;
        uint8_t* wd = smem + k8OffW + slot * k8Part + (wave * 4 + q) * 1024;
        if (c * 8 + 8 <= KB) load_lds<16>(wb, off, wd);
        else load_lds<16>(within(c * 8 + (cu ^ (q & 1)) < KB, wb + off), wd);
    };
    int spair = 0;                                       // slot of the next scales
    auto issue_scales = [&](int c) {                     // ALIGNED: at even chunks this one's and the next's
        if (ALIGNED && (c & 1)) return;
        const uint32_t mis = ALIGNED ? 0 : (uint32_t)reinterpret_cast<uintptr_t>(sbase) & 3;
        const uint8_t* sb = sbase - mis + (int64_t)c * 8;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (wave >= 4 && srow > smax) break;
            const uint32_t row = min(srow + q * 16 + (lane >> 2), smax) * (uint32_t)KB + mis;
            const uint32_t off = (row & ~3u) + (lane & 3) * 4;
            uint8_t* sd = smem + spair * 2 * k8Scales + sdst + srow * 16 + q * 256;
            if (!ALIGNED) load_lds<4>(within(c * 8 + off < (smax + 1) * (uint32_t)KB + mis, sb + off), sd);
            else if (c * 8 + 16 <= KB) load_lds<4>(sb, off, sd);
            else load_lds<4>(within(c * 8 + (lane & 3) * 4 < KB, sb + off), sd);
        }
        spair ^= 1;
    };
    // positions of the next loads: the rows' half chunk, the weight's chunk and its slot
    int rs = 0, rnext = mine, wc = 0, wslot = 0, wnext = mine;
    bool rmore = true, wmore = true;
    auto advance_rows = [&]() {
        if (++rs < 2 * nc) return;
        rs = 0;
        rnext += stride;
        rmore = rnext < end;
        if (rmore) rows_from(wt);                        // the weight's loads have just come to this tile
    };
    auto advance_weight = [&]() {
        wslot ^= 1;
        if (++wc < nc) return;
        wc = 0;
        wnext += stride;
        wmore = wnext < end;
        if (wmore) weight_from(band_tile(p, table, wnext, NT));
    };

    // ---- the multiplication: a half chunk is two groups of 64 k ----
    f32x16_t acc[4][2];
    u32x4_t wv[4], av[2][2][2];                          // operands; the rows' by parity of the group
    uint32_t ws[4], as[2], wsn[4], asn[2];               // a chunk's scales, four groups'; the next chunk's
    // of group m of half chunk `half`, the chunk's weight in `slot`
    auto weights = [&](int half, int slot, int m, int j) {
        wv[j] = *reinterpret_cast<const u32x4_t*>(smem + k8OffW + slot * k8Part +
                                                  swz8(wn * 128 + j * 32 + r32, 4 * half + 2 * m + h));
    };
    auto tokens = [&](int half, auto m_c) {
        constexpr int m = decltype(m_c)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                av[m][i][q] = *reinterpret_cast<const u32x4_t*>(
                    smem + half * k8Part + swz8(wm * 64 + i * 32 + r32, 4 * m + 2 * q + h));
    };
    // blocks h, 2 + h, 4 + h, 6 + h of row r's eight
    auto row_scales = [&](const uint8_t* S, int r, uint32_t shift, int left) {
        const uint32_t pick = h ? 0x07050301u : 0x06040200u;
        if (ALIGNED) {
            const u32x2_t v = *reinterpret_cast<const u32x2_t*>(S + r * 16);
            return __builtin_amdgcn_perm(v.y, v.x, pick);
        }
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(S + r * 16);
        uint32_t lo = __builtin_amdgcn_alignbyte(v.y, v.x, shift), hi = __builtin_amdgcn_alignbyte(v.z, v.y, shift);
        if (left < 8) {                                  // past K come another row's: its NaN times a 0 would stay
            lo &= left >= 4 ? ~0u : (1u << (8 * left)) - 1;
            hi &= left <= 4 ? 0u : (1u << (8 * (left - 4))) - 1;
        }
        return __builtin_amdgcn_perm(hi, lo, pick);
    };
    int rpair = 1;                                       // slot of the scales being read
    auto scales = [&](int c, int j) {                    // of chunk c of its tile: part j of 4
        if (j == 0 && (!ALIGNED || !(c & 1))) rpair ^= 1;
        const uint8_t* S = smem + k8OffS + rpair * 2 * k8Scales + (ALIGNED ? (c & 1) * 8 : 0);
        const int left = KB - c * 8;
        wsn[j] = row_scales(S, wn * 128 + j * 32 + r32, wshift, left);
        if (j < 2) asn[j] = row_scales(S + k8Scales, wm * 64 + j * 32 + r32, ashift, left);
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) ws[j] = wsn[j];
#pragma unroll
        for (int i = 0; i < 2; ++i) as[i] = asn[i];
    };
    auto mfmas = [&](auto half_c, auto m_c, int j, int nv) {
        constexpr int half = decltype(half_c)::value, m = decltype(m_c)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i < nv)
                acc[j][i] = mfma_w4a8_32<2 * half + m>(wv[j], ws[j], av[m][i][0], av[m][i][1], as[i], acc[j][i]);
    };

    // A tile's chunks.  A group's tokens are read before the MFMAs of the group before it, each
    // weight operand after the last MFMA on the one before it, three operands ahead of its own
    // MFMAs, so that the matrix cores do not wait for LDS.  The barrier stands before a half
    // chunk's last MFMAs, where its slot has been read and the half chunk after the next may take
    // it.  Loads return in order: at a chunk's middle the rows' next half must have landed and the
    // weight loads issued after them (always the last four) may be under way; at its end everything.
    constexpr std::integral_constant<int, 0> c0{};
    constexpr std::integral_constant<int, 1> c1{};
    int slot = 0;
    bool wflight = false;                                // weight loads were issued last
    auto stages = [&](int nv) {                          // nv: 32-row blocks of this wave with rows
        for (int c = 0; c < nc; ++c) {
            tokens(0, c1);
            keep_order();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mfmas(c0, c0, j, nv);
                weights(0, slot, 1, j);
                keep_order();
            }
            if (wflight) asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            tokens(1, c0);
            keep_order();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mfmas(c0, c1, j, nv);
                weights(1, slot, 0, j);
                keep_order();
                if (rmore) issue_rows(rs, j);
                keep_order();
            }
            if (rmore) advance_rows();

            tokens(1, c1);
            keep_order();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mfmas(c1, c0, j, nv);
                weights(1, slot, 1, j);
                keep_order();
            }
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            tokens(0, c0);
            keep_order();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mfmas(c1, c1, j, nv);
                weights(0, slot ^ 1, 0, j);
                scales(c + 1 < nc ? c + 1 : 0, j);
                keep_order();
                if (rmore) issue_rows(rs, j);
                keep_order();
            }
            wflight = wmore;
            if (wmore) {
                issue_scales(wc);
#pragma unroll
                for (int q = 0; q < 4; ++q) issue_weight(wc, wslot, q);
            }
            if (rmore) advance_rows();
            if (wmore) advance_weight();
            take_scales();
            slot ^= 1;
        }
    };

    rows_from(t);
    weight_from(t);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (rmore) {
#pragma unroll
            for (int q = 0; q < 4; ++q) issue_rows(rs, q);
            advance_rows();
        }
        if (wmore) {
            issue_scales(wc);
#pragma unroll
            for (int q = 0; q < 4; ++q) issue_weight(wc, wslot, q);
            advance_weight();
        }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    tokens(0, c0);
    const uint32_t wlater = wshift, alater = ashift;     // (a tile of one chunk: the rows' loads have come to the next)
    scales_from(t);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        weights(0, 0, 0, j);
        scales(0, j);
    }
    take_scales();
    wshift = wlater;
    ashift = alater;
    for (;;) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
        const bool cols = t.nt * kTN + wn * 128 < p.N;
        const int nvi = cols ? max(0, min(2, (t.re - t.rb - wm * 64 + 31) >> 5)) : 0;    // 32-row blocks with rows
        stages(nvi);
        uint8_t* stage = smem + k8OffStage + wave * kWaveStage / 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= nvi) break;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wave_store_halves(p, stage, t, wm * 64 + i * 32, wn * 128 + j * 32, p.N, acc[j][i]);
        }
        mine += stride;
        if (mine >= end) break;
        t = band_tile(p, table, mine, NT);
    }
}

// ---------------------------------------------------------------------------
// Short tiles: 64 rows x 256 outputs, for groups of some dozens of rows, where the weight's bytes
// are the cost and what counts is how many of them are under way: three stages of 256 k, of which
// two load while one is multiplied (the tiles above have one under way on average).  A wave takes
// 32 outputs and all rows.  Scale rows that can be read in dwords only (as ALIGNED above).  24 / 48
// rows a group over 320 experts of 2048 x 4096: 282 / 345 us, 5.3 / 4.6 TB/s (a large copy: 4.95).
// ---------------------------------------------------------------------------
constexpr int kSM = 64;
// a stage: weight [256][128 bytes] | rows [2 halves][64][128 bytes] | weight scales [256][8] | rows' [64][8]
constexpr int kSRows = 256 * 128, kSWs = kSRows + 2 * kSM * 128, kSAs = kSWs + 256 * 8, kSStage = kSAs + kSM * 8;
constexpr int kSTable = 3 * kSStage, kSLds = kSTable + kTable;
constexpr int kSLoads = 8;                               // a wave's of a stage

__global__ __launch_bounds__(kTThreads) void w4a8_short_kernel(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, r32 = lane & 31, NT = (p.N + kTN - 1) / kTN, KB = p.K / 32, nc = (KB + 7) / 8;

    int* table = reinterpret_cast<int*>(smem + kSTable);
    const int all = tile_table<kSM>(p, table) * NT, per = (all + 7) >> 3, stride = gridDim.x >> 3;
    const int end = min(((int)blockIdx.x & 7) * per + per, all);
    int mine = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (mine >= end) return;

    // ---- loads: a stage at a time, two ahead of the multiplication, over the tiles' ends; lane i of
    // a 16-byte load fills row i / 8, slot i % 8 (swz8), of a scale load row i / 2, dword i % 2.
    // Rows and outputs past the tile's end: any valid row.
    const uint8_t *wbase, *abase, *wsbase, *asbase;
    int wmax, amax, lmine = mine, lc = 0, lslot = 0;
    bool more = true;
    auto load_from = [&](const Tile& n) {
        const int64_t w0 = (int64_t)n.g * p.N + n.nt * kTN;
        wbase = p.w + w0 * (p.K / 2);
        wsbase = p.w_s + w0 * KB;
        wmax = p.N - 1 - n.nt * kTN;
        abase = static_cast<const uint8_t*>(p.a) + (int64_t)n.rb * p.K;
        asbase = p.a_s + (int64_t)n.rb * KB;
        amax = n.re - 1 - n.rb;
    };
    auto load_stage = [&]() {
        uint8_t* d = smem + lslot * kSStage;
        const bool whole = lc * 8 + 8 <= KB;
        auto load = [&](auto bytes, const uint8_t* base, uint32_t off, bool in, uint8_t* dst) {
            constexpr int B = decltype(bytes)::value;
            if (whole) load_lds<B>(base, off, dst);
            else load_lds<B>(within(in, base + off), dst);
        };
        constexpr std::integral_constant<int, 16> b16{};
        constexpr std::integral_constant<int, 4> b4{};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int u = (lane & 7) ^ (lane >> 3) ^ (q & 1), r = wave * 32 + q * 8 + (lane >> 3);
            load(b16, wbase + (int64_t)lc * 128, min(r, wmax) * (uint32_t)(p.K / 2) + u * 16, lc * 8 + u < KB,
                 d + (wave * 4 + q) * 1024);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int half = wave >> 2, at = (wave & 3) * 2 + q;
            const int u = (lane & 7) ^ (lane >> 3) ^ (q & 1), r = at * 8 + (lane >> 3);
            load(b16, abase + (int64_t)lc * 256, min(r, amax) * (uint32_t)p.K + half * 128 + u * 16,
                 lc * 256 + half * 128 + u * 16 < p.K, d + kSRows + (half * 8 + at) * 1024);
        }
        const int dw = (lane & 1) * 4, half = wave & 1;      // (of the rows' scales four waves load the same)
        load(b4, wsbase + lc * 8, min(wave * 32 + (lane >> 1), wmax) * (uint32_t)KB + dw, lc * 8 + dw < KB,
             d + kSWs + wave * 256);
        load(b4, asbase + lc * 8, min(half * 32 + (lane >> 1), amax) * (uint32_t)KB + dw, lc * 8 + dw < KB,
             d + kSAs + half * 256);
        lslot = lslot == 2 ? 0 : lslot + 1;
        if (++lc < nc) return;
        lc = 0;
        lmine += stride;
        more = lmine < end;
        if (more) load_from(table_tile<kSM>(p, table, lmine, NT));
    };

    Tile t = table_tile<kSM>(p, table, mine, NT);
    load_from(t);
    load_stage();
    bool ahead = more;                                   // the stage after the next to multiply is under way
    if (more) load_stage();
    int slot = 0;
    for (;;) {
        f32x16_t acc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][v] = 0.f;
        const bool cols = t.nt * kTN + wave * 32 < p.N;
        const int nv = cols ? (t.re - t.rb + 31) >> 5 : 0;   // 32-row blocks with rows
        for (int c = 0; c < nc; ++c) {
            // loads return in order: this stage's are here when at most the next one's are not
            if (ahead) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kSLoads) : "memory");
            else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            ahead = more;
            if (more) load_stage();                      // (into the slot that all have read before the barrier)
            const uint8_t* S = smem + slot * kSStage;
            slot = slot == 2 ? 0 : slot + 1;
            if (!nv) continue;
            const uint32_t pick = h ? 0x07050301u : 0x06040200u;      // blocks h, 2 + h, 4 + h, 6 + h
            auto scales = [&](const uint8_t* at) {
                const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at);
                return __builtin_amdgcn_perm(v.y, v.x, pick);
            };
            const uint32_t ws = scales(S + kSWs + (wave * 32 + r32) * 8);
            uint32_t as[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) as[i] = scales(S + kSAs + (i * 32 + r32) * 8);
            auto group = [&](auto m_c) {
                constexpr int m = decltype(m_c)::value;
                const u32x4_t w = *reinterpret_cast<const u32x4_t*>(S + swz8(wave * 32 + r32, 2 * m + h));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i >= nv) break;
                    u32x4_t a[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        a[q] = *reinterpret_cast<const u32x4_t*>(S + kSRows + (m >> 1) * kSM * 128 +
                                                                 swz8(i * 32 + r32, 4 * (m & 1) + 2 * q + h));
                    acc[i] = mfma_w4a8_32<m>(w, ws, a[0], a[1], as[i], acc[i]);
                }
            };
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            group(std::integral_constant<int, 2>{});
            group(std::integral_constant<int, 3>{});
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= nv) break;
            const int row = t.rb + i * 32 + r32, left = p.N - t.nt * kTN - wave * 32;
            const int64_t el = row * p.os + t.nt * kTN + wave * 32;
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                // the lane's values 4 g .. + 4 are outputs 8 g + 4 h .. + 4
                if (p.out_dtype == kF32) {
#pragma unroll
                    for (int x = g; x < g + 2; ++x)
                        if (row < t.re)
                            store4(p.out, kF32, el + 8 * x + 4 * h,
                                   f32x4_t{acc[i][4 * x], acc[i][4 * x + 1], acc[i][4 * x + 2], acc[i][4 * x + 3]},
                                   left - 8 * x - 4 * h);
                    continue;
                }
                // the halves of the wave trade: eight outputs a lane, 8 (g + h) .. + 8
                const u32x2_t lo = pack4(p.out_dtype, acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]);
                const u32x2_t hi = pack4(p.out_dtype, acc[i][4 * g + 4], acc[i][4 * g + 5], acc[i][4 * g + 6], acc[i][4 * g + 7]);
                const u32x2_t give = h ? lo : hi;
                const u32x2_t got = {(uint32_t)__shfl_xor((int)give.x, 32, 64), (uint32_t)__shfl_xor((int)give.y, 32, 64)};
                const u32x4_t v = h ? u32x4_t{got.x, got.y, hi.x, hi.y} : u32x4_t{lo.x, lo.y, got.x, got.y};
                if (row >= t.re) continue;
                const int col = 8 * (g + h);
                uint16_t* o = static_cast<uint16_t*>(p.out) + el + col;
                if (col + 8 <= left) {
                    *reinterpret_cast<u32x4_any_t*>(o) = v;
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (col + x < left) o[x] = (uint16_t)(v[x / 2] >> (16 * (x & 1)));
                }
            }
        }
        mine += stride;
        if (mine >= end) break;
        t = table_tile<kSM>(p, table, mine, NT);
    }
}

bool product8_dwords(const ProductArgs& p) {
    return p.K % 128 == 0 && ((reinterpret_cast<uintptr_t>(p.w_s) | reinterpret_cast<uintptr_t>(p.a_s)) & 3) == 0;
}

// Short tiles where the weight's bytes are the cost (up to 64 rows a group on average), and as long
// as they come to about two rounds of the card: one takes half a tall one's time.  Short / tall us:
// 320 experts of 2048 x 4096 345 / 444 at 48 rows a group, 420 / 455 at 64, 471 / 459 at 72; of 4096 x
// 1024 193 / 296 and 241 / 304; 16 experts 26 / 42 at 96, 48 / 51 at 192, 68 / 54 at 256; 24 of 1024 x
// 2048 28 / 31 at 256, 40 / 32 at 384; one product of 768 x 4096 x 4096 26 / 51, of 1280 47 / 52.
static bool short_tiles(const ProductArgs& p, int cus) {
    const int64_t NT = (p.N + kTN - 1) / kTN;
    return p.M <= (int64_t)p.G * 64 || (p.M / kSM + p.G / 2) * NT <= 2 * cus;
}

hipError_t launch_product8_tiles(const ProductArgs& p, int cus, hipStream_t s) {
    const bool dwords = product8_dwords(p);
    const int NT = (p.N + kTN - 1) / kTN;
    const int64_t most = max(cus / 8 * 8, 8);            // one workgroup a CU
    if (dwords && short_tiles(p, cus)) return launch_tiles<w4a8_short_kernel, kSLds>(p, min(tile_grid<kSM>(p, NT), most), s);
    const int64_t grid = min(tile_grid(p, NT), most);
    return dwords ? launch_tiles<w4a8_tile_kernel<true>, k8Lds>(p, grid, s)
                  : launch_tiles<w4a8_tile_kernel<false>, k8Lds>(p, grid, s);
}

}  // namespace moe

int moe_internal_product8_short(int M, int N, int K, int G, int cus) {
    moe::ProductArgs p{};
    p.M = M; p.N = N; p.K = K; p.G = G;
    return moe::product8_dwords(p) && moe::short_tiles(p, cus);
}
