// Dispatch and combine (gfx950): pairs sorted by local expert, token rows gathered
// in that order and weighted back, and the gradients of both.
//
// With pair p = t k + j, e_p its local expert and kept pairs ordered by (e_p, p):
//   inv_p     = #{kept q : e_q < e_p} + #{q < p : e_q = e_p}
//   rows[inv_p] = x_t                           dx_t = sum_j drows[inv_tj]
//   out_t     = sum_j w_tj rows[inv_tj]         drows[inv_tj] = w_tj dout_t
//                                               dw_tj = dout_t . rows[inv_tj]
// All of it moves bytes: a row element costs at most three operations, so every
// kernel reads or writes 16 bytes a lane and each row once.  Rows need no alignment and
// no particular width: a row's last unit ends with the row and overlaps the one before.
// The gather runs by token (a token's row is loaded once and stored to its k places),
// not by sorted row (which would load it k times).
//
// T=8192, k=8, d=4096 bf16, 320 experts (65536 rows, 537 MB): dispatch 116 us (5.2 TB/s of
// rows read and written; a large copy reaches 4.95), its gradient and the combine 109
// us, the combine's gradient 232 us (4.9 TB/s).  T=64: 5.0 us and 3.5 us of kernel.
#include "device_common.h"
#include "ops.h"
#include "rows.h"

namespace moe {

constexpr int kThreads = 256;
constexpr int kChunk = 256;                    // pairs per block at most
constexpr int kMaxExperts = 1024;

// Row of pair value r (an entry of inv), or -1.
__device__ __forceinline__ int valid_row(int r, int pairs) { return (uint32_t)r < (uint32_t)pairs ? r : -1; }

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
// Exclusive scan over n <= 1024 values in LDS by 256 threads (4 each); returns the
// total.  part: 4 words of scratch.
__device__ __forceinline__ int block_scan(int* v, int n, int* part) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int x[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = 4 * tid + i < n ? v[4 * tid + i] : 0;
        sum += x[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(inc, o, 64);
        if (lane >= o) inc += y;
    }
    if (lane == 63) part[wave] = inc;
    __syncthreads();
    int at = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wave) at += part[w];
        total += part[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * tid + i < n) v[4 * tid + i] = at;
        at += x[i];
    }
    __syncthreads();
    return total;
}

__device__ __forceinline__ int local_expert(const DispatchArgs& a, int p) {
    // 64-bit: an id outside the model must not wrap into the shard
    const int64_t e = (int64_t)a.ids[p] - a.offset;
    return e >= 0 && e < a.L ? (int)e : -1;
}

// One block takes the pairs of tpb tokens (at most kChunk pairs): their places,
// then their rows' copies in units U (a row: `bytes` bytes; strides in bytes).  grid.y
// splits the columns.
//
// COUNTED = false (one launch): the block counts all T k ids by itself, those
// before its own pairs and the rest apart, in LDS; integer counts do not depend
// on the order of the atomics.  COUNTED = true: the two kernels below have left
// the counts per block in the workspace.
template <typename U, bool COUNTED>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(DispatchArgs a, int tpb, int blocks, int units, int bytes,
                                                            int64_t xs, int64_t rs) {
    __shared__ int before[kMaxExperts], base[kMaxExperts], lid[kChunk], dest[kChunk], part[4];
    const int tid = threadIdx.x, L = a.L;
    const int t0 = blockIdx.x * tpb, nt = min(tpb, a.T - t0);
    const int p0 = t0 * a.k, np = nt * a.k;

    if (COUNTED) {
        for (int e = tid; e < L; e += kThreads) base[e] = a.totals[e];
    } else {
        for (int e = tid; e < L; e += kThreads) before[e] = base[e] = 0;
        __syncthreads();
        const int n = a.T * a.k;
        for (int q0 = tid; q0 < n; q0 += 8 * kThreads) {    // eight loads in flight
            int e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = q0 + i * kThreads < n ? local_expert(a, q0 + i * kThreads) : -1;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e[i] >= 0) atomicAdd(q0 + i * kThreads < p0 ? &before[e[i]] : &base[e[i]], 1);
        }
    }
    int mine = -1;
    if (tid < np) mine = lid[tid] = local_expert(a, p0 + tid);
    __syncthreads();
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;
    if (!COUNTED)
        for (int e = tid; e < L; e += kThreads) base[e] += before[e];
    if (!COUNTED) __syncthreads();
    if (first && a.counts)
        for (int e = tid; e < L; e += kThreads) a.counts[e] = base[e];
    if (first) __syncthreads();
    const int total = block_scan(base, L, part);
    if (first && a.offsets) {
        for (int e = tid; e < L; e += kThreads) a.offsets[e] = base[e];
        if (tid == 0) a.offsets[L] = total;
    }
    if (tid < np) {
        int at = -1;
        if (mine >= 0) {
            at = base[mine] + (COUNTED ? a.block_counts[(size_t)mine * blocks + blockIdx.x] : before[mine]);
            for (int q = 0; q < tid; ++q) at += lid[q] == mine ? 1 : 0;
            if (blockIdx.y == 0 && a.perm) a.perm[at] = p0 + tid;
        }
        dest[tid] = at;
        if (blockIdx.y == 0 && a.inv) a.inv[p0 + tid] = at;
    }
    if (!a.x) return;
    __syncthreads();

    const char* x = static_cast<const char*>(a.x);
    char* rows = static_cast<char*>(a.rows);
    const int per = (units + gridDim.y - 1) / gridDim.y, u0 = blockIdx.y * per, nu = min(per, units - u0);
    if (nu <= 0) return;
    for (int i = tid; i < nt * nu; i += kThreads) {
        const int t = i / nu, c = min((u0 + (i - t * nu)) * (int)sizeof(U), bytes - (int)sizeof(U));
        const U v = *reinterpret_cast<const U*>(x + (t0 + t) * xs + c);
        for (int j = 0; j < a.k; ++j) {
            const int r = dest[t * a.k + j];
            if (r >= 0) __builtin_nontemporal_store(v, reinterpret_cast<U*>(rows + r * rs + c));
        }
    }
}

// Large batches, first: kept pairs per (expert, block).
__global__ __launch_bounds__(kThreads) void dispatch_count_kernel(DispatchArgs a, int tpb, int blocks) {
    __shared__ int hist[kMaxExperts];
    const int tid = threadIdx.x;
    for (int e = tid; e < a.L; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * tpb, np = min(tpb, a.T - t0) * a.k;
    if (tid < np) {
        const int e = local_expert(a, t0 * a.k + tid);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = tid; e < a.L; e += kThreads) a.block_counts[(size_t)e * blocks + blockIdx.x] = hist[e];
}

// Second: per expert (a workgroup each), an exclusive scan over the blocks and the total.
__global__ __launch_bounds__(kThreads) void dispatch_scan_kernel(DispatchArgs a, int blocks) {
    __shared__ int v[kMaxExperts], part[4];
    int32_t* c = a.block_counts + (size_t)blockIdx.x * blocks;
    int sum = 0;
    for (int b0 = 0; b0 < blocks; b0 += kMaxExperts) {
        const int n = min(blocks - b0, kMaxExperts);
        for (int i = threadIdx.x; i < n; i += kThreads) v[i] = c[b0 + i];
        __syncthreads();
        const int total = block_scan(v, n, part);
        for (int i = threadIdx.x; i < n; i += kThreads) c[b0 + i] = sum + v[i];
        __syncthreads();
        sum += total;
    }
    if (threadIdx.x == 0) a.totals[blockIdx.x] = sum;
}

// Up to this many pairs each block counts them all by itself.  One launch against three:
// T=1024, k=4, d=512 7 against 20 us; T=2048, k=8 (the bound) 17 against 20 us at d=512,
// 39 against 36 us at d=4096.
constexpr int kOneLaunchPairs = 16384;

DispatchPlan dispatch_plan(int T, int k) {
    DispatchPlan p;
    p.one_launch = (int64_t)T * k <= kOneLaunchPairs;
    // one launch: one token a block until there are blocks enough to fill the card; else
    // a block a CU before blocks take whole chunks, for each leaves a count per expert
    const int most = kChunk / k, few = T / (p.one_launch ? 1024 : 256);
    p.tokens_per_block = few < 1 ? 1 : (few > most ? most : few);
    p.blocks = (T + p.tokens_per_block - 1) / p.tokens_per_block;
    return p;
}

template <typename U>
static void dispatch_units(const DispatchArgs& a, const DispatchPlan& p, hipStream_t s) {
    const int eb = dtype_bytes(a.dtype), bytes = a.d * eb;
    const int units = a.x ? (bytes + (int)sizeof(U) - 1) / (int)sizeof(U) : 0;
    // few blocks: the columns over several too, at least 64 units each
    const int want = p.one_launch ? 256 : 512, most = (units + 63) / 64;
    int split = want / p.blocks;
    split = split > most ? most : split;
    if (split < 1) split = 1;
    const dim3 grid(p.blocks, split);
    if (p.one_launch) {
        hipLaunchKernelGGL((dispatch_kernel<U, false>), grid, dim3(kThreads), 0, s, a, p.tokens_per_block, p.blocks,
                           units, bytes, a.xs * eb, a.rs * eb);
        return;
    }
    hipLaunchKernelGGL(dispatch_count_kernel, dim3(p.blocks), dim3(kThreads), 0, s, a, p.tokens_per_block, p.blocks);
    hipLaunchKernelGGL(dispatch_scan_kernel, dim3(a.L), dim3(kThreads), 0, s, a, p.blocks);
    hipLaunchKernelGGL((dispatch_kernel<U, true>), grid, dim3(kThreads), 0, s, a, p.tokens_per_block, p.blocks, units,
                       bytes, a.xs * eb, a.rs * eb);
}

// Blocks of a grid-stride launch: a grid holds fewer than 2^32 threads.
static unsigned grid_blocks(int64_t n) { return (unsigned)(n < (1 << 22) ? n : (1 << 22)); }

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s) {
    const DispatchPlan p = dispatch_plan(a.T, a.k);
    if (a.d * dtype_bytes(a.dtype) >= 16) dispatch_units<u32x4_any_t>(a, p, s);
    else dispatch_units<uint8_t>(a, p, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// combine and the dispatch's gradient: one thread per vector of a token's output,
// the slots eight at a time (row numbers and weights, then the rows, so a group
// costs two memory round trips), summed in slot order in fp32.
// ---------------------------------------------------------------------------
template <int DT, bool VECTOR, bool WEIGHTED>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(CombineRowsArgs a, int units) {
    typedef Row<DT, VECTOR> R;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)a.T * units;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int t = (int)(i / units), c0 = R::unit_start((int)(i - (int64_t)t * units), a.d), pairs = a.T * a.k;
        float acc[R::VEC];
#pragma unroll
        for (int e = 0; e < R::VEC; ++e) acc[e] = 0.f;
        for (int j0 = 0; j0 < a.k; j0 += 8) {
            int row[8];
            float w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int64_t at = (int64_t)t * a.k + j0 + q;
                row[q] = j0 + q < a.k ? valid_row(a.inv[at], pairs) : -1;
                if (WEIGHTED) w[q] = j0 + q < a.k ? a.w[at] : 0.f;
            }
            typename R::Raw y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (row[q] >= 0) y[q] = R::load(a.rows, row[q] * a.rs + c0);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (row[q] < 0) continue;
#pragma unroll
                for (int e = 0; e < R::VEC; ++e)
                    acc[e] = WEIGHTED ? fmaf(w[q], R::get(y[q], e), acc[e]) : acc[e] + R::get(y[q], e);
            }
        }
        R::store(a.out, t * a.os + c0, acc);
    }
}

template <int DT, bool VECTOR>
static void combine_rows(const CombineRowsArgs& a, hipStream_t s) {
    const int units = Row<DT, VECTOR>::units(a.d);
    const int64_t n = (int64_t)a.T * units;
    // few outputs: one wave a block, so that they spread over the CUs
    const int threads = n <= 64 * 256 ? 64 : kThreads;
    const dim3 grid(grid_blocks((n + threads - 1) / threads));
    if (a.w)
        hipLaunchKernelGGL((combine_rows_kernel<DT, VECTOR, true>), grid, dim3(threads), 0, s, a, units);
    else
        hipLaunchKernelGGL((combine_rows_kernel<DT, VECTOR, false>), grid, dim3(threads), 0, s, a, units);
}

hipError_t launch_combine_rows(const CombineRowsArgs& a, hipStream_t s) {
    const bool v = a.d * dtype_bytes(a.dtype) >= 16;
    if (a.dtype == kBF16) v ? combine_rows<kBF16, true>(a, s) : combine_rows<kBF16, false>(a, s);
    else if (a.dtype == kF16) v ? combine_rows<kF16, true>(a, s) : combine_rows<kF16, false>(a, s);
    else v ? combine_rows<kF32, true>(a, s) : combine_rows<kF32, false>(a, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// combine's gradient: WAVES waves per token walk its columns; dout's vector is
// loaded once for eight slots, each slot's row once for its dot product, each
// gradient row stored once.  The eight partial dots stay in registers and are
// summed over the lanes (and waves) in a fixed order at the end.
// ---------------------------------------------------------------------------
template <int DT, bool VECTOR, int WAVES>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGradArgs a, int units) {
    typedef Row<DT, VECTOR> R;
    constexpr int TOKENS = kThreads / 64 / WAVES;
    __shared__ float red[kThreads / 64][8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wt = wave % WAVES, pairs = a.T * a.k;
    const bool tail = a.d % R::VEC != 0;                        // a row's last unit overlaps the one before
    // tokens TOKENS * gridDim.x apart; with four waves a token, a block's waves share t
    for (int64_t t = (int64_t)blockIdx.x * TOKENS + wave / WAVES; t < a.T; t += (int64_t)gridDim.x * TOKENS)
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        int row[8];
        float w[8], dot[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t at = t * a.k + j0 + q;
            row[q] = j0 + q < a.k ? valid_row(a.inv[at], pairs) : -1;
            w[q] = j0 + q < a.k ? a.w[at] : 0.f;
            dot[q] = 0.f;
        }
        for (int u = wt * 64 + lane; u < units; u += 64 * WAVES) {
            const int c0 = R::unit_start(u, a.d), old = u * R::VEC - c0;   // elements of the unit before
            const typename R::Raw g = R::load(a.dout, t * a.dos + c0);
            typename R::Raw y[8];
            if (a.dw) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (row[q] >= 0) y[q] = R::load(a.rows, row[q] * a.rs + c0);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (row[q] < 0) continue;
                if (a.drows) {
                    float o[R::VEC];
#pragma unroll
                    for (int e = 0; e < R::VEC; ++e) o[e] = w[q] * R::get(g, e);
                    R::store(a.drows, row[q] * a.drs + c0, o);
                }
                if (a.dw && !tail) {
#pragma unroll
                    for (int e = 0; e < R::VEC; ++e) dot[q] = fmaf(R::get(g, e), R::get(y[q], e), dot[q]);
                } else if (a.dw) {
#pragma unroll
                    for (int e = 0; e < R::VEC; ++e)
                        if (e >= old) dot[q] = fmaf(R::get(g, e), R::get(y[q], e), dot[q]);
                }
            }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) dot[q] += __shfl_xor(dot[q], o, 64);
        }
        if (WAVES == 1) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (lane == q && j0 + q < a.k) a.dw[t * a.k + j0 + q] = dot[q];
        } else {
            __syncthreads();                               // red's previous readers are done
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q < 8; ++q) red[wave][q] = dot[q];
            }
            __syncthreads();
            const int q = threadIdx.x;
            if (q < 8 && j0 + q < a.k)
                a.dw[t * a.k + j0 + q] = (red[0][q] + red[1][q]) + (red[2][q] + red[3][q]);
        }
    }
}

template <int DT, bool VECTOR>
static void combine_grad(const CombineGradArgs& a, hipStream_t s) {
    const int units = Row<DT, VECTOR>::units(a.d);
    // a wave walks a narrow row alone; four share a wide one
    if (units <= 128)
        hipLaunchKernelGGL((combine_grad_kernel<DT, VECTOR, 1>), dim3(grid_blocks(((int64_t)a.T + 3) / 4)), dim3(kThreads), 0, s,
                           a, units);
    else
        hipLaunchKernelGGL((combine_grad_kernel<DT, VECTOR, 4>), dim3(grid_blocks(a.T)), dim3(kThreads), 0, s, a,
                           units);
}

hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t s) {
    const bool v = a.d * dtype_bytes(a.dtype) >= 16;
    if (a.dtype == kBF16) v ? combine_grad<kBF16, true>(a, s) : combine_grad<kBF16, false>(a, s);
    else if (a.dtype == kF16) v ? combine_grad<kF16, true>(a, s) : combine_grad<kF16, false>(a, s);
    else v ? combine_grad<kF32, true>(a, s) : combine_grad<kF32, false>(a, s);
    return hipGetLastError();
}

}  // namespace moe
