// layer.cu -- what surrounds the GEMMs of a linear layer and of a layer of
// experts: the activation's gradient with the bias gradient, the sort of
// token copies by expert, and the row movements there and back.
//
// All of it is bound by HBM (the sort by latency): every matrix element is
// read once and written once, in 16-byte vectors with several loads in flight
// per thread.  Sums are binary32 in a fixed order (no atomics), so results
// repeat bit for bit; the only atomics are maxima of |x|, which do not depend
// on their order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// 16-byte load of data that the kernel ahead may have written (see launch.cuh)
// or that the same thread may overwrite in place.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x);
    f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z);
    f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ uint32_t absmax8(uint32_t acc, const uint4& w) {
    return absmax2_nan(absmax2_nan(absmax2_nan(absmax2_nan(acc, w.x), w.y), w.z), w.w);
}

// Fold every thread's packed |bf16| maximum into *amax (binary32, zeroed by
// the caller): one atomic per CTA, none where the word is already as large.
// As bits a NaN is above every number, so it stays.
__device__ __forceinline__ uint32_t cta_max(uint32_t m) {   // the result in thread 0
    __shared__ uint32_t s_max[kWarps];
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 0; w < kWarps; ++w) m = max(m, s_max[w]);
    return m;
}
__device__ __forceinline__ void publish_amax(float* amax, uint32_t acc) {
    const uint32_t b = cta_max(absmax2_fold(acc));
    if (threadIdx.x == 0) {
        uint32_t* word = reinterpret_cast<uint32_t*>(amax);
        if (b > *reinterpret_cast<volatile uint32_t*>(word)) atomicMax(word, b);
    }
}

// ------------------------------------------------------ activation gradient --
// dz = dy * act'(z) and the column sums of dz.  A CTA takes 128 (or 32) rows x
// 256 columns, and since segments start at multiples of 128 no tile crosses
// one; a warp takes every 8th of the rows, a lane 8 columns.  6 bytes per
// element moved; the sums of a tile's rows go to the workspace, [row tiles x N]
// binary32 (1/192 of the bytes with 128 rows, 1/48 with 32), and
// bias_grad_kernel adds them up in order.  With 128 rows a thread goes through its rows in four steps of
// four; where that leaves fewer than 4 CTAs to an SM, 32 rows give every
// thread one step: 1000 x 4100 16.4 -> 12.3 us.
// Four CTAs to an SM (64 registers): with gelu's 74, 16384 x 14336 takes 243 us
// instead of 227.
constexpr int kColTile = 256;
constexpr int64_t kRowTile = 128, kRowTileFew = 32;

struct ActGradParams {
    const __nv_bfloat16* dy;
    const __nv_bfloat16* z;
    __nv_bfloat16* dz;
    int64_t ldy, ldz, lddz;
    int64_t M, N;
    int64_t strips;        // ceil(N / kColTile)
    int tile_rows;
    const int* offsets;    // nullable: rows in expert segments
    const int* counts;
    int experts;
    float* sums;           // [row tiles x N], or dbias itself when one row tile is all there is; nullable
    float* amax;           // nullable: one word for all CTAs
    uint32_t* maxima;      // nullable: a word for each CTA instead
};

// Rows of the row tile at m0 that belong to tokens: all of M, or those inside
// the segment that covers the tile.  offsets are unchecked device data; the
// result lies in [m0, M] whatever they hold.
__device__ __forceinline__ int64_t live_rows(const int* offsets, const int* counts, int experts, int64_t m0, int64_t M) {
    if (!offsets) return M;
    int lo = 0, hi = experts;   // last entry with offsets[lo] <= m0
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets[mid] <= m0) lo = mid;
        else hi = mid - 1;
    }
    if (lo >= experts) return m0;
    const int64_t end = min((int64_t)offsets[lo] + counts[lo], (int64_t)offsets[lo + 1]);
    return max(m0, min(end, M));
}

template <int ACT>
__global__ void __launch_bounds__(kThreads, 4) act_grad_kernel(ActGradParams p) {
    __shared__ float s_sum[kWarps][kColTile];
    wait_for_stream();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / p.strips, strip = blockIdx.x - tile * p.strips;   // columns fastest
    const int64_t m0 = tile * p.tile_rows, col = strip * kColTile + 8 * lane;
    const int64_t stop = min(m0 + p.tile_rows, p.M);                               // rows to write
    const int64_t live = min(live_rows(p.offsets, p.counts, p.experts, m0, p.M), stop);   // rows to compute
    const int64_t n = p.N - col;
    float sum[8] = {};
    uint32_t peak = 0;
    constexpr int U = 4;
    for (int64_t r0 = m0 + warp; r0 < stop; r0 += U * kWarps) {
        uint4 g[U], z[U];
        if (n >= 8) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + u * kWarps;
                g[u] = z[u] = make_uint4(0, 0, 0, 0);
                if (r < live) {
                    g[u] = ld_stream(p.dy + r * p.ldy + col);
                    if (ACT != ACT_NONE) z[u] = ld_stream(p.z + r * p.ldz + col);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + u * kWarps;
                if (r >= stop) break;
                float a[8], b[8];
                unpack8(g[u], a);
                unpack8(z[u], b);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 v = act_grad_value2<ACT>(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
                    a[e] = r < live ? v.x : 0.0f;
                    a[e + 1] = r < live ? v.y : 0.0f;
                    sum[e] += a[e];
                    sum[e + 1] += a[e + 1];
                }
                const uint4 o = pack8(a);
                peak = absmax8(peak, o);
                *reinterpret_cast<uint4*>(p.dz + r * p.lddz + col) = o;
            }
        } else if (n > 0) {
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + u * kWarps;
                if (r >= stop) break;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) {
                        float v = 0.0f;
                        if (r < live)
                            v = act_grad_value<ACT>(__bfloat162float(p.dy[r * p.ldy + col + e]),
                                                    ACT == ACT_NONE ? 0.0f : __bfloat162float(p.z[r * p.ldz + col + e]));
                        sum[e] += v;
                        const __nv_bfloat16 h = __float2bfloat16_rn(v);
                        peak = absmax2_nan(peak, (uint32_t)__bfloat16_as_ushort(h));
                        p.dz[r * p.lddz + col + e] = h;
                    }
            }
        }
    }
    if (p.sums) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_sum[warp][8 * lane + e] = sum[e];
        __syncthreads();
        const int64_t c = strip * kColTile + threadIdx.x;
        if (c < p.N) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t += s_sum[w][threadIdx.x];
            p.sums[tile * p.N + c] = t;
        }
    }
    if (p.amax) publish_amax(p.amax, peak);
    if (p.maxima) {
        const uint32_t m = cta_max(absmax2_fold(peak));
        if (threadIdx.x == 0) p.maxima[blockIdx.x] = m;
    }
}

// dbias [experts x N] from the sums of the row tiles: 64 columns per CTA, the
// tiles of a segment dealt to 4 threads per column, then added in order.  With
// `amax`, one more CTA takes the maximum of the first kernel's CTAs.
__global__ void __launch_bounds__(kThreads) bias_grad_kernel(const float* sums, int64_t M, int64_t N,
                                                             int tile_rows, const int* offsets, const int* counts, float* dbias,
                                                             const uint32_t* maxima, int n_maxima, float* amax) {
    __shared__ float s[4][64];
    wait_for_stream();
    if ((int64_t)blockIdx.x * 64 >= N) {
        if (blockIdx.y) return;
        uint32_t m = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < n_maxima; i += kThreads) m = max(m, maxima[i]);
        m = cta_max(m);
        if (threadIdx.x == 0) *amax = __uint_as_float(m);
        return;
    }
    const int e = blockIdx.y, part = threadIdx.x >> 6, c = threadIdx.x & 63;
    const int64_t col = (int64_t)blockIdx.x * 64 + c;
    const int64_t tiles = (M + tile_rows - 1) / tile_rows;
    int64_t first = 0, last = tiles;
    if (offsets) {
        const int64_t o = offsets[e];
        const int64_t end = min(o + counts[e], (int64_t)offsets[e + 1]);
        first = max(o, (int64_t)0) / tile_rows;
        last = min(tiles, (end + tile_rows - 1) / tile_rows);
    }
    float t = 0.0f;
    if (col < N) {
#pragma unroll 8
        for (int64_t i = first + part; i < last; i += 4) t += sums[i * N + col];
    }
    s[part][c] = t;
    __syncthreads();
    if (part == 0 && col < N) dbias[(int64_t)e * N + col] = (s[0][c] + s[1][c]) + (s[2][c] + s[3][c]);
}

// ------------------------------------------------------------ sort by expert --
// A stable counting sort of n copies by expert.  The copies are dealt to CTAs
// in consecutive chunks, to a CTA's warps in consecutive parts, to a warp's
// lanes 32 at a time; a copy's rank among its expert's is the sum of what came
// before on each of these levels, so it depends on the input alone.
struct SortParams {
    const int* ids;       // [n]
    int n, experts, rows;
    int chunk;            // copies per CTA, a multiple of kThreads
    int* hist;            // [CTAs x experts], only with more than one CTA
    int* offsets;
    int* counts;
    int* row_copy;        // [rows]
    int* copy_row;        // [n]
};

__global__ void __launch_bounds__(kThreads) sort_count_kernel(SortParams p) {
    extern __shared__ int s_count[];
    wait_for_stream();
    for (int e = threadIdx.x; e < p.experts; e += kThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(begin + p.chunk, (int64_t)p.n);
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.experts) atomicAdd(s_count + e, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kThreads) p.hist[(int64_t)blockIdx.x * p.experts + e] = s_count[e];
}

__global__ void __launch_bounds__(kThreads) sort_place_kernel(SortParams p) {
    extern __shared__ int s_mem[];
    int* s_at = s_mem;                              // [warps x experts] next row of each warp's copies of an expert
    int* s_off = s_mem + kWarps * p.experts;        // [experts + 1]
    int* s_total = s_off + p.experts + 1;           // [experts]
    __shared__ int s_scan[kWarps], s_carry;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kWarps * p.experts; i += kThreads) s_at[i] = 0;
    if (threadIdx.x == 0) s_carry = 0;
    __syncthreads();
    wait_for_stream();
    // this CTA's copies, counted per warp
    const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(begin + p.chunk, (int64_t)p.n);
    const int part = p.chunk / kWarps;
    const int64_t wb = begin + (int64_t)warp * part, we = min(wb + part, end);
    for (int64_t i = wb + lane; i < we; i += 32) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.experts) atomicAdd(s_at + warp * p.experts + e, 1);
    }
    __syncthreads();
    // per expert: the total over all CTAs, and where this CTA's first copy goes among them
    for (int base = 0; base < p.experts; base += kThreads) {
        const int e = base + threadIdx.x;
        int before = 0, total = 0;
        if (e < p.experts) {
            if (gridDim.x == 1) {
                for (int w = 0; w < kWarps; ++w) total += s_at[w * p.experts + e];
            } else {
#pragma unroll 4
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int h = p.hist[(int64_t)b * p.experts + e];
                    total += h;
                    if (b < (int)blockIdx.x) before += h;
                }
            }
            s_total[e] = total;
        }
        // exclusive running sum of the padded totals over the CTA's threads
        const int padded = (total + 127) & ~127;
        int incl = padded;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += u;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        int lead = s_carry;
        for (int w = 0; w < warp; ++w) lead += s_scan[w];
        if (e < p.experts) {
            s_off[e] = lead + incl - padded;
            int at = s_off[e] + before;
            for (int w = 0; w < kWarps; ++w) {
                const int c = s_at[w * p.experts + e];
                s_at[w * p.experts + e] = at;
                at += c;
            }
            if (e == p.experts - 1) s_off[p.experts] = lead + incl;
        }
        __syncthreads();
        if (threadIdx.x == kThreads - 1) s_carry = lead + incl;
        __syncthreads();
    }
    // offsets and counts, no further than the rows there are
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= p.experts; e += kThreads) {
            const int o = min(s_off[e], p.rows);
            p.offsets[e] = o;
            if (e < p.experts) p.counts[e] = min(s_total[e], min(s_off[e + 1], p.rows) - o);
        }
    }
    // place the copies
    for (int64_t i0 = wb; i0 < we; i0 += 32) {
        const int64_t i = i0 + lane;
        const int e = i < we ? p.ids[i] : -1;
        const bool ok = e >= 0 && e < p.experts;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, ok ? e : -1);
        int row = -1;
        if (ok) row = s_at[warp * p.experts + e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (ok && (same >> lane) == 1u) s_at[warp * p.experts + e] = row + 1;   // the last of its kind
        __syncwarp();
        if (row >= p.rows) row = -1;
        if (i < we) p.copy_row[i] = row;
        if (row >= 0) p.row_copy[row] = (int)i;
    }
    // rows without a copy
    for (int e = blockIdx.x; e <= p.experts; e += gridDim.x) {
        const int from = min(e < p.experts ? s_off[e] + s_total[e] : s_off[e], p.rows);
        const int to = e < p.experts ? min(s_off[e + 1], p.rows) : p.rows;
        for (int r = from + threadIdx.x; r < to; r += kThreads) p.row_copy[r] = -1;
    }
}

// -------------------------------------------------------- rows there and back --
struct MoveParams {
    const __nv_bfloat16* src;       // gather: x; combine: y; gradient: dout
    const __nv_bfloat16* other;     // combine: residual (nullable); gradient: y (nullable)
    __nv_bfloat16* dst;             // gather: sorted rows; combine: out; gradient: dy
    int64_t lds, ldo, ldd;
    const int* copy_row;            // [tokens x topk]
    const int* row_copy;            // [rows]
    const float* weights;           // [tokens x topk], nullable: 1
    float* dweights;                // gradient, nullable
    float* amax;                    // nullable
    int64_t tokens, rows, cols;
    int topk;
};

__device__ __forceinline__ int row_of(const MoveParams& p, int64_t copy) {
    const int r = p.copy_row[copy];
    return r >= 0 && r < p.rows ? r : -1;
}

// Rows that hold no copy become zeros: one warp looks at 8 rows x 1024 columns
// (few, because padding rows lie together: up to 127 behind each segment).
constexpr int kZeroRows = 8;
__device__ __forceinline__ int64_t zero_units(const MoveParams& p) {
    return (p.rows + kZeroRows - 1) / kZeroRows * ((p.cols + 1023) / 1024);
}
__device__ __forceinline__ void zero_unit(const MoveParams& p, int64_t unit, int lane) {
    const int64_t groups = (p.rows + kZeroRows - 1) / kZeroRows;
    const int64_t r0 = unit % groups * kZeroRows, c0 = unit / groups * 1024;
    bool empty = false;
    if (lane < kZeroRows && r0 + lane < p.rows) {
        const int c = p.row_copy[r0 + lane];
        empty = c < 0 || c >= p.tokens * p.topk;
    }
    unsigned todo = __ballot_sync(0xFFFFFFFFu, empty);
    while (todo) {
        const int64_t r = r0 + __ffs(todo) - 1;
        todo &= todo - 1;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t c = c0 + 256 * v + 8 * lane;
            if (c < p.cols) *reinterpret_cast<uint4*>(p.dst + r * p.ldd + c) = make_uint4(0, 0, 0, 0);
        }
    }
}

// Sorted rows from token rows.  A warp takes 1024 columns of one token: reads
// them once, 4 loads in flight per lane, and writes them topk times.
__global__ void __launch_bounds__(kThreads) gather_kernel(MoveParams p) {
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int64_t segs = (p.cols + 1023) / 1024, units = p.tokens * segs, all = units + zero_units(p);
    uint32_t peak = 0;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < all; u += (int64_t)gridDim.x * kWarps) {
        if (u >= units) {
            zero_unit(p, u - units, lane);
            continue;
        }
        const int64_t t = u / segs, c0 = (u - t * segs) * 1024 + 8 * lane;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = c0 + 256 * i < p.cols ? ld_stream(p.src + t * p.lds + c0 + 256 * i) : make_uint4(0, 0, 0, 0);
        bool used = false;
        for (int j = 0; j < p.topk; ++j) {
            const int r = row_of(p, t * p.topk + j);
            if (r < 0) continue;
            used = true;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + 256 * i < p.cols) *reinterpret_cast<uint4*>(p.dst + r * p.ldd + c0 + 256 * i) = v[i];
        }
        if (used) {
#pragma unroll
            for (int i = 0; i < 4; ++i) peak = absmax8(peak, v[i]);
        }
    }
    if (p.amax) publish_amax(p.amax, peak);
}

// Token rows from sorted rows: a warp takes 512 columns of one token, the rows
// of 2 copies in flight at a time, and sums in the order of the copies.
// 16384 x 2 x 8192 with the residual (VECS, COPIES): (2, 2) 0.162 ms, (4, 2)
// 0.161, (2, 4) 0.197, (1, 2) 0.201, (1, 4) 0.269; of (2, 2) and (4, 2) the one
// with more units for few tokens.
constexpr int VECS = 2, COPIES = 2;
__global__ void __launch_bounds__(kThreads) combine_kernel(MoveParams p) {
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    constexpr int kCols = 256 * VECS;
    const int64_t segs = (p.cols + kCols - 1) / kCols, units = p.tokens * segs;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
        const int64_t t = u / segs, c0 = (u - t * segs) * kCols + 8 * lane;
        bool in[VECS];
        float acc[VECS][8] = {};
        uint4 res[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            in[i] = c0 + 256 * i < p.cols;
            res[i] = p.other && in[i] ? ld_stream(p.other + t * p.ldo + c0 + 256 * i) : make_uint4(0, 0, 0, 0);
        }
        for (int j0 = 0; j0 < p.topk; j0 += COPIES) {
            uint4 v[COPIES][VECS];
            float w[COPIES];
            int r[COPIES];
#pragma unroll
            for (int j = 0; j < COPIES; ++j) {
                r[j] = j0 + j < p.topk ? row_of(p, t * p.topk + j0 + j) : -1;
                w[j] = r[j] < 0 ? 0.0f : p.weights ? p.weights[t * p.topk + j0 + j] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < COPIES; ++j)
#pragma unroll
                for (int i = 0; i < VECS; ++i)
                    v[j][i] = r[j] >= 0 && in[i] ? ld_stream(p.src + r[j] * p.lds + c0 + 256 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < COPIES; ++j)
#pragma unroll
                for (int i = 0; i < VECS; ++i) {
                    float f[8];
                    unpack8(v[j][i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i][e] = fmaf(w[j], f[e], acc[i][e]);
                }
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            if (!in[i]) continue;
            float f[8];
            unpack8(res[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i][e] += f[e];
            *reinterpret_cast<uint4*>(p.dst + t * p.ldd + c0 + 256 * i) = pack8(acc[i]);
        }
    }
}

// The gradient of combine.  WARPS warps (1, or the CTA's 8) take up to 4 copies
// of one token: its row of dout is read (by a second group of 4 from L2), each
// copy's row of dy is written, each copy's row of y is read for dweights =
// <dout, y>.  A lane's binary32 partial sums are added over lanes, then over
// warps in order.  Further units zero the rows that hold no copy.  One warp per
// unit needs no block-wide step and serves many tokens; with few, 8 warps share
// a row, so that its loads are all in flight at once.
constexpr int kDots = 4;

template <int WARPS>
__global__ void __launch_bounds__(kThreads, 4) combine_grad_kernel(MoveParams p) {
    __shared__ float s_dot[kWarps][kDots];
    wait_for_stream();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = WARPS == 1 ? 0 : warp;
    const int groups = (p.topk + kDots - 1) / kDots;
    const int64_t units = p.tokens * groups, all = units + (zero_units(p) + WARPS - 1) / WARPS;
    const bool dots = p.dweights != nullptr;
    uint32_t peak = 0;
    const int64_t first = WARPS == 1 ? (int64_t)blockIdx.x * kWarps + warp : blockIdx.x;
    for (int64_t u = first; u < all; u += (int64_t)gridDim.x * (kWarps / WARPS)) {
        if (u >= units) {
            const int64_t z = (u - units) * WARPS + sub;
            if (z < zero_units(p)) zero_unit(p, z, lane);
            continue;
        }
        const int64_t t = u / groups;
        const int j0 = (int)(u - t * groups) * kDots, m = min(kDots, p.topk - j0);
        const int64_t copy0 = t * p.topk + j0;
        int row[kDots];
        float w[kDots], dot[kDots];
#pragma unroll
        for (int j = 0; j < kDots; ++j) {
            row[j] = j < m ? row_of(p, copy0 + j) : -1;
            w[j] = j < m && p.weights ? p.weights[copy0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int64_t c = 8 * (sub * 32 + lane); c < p.cols; c += 8 * 32 * WARPS) {
            const uint4 g = *reinterpret_cast<const uint4*>(p.src + t * p.lds + c);
            uint4 y[kDots];
#pragma unroll
            for (int j = 0; j < kDots; ++j)
                if (dots && row[j] >= 0) y[j] = ld_stream(p.other + row[j] * p.ldo + c);
            float f[8];
            unpack8(g, f);
#pragma unroll
            for (int j = 0; j < kDots; ++j) {
                if (row[j] < 0) continue;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = w[j] * f[e];
                const uint4 d = pack8(o);
                peak = absmax8(peak, d);
                *reinterpret_cast<uint4*>(p.dst + row[j] * p.ldd + c) = d;
                if (dots) {
                    unpack8(y[j], o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = fmaf(o[e], f[e], dot[j]);
                }
            }
        }
        if (dots) {
#pragma unroll
            for (int j = 0; j < kDots; ++j)
#pragma unroll
                for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
            if constexpr (WARPS == 1) {
#pragma unroll
                for (int j = 0; j < kDots; ++j)
                    if (lane == j && j < m) p.dweights[copy0 + j] = dot[j];
            } else {
#pragma unroll
                for (int j = 0; j < kDots; ++j)
                    if (lane == 0) s_dot[warp][j] = dot[j];
                __syncthreads();
                if (threadIdx.x < m) {
                    float s = 0.0f;
                    for (int v = 0; v < kWarps; ++v) s += s_dot[v][threadIdx.x];
                    p.dweights[copy0 + threadIdx.x] = s;
                }
                __syncthreads();
            }
        }
    }
    if (p.amax) publish_amax(p.amax, peak);
}

// ----------------------------------------------------------- host side -----
int sm_count() {
    static int cached[64];
    static std::mutex mu;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!cached[dev]) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        cached[dev] = n > 0 ? n : 148;
    }
    return cached[dev];
}

MoveParams move_params(const MoveArgs& a) {
    MoveParams p{};
    p.src = static_cast<const __nv_bfloat16*>(a.src);
    p.other = static_cast<const __nv_bfloat16*>(a.other);
    p.dst = static_cast<__nv_bfloat16*>(a.dst);
    p.lds = a.lds;
    p.ldo = a.ldo;
    p.ldd = a.ldd;
    p.copy_row = a.copy_row;
    p.row_copy = a.row_copy;
    p.weights = a.weights;
    p.dweights = a.dweights;
    p.amax = a.amax;
    p.tokens = a.tokens;
    p.rows = a.rows;
    p.cols = a.cols;
    p.topk = (int)a.topk;
    return p;
}

// Enough CTAs for the units, at most 8 (2048 threads) on each SM.
int grid_for_units(int64_t units) { return (int)std::max<int64_t>(1, std::min<int64_t>(units, (int64_t)sm_count() * 8)); }
int64_t zero_units_host(const MoveArgs& a) { return ceil_div(a.rows, kZeroRows) * ceil_div(a.cols, 1024); }

__global__ void zero_word_kernel(float* word) {
    wait_for_stream();
    if (threadIdx.x == 0) *word = 0.0f;
}

}  // namespace

// A maximum starts at 0.  (A memset in front of a kernel costs 3 us in a chain of small kernels, this 1.5.)
cudaError_t zero_word(float* amax, cudaStream_t s) {
    return amax ? launch_early(zero_word_kernel, 1, 32, 0, s, 1, amax) : cudaSuccess;
}

static int64_t act_grad_tile_rows(int64_t M, int64_t N) {
    return ceil_div(M, kRowTile) * ceil_div(N, kColTile) < 4 * (int64_t)sm_count() ? kRowTileFew : kRowTile;
}
// The sums of the row tiles and the maxima of the CTAs.
size_t act_grad_workspace(int64_t M, int64_t N) {
    return (size_t)(ceil_div(M, act_grad_tile_rows(M, N)) * (N + ceil_div(N, kColTile))) * sizeof(float);
}

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s, int* launches) {
    ActGradParams p{};
    p.dy = static_cast<const __nv_bfloat16*>(a.dy);
    p.z = static_cast<const __nv_bfloat16*>(a.z);
    p.dz = static_cast<__nv_bfloat16*>(a.dz);
    p.ldy = a.ldy;
    p.ldz = a.ldz;
    p.lddz = a.lddz;
    p.M = a.M;
    p.N = a.N;
    p.offsets = a.offsets;
    p.counts = a.counts;
    p.experts = (int)a.experts;
    p.amax = a.amax;
    p.strips = ceil_div(a.N, kColTile);
    p.tile_rows = (int)act_grad_tile_rows(a.M, a.N);
    const int64_t tiles = ceil_div(a.M, p.tile_rows);
    const bool direct = a.dbias && tiles == 1 && !a.offsets;   // one row tile: its sums are the result
    p.sums = direct ? a.dbias : a.dbias ? a.workspace : nullptr;
    const bool second = a.dbias && !direct;   // a second kernel, which then takes the maximum too
    cudaError_t e = cudaSuccess;
    if (second && a.amax) {
        p.amax = nullptr;
        p.maxima = reinterpret_cast<uint32_t*>(a.workspace + tiles * a.N);
    } else if (a.amax) {
        *launches += 1;
        e = zero_word(a.amax, s);
        if (e != cudaSuccess) return e;
    }
    const unsigned grid = (unsigned)(tiles * p.strips);
    switch (a.act) {
        case ACT_RELU: e = launch_early(act_grad_kernel<ACT_RELU>, grid, kThreads, 0, s, 1, p); break;
        case ACT_RELU2: e = launch_early(act_grad_kernel<ACT_RELU2>, grid, kThreads, 0, s, 1, p); break;
        case ACT_GELU: e = launch_early(act_grad_kernel<ACT_GELU>, grid, kThreads, 0, s, 1, p); break;
        case ACT_GELU_TANH: e = launch_early(act_grad_kernel<ACT_GELU_TANH>, grid, kThreads, 0, s, 1, p); break;
        case ACT_SILU: e = launch_early(act_grad_kernel<ACT_SILU>, grid, kThreads, 0, s, 1, p); break;
        default: e = launch_early(act_grad_kernel<ACT_NONE>, grid, kThreads, 0, s, 1, p); break;
    }
    *launches += 1;
    if (e != cudaSuccess || !second) return e;
    const dim3 bgrid((unsigned)(ceil_div(a.N, 64) + (a.amax ? 1 : 0)), (unsigned)(a.offsets ? a.experts : 1));
    *launches += 1;
    return launch_early(bias_grad_kernel, bgrid, kThreads, 0, s, 1, a.workspace, a.M, a.N, p.tile_rows, a.offsets, a.counts,
                        a.dbias, p.maxima, (int)grid, a.amax);
}

// CTAs of the sort: about 1024 copies each, fewer where the table of counts
// that every CTA reads (CTAs x experts) would grow past 64K entries.
static int64_t sort_ctas(int64_t n, int64_t experts) {
    return std::max<int64_t>(1, std::min<int64_t>(ceil_div(n, 1024), (1 << 16) / experts));
}
size_t moe_sort_workspace(int64_t n, int64_t experts) { return (size_t)(sort_ctas(n, experts) * experts * 4); }

cudaError_t launch_moe_sort(const SortArgs& a, cudaStream_t s, int* launches) {
    SortParams p{};
    p.ids = a.ids;
    p.n = (int)a.n;
    p.experts = (int)a.experts;
    p.rows = (int)a.rows;
    p.hist = a.workspace;
    p.offsets = a.offsets;
    p.counts = a.counts;
    p.row_copy = a.row_copy;
    p.copy_row = a.copy_row;
    p.chunk = (int)(ceil_div(ceil_div(a.n, sort_ctas(a.n, a.experts)), kThreads) * kThreads);
    const int ctas = (int)ceil_div(a.n, p.chunk);
    const int smem = (int)(((kWarps + 2) * a.experts + 1) * 4);   // at most 20 KB: 512 experts
    if (ctas > 1) {
        *launches += 1;
        cudaError_t e = launch_early(sort_count_kernel, ctas, kThreads, p.experts * 4, s, 1, p);
        if (e != cudaSuccess) return e;
    }
    *launches += 1;
    return launch_early(sort_place_kernel, ctas, kThreads, smem, s, 1, p);
}

cudaError_t launch_moe_gather(const MoveArgs& a, cudaStream_t s, int* launches) {
    cudaError_t e = zero_word(a.amax, s);
    if (e != cudaSuccess) return e;
    const int64_t units = a.tokens * ceil_div(a.cols, 1024) + zero_units_host(a);
    *launches += a.amax ? 2 : 1;
    return launch_early(gather_kernel, grid_for_units(ceil_div(units, kWarps)), kThreads, 0, s, 1, move_params(a));
}

cudaError_t launch_moe_combine(const MoveArgs& a, cudaStream_t s, int* launches) {
    *launches += 1;
    const int64_t units = a.tokens * ceil_div(a.cols, 256 * VECS);
    return launch_early(combine_kernel, grid_for_units(ceil_div(units, kWarps)), kThreads, 0, s, 1, move_params(a));
}

cudaError_t launch_moe_combine_grad(const MoveArgs& a, cudaStream_t s, int* launches) {
    cudaError_t e = zero_word(a.amax, s);
    if (e != cudaSuccess) return e;
    const int64_t units = a.tokens * ceil_div(a.topk, kDots), zeros = zero_units_host(a);
    *launches += a.amax ? 2 : 1;
    if (units >= 16 * (int64_t)sm_count())
        return launch_early(combine_grad_kernel<1>, grid_for_units(ceil_div(units + zeros, kWarps)), kThreads, 0, s, 1,
                            move_params(a));
    return launch_early(combine_grad_kernel<kWarps>, grid_for_units(units + ceil_div(zeros, kWarps)), kThreads, 0, s, 1,
                        move_params(a));
}

}  // namespace nvfp4
