// few.cu -- the linear layer's product for few rows (tokens): one to 128, and
// experts that have a few rows each.
//
// C[t][n] = act(alpha sum_k x_tk w_nk + bias_n) + residual_tn.  With few rows
// the weight is read once and hardly used: 0.5625 bytes per element against
// 2 t flops, far on the memory side up to some hundred rows.  So the weight takes
// the place of the matrix product's wide operand and the tokens that of the
// narrow one: tcgen05.mma M = 128 features x N = 16 .. 128 tokens, K = 64.
//   - A CTA takes 128 features and a part of K; the CTAs of a cluster (1 to 8)
//     share K, so that a small weight still fills the GPU.  Their accumulators
//     meet in distributed shared memory, tokens dealt to the CTAs, and are
//     added in the order of the CTAs: no workspace, no atomics, the same
//     result every time.
//   - Two CTAs to an SM, each with 72 KB (more than 32 tokens: 54 KB) of weight
//     in flight, several times what hides the latency of HBM.
//   - Weights with more tiles than the GPU has SMs need no split: then a CTA
//     streams through tiles (gemm_few_stream_kernel).
//   - Experts with more rows than a pass takes (32 streaming, 128 in a cluster,
//     where the few tiles leave more to gain: 2048 x 2048 with 128 rows 19 -> 10
//     us): the passes behind the first are dealt to all CTAs or clusters, so
//     that an expert which got most of the tokens does not leave the GPU to a
//     few of them (2048 rows at one of 64 experts of 256 x 2048: 340 -> 15 us).
// Measured in a captured graph, 400 MB of weights in turn (us, share of HBM's
// rate on the weight's bytes): one token through 14336 x 4096 9.5 (0.53), 28672
// x 8192 24.5 (0.82), 131072 x 4096 51.5 (0.89); 16 tokens x 2 through 8 experts
// of 14336 x 4096 57 (0.71).
//   - Warp 0: TMA producer.  Warp 1: the MMAs.  Warps 2 .. 5: block scales to
//     tensor memory (a copy by the tensor core, tcgen05.cp, costs its pipe 64
//     cycles; with 8 of them a block of K = 256 took 1015 cycles instead of
//     the MMAs' 500, more than the time of its bytes), then the
//     way out of tensor memory (a feature to a lane); all warps then finish
//     rows, four features to a lane.
// Every wait is bounded, as in the large product.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "activation.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "segments.cuh"
#include "tc.cuh"

namespace nvfp4 {

namespace {

constexpr int F_ROWS = 128;                     // features of a CTA
constexpr int F_BKB = 128;                      // bytes of codes per row and stage: K = 256
constexpr int F_W_STAGE = F_ROWS * F_BKB;       // 16 KB
constexpr int F_SF_STAGE = 4 * 512;             // 4 K steps of 128 rows x 4 scales
constexpr int F_THREADS = 192;
constexpr uint32_t F_TMEM = 256;
constexpr int F_GROUPS = 5;                     // 32 experts each: more than 160 experts are never split

// TOK: most tokens of one pass.
template <int TOK>
struct Layout {
    static constexpr int kStages = TOK == 128 ? 3 : 4;
    static constexpr int kX = TOK * F_BKB;
    static constexpr int kStage = F_W_STAGE + kX + 2 * F_SF_STAGE;
    static constexpr int kOffX = F_W_STAGE, kOffSfw = kOffX + kX, kOffSfx = kOffSfw + F_SF_STAGE;
    // Partial sums of a cluster, [CTA][token][feature]: with few tokens in memory of their own, else in the stages,
    // which the cluster first has to be done with.
    static constexpr bool kOwnSums = TOK == 16;
    static constexpr int kOffSums = kOwnSums ? kStages * kStage : 0;
    static constexpr int kOffBar = kStages * kStage + (kOwnSums ? TOK * F_ROWS * 4 : 0);
    static constexpr int kOffMisc = kOffBar + (3 * kStages + 2) * 8;
    static constexpr int kBytes = kOffMisc + 16 + 1008;
    static constexpr uint32_t kSf = TOK;               // first tensor-memory column of the scales, 32 per stage
    static_assert(kStage % 1024 == 0 && kSf + kStages * 32 <= F_TMEM, "layout");
    static_assert(TOK >= 8 && kOffSums + TOK * F_ROWS * 4 <= kOffBar, "partial sums of a cluster of up to 8");
    // full, empty, scales per stage; accumulator, drain: at kOffBar
};

struct FewParams {
    const uint8_t* sfx;
    const uint8_t* sfw;
    const float* x_gs;
    const float* w_gs;
    int M, N, K;
    int chunks_k;
    int tiles;                      // ceil(N / 128)
    int64_t sfw_stride;             // bytes of one expert's weight scales
    const int* offsets;             // nullable: rows in expert segments
    const int* counts;
    int experts;
    const __nv_bfloat16* bias;
    const __nv_bfloat16* residual;
    int64_t ldr;
    int out_bf16;
    void* c;
    int64_t ldc;
    __nv_bfloat16* pre;
    int64_t ldp;
    unsigned int* c_amax;
    int act;
};

// One thread issues the MMAs of the CTA, and little should stand between them:
// the upper words of the descriptors are constants, the lower ones, which hold
// address / 16, a base per stage plus constants.
constexpr uint32_t kCodesLo = 1u << 16, kCodesHi = (1024u >> 4) | 1u << 14 | 2u << 29;   // as desc_sw128
__device__ __forceinline__ uint64_t codes_desc(uint32_t at16) { return (uint64_t)kCodesHi << 32 | (kCodesLo + at16); }
// The K steps of one stage; `at` is its address / 16, `sf` its scales' columns.
template <int OFF_X>
__device__ __forceinline__ void issue_steps(uint32_t tmem, uint32_t at, uint32_t sf, uint32_t idesc, int nk, bool add) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < nk)
            tc_mma_nvf4(tmem, codes_desc(at + 2 * j), codes_desc(at + OFF_X / 16 + 2 * j), idesc, sf + 4 * j, sf + 16 + 4 * j,
                        j > 0 || add, false);
}
__device__ __forceinline__ void tc_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t rank, float v) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %0, %1;\n\t"
        "st.shared::cluster.f32 [ra], %2;\n\t}"
        ::"r"(addr), "r"(rank), "f"(v)
        : "memory");
}

// Four consecutive features of one token, from their sums over K.
struct Finish {
    float2 alpha;
    float bias[4];
    int64_t n;      // first feature
    int count;      // how many of them exist
};
__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(__nv_bfloat16* q, const uint2& w, int count) {
    if (count >= 4) {
        *reinterpret_cast<uint2*>(q) = w;
    } else {
        const uint32_t h[2] = {w.x, w.y};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < count) reinterpret_cast<uint16_t*>(q)[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
    }
}
template <int ACT>
__device__ __forceinline__ void finish(const FewParams& p, const Finish& f, int64_t row, const float4& sum, uint32_t& amax) {
    if (f.count <= 0) return;
    float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaf(v[e] * f.alpha.x, f.alpha.y, f.bias[e]);
    if (p.pre) store4(p.pre + row * p.ldp + f.n, pack4(v), f.count);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = act_value<ACT>(v[e]);
    if (p.residual) {
        const __nv_bfloat16* r = p.residual + row * p.ldr + f.n;
        if (f.count >= 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(r);
            v[0] += bf16_lo(w.x);
            v[1] += bf16_hi(w.x);
            v[2] += bf16_lo(w.y);
            v[3] += bf16_hi(w.y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < f.count) v[e] += __bfloat162float(r[e]);
        }
    }
    if (p.out_bf16) {
        const uint2 w = pack4(v);
        store4(static_cast<__nv_bfloat16*>(p.c) + row * p.ldc + f.n, w, f.count);
        v[0] = bf16_lo(w.x);
        v[1] = bf16_hi(w.x);
        v[2] = bf16_lo(w.y);
        v[3] = bf16_hi(w.y);
    } else {
        float* q = static_cast<float*>(p.c) + row * p.ldc + f.n;
        if (f.count >= 4) {
            *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < f.count) q[e] = v[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < f.count) amax = max(amax, __float_as_uint(fabsf(v[e])));
}

// One stage: K block kb of the weight tile at row w_row and of the tokens from t0.
struct Source {
    const uint8_t* sfw;
    const uint8_t* sfx;
    int w_row, t0, boxes;
};
template <int TOK>
__device__ __forceinline__ void load_stage(uint32_t at, uint32_t full, const CUtensorMap& map_w, const CUtensorMap& map_x,
                                           const Source& src, int kb, int nk) {
    using L = Layout<TOK>;
    mbar_expect_tx(full, (uint32_t)(F_W_STAGE + src.boxes * 16 * F_BKB + 2 * nk * 512));
    tma_load_2d(at, &map_w, full, kb * F_BKB, src.w_row);
    bulk_load(at + L::kOffSfw, src.sfw + (int64_t)kb * 2048, nk * 512, full);
    for (int b = 0; b < src.boxes; ++b)
        tma_load_2d(at + L::kOffX + b * 16 * F_BKB, &map_x, full, kb * F_BKB, src.t0 + 16 * b);
    bulk_load(at + L::kOffSfx, src.sfx + (int64_t)kb * 2048, nk * 512, full);
}
__device__ __forceinline__ Source source(const FewParams& p, int e, int tile, int t0, int tokens) {
    return Source{p.sfw + e * p.sfw_stride + (int64_t)tile * p.chunks_k * 512, p.sfx + (int64_t)(t0 >> 7) * p.chunks_k * 512,
                  e * p.N + tile * F_ROWS, t0, (tokens + 15) / 16};
}
// A stage's block scales, shared memory -> this warp's lane quarter of tensor memory.  32 rows go to a column: a pass of
// up to 32 tokens starts at the column of its rows in the chunk of 128.
template <int TOK>
__device__ __forceinline__ void scale_stage(uint32_t smem_scales, uint32_t taddr, int t0, int lane) {
    const int quarter = (t0 >> 5) & 3;
    uint32_t w[16], x[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 a = lds128(smem_scales + 16 * lane + 512 * j), b = lds128(smem_scales + F_SF_STAGE + 16 * lane + 512 * j);
        w[4 * j] = a.x; w[4 * j + 1] = a.y; w[4 * j + 2] = a.z; w[4 * j + 3] = a.w;
        x[4 * j] = TOK == 128 || quarter == 0 ? b.x : quarter == 1 ? b.y : quarter == 2 ? b.z : b.w;
        x[4 * j + 1] = b.y; x[4 * j + 2] = b.z; x[4 * j + 3] = b.w;
    }
    tc_st_32x32b_x16(taddr, w);
    tc_st_32x32b_x16(taddr + 16, x);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
}
__device__ __forceinline__ uint32_t few_idesc(int boxes) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(16 * boxes >> 3) << 17) | ((uint32_t)(F_ROWS >> 4) << 24);
}
__device__ __forceinline__ Finish finish_at(const FewParams& p, int e, int64_t n) {
    Finish f;
    f.n = n;
    f.count = (int)min((int64_t)4, p.N - n);
    const float sx = *p.x_gs, sw = p.w_gs[e], a = __fmul_rn(sx, sw);
    // as the large product: one factor, or two where it leaves the normal range
    f.alpha = a >= 0x1p-126f && a <= 0x1.fffffep127f ? make_float2(a, 1.0f) : make_float2(sx, sw);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f.bias[i] = p.bias && i < f.count ? __bfloat162float(p.bias[(int64_t)e * p.N + n + i]) : 0.0f;
    return f;
}
// Rows without a token become zeros: the segment's behind `stop`, in this tile's columns.
__device__ __forceinline__ void zero_padding(const FewParams& p, int e, int n0, int stop, int worker, int workers, int lane) {
    const int esz = p.out_bf16 ? 2 : 4, cols = min(F_ROWS, p.N - n0);
    const int end = max(segment_start(p.offsets, e + 1, p.M), stop);
    zero_rows(static_cast<uint8_t*>(p.c) + (int64_t)n0 * esz, (int64_t)cols * esz, p.ldc * esz, stop, end, worker, workers, lane);
    if (p.pre) zero_rows(p.pre + n0, cols * 2, p.ldp * 2, stop, end, worker, workers, lane);
}
// ... and all rows behind the last segment.
__device__ __forceinline__ void zero_tail(const FewParams& p, int worker, int workers, int lane) {
    const int esz = p.out_bf16 ? 2 : 4, tail = segment_start(p.offsets, p.experts, p.M);
    zero_rows(p.c, (int64_t)p.N * esz, p.ldc * esz, tail, p.M, worker, workers, lane);
    if (p.pre) zero_rows(p.pre, (int64_t)p.N * 2, p.ldp * 2, tail, p.M, worker, workers, lane);
}

template <int TOK, int ACT>
__global__ void __launch_bounds__(F_THREADS, 2)
gemm_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, FewParams p) {
    using L = Layout<TOK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + L::kOffBar, bar_empty = bar_full + 8 * L::kStages;
    const uint32_t bar_sf = bar_empty + 8 * L::kStages, bar_acc = bar_sf + 8 * L::kStages, bar_drain = bar_acc + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
    unsigned int* s_amax = reinterpret_cast<unsigned int*>(smem + L::kOffMisc + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), splits = (int)cluster_size();
    const int unit = blockIdx.x / splits, units = gridDim.x / splits;
    const int own = unit / p.tiles, own_tile = unit - own * p.tiles;
    const int steps = p.K / 64, blocks = (steps + 3) / 4;
    const int kb0 = (int)((int64_t)blocks * rank / splits), kb1 = (int)((int64_t)blocks * (rank + 1) / splits);

    if (threadIdx.x == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_x);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
            mbar_init(bar_sf + 8 * s, 4);
        }
        mbar_init(bar_acc, 1);
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        *s_amax = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(F_TMEM));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    wait_for_stream();
    const int own_start = p.offsets ? segment_start(p.offsets, own, p.M) : 0;
    const int own_stop = p.offsets ? segment_end(p.offsets, p.counts, own, p.M) : p.M;
    int rows[F_GROUPS];             // of experts 32 g + lane: under way during the first pass, looked at behind it
#pragma unroll
    for (int g = 0; g < F_GROUPS; ++g) rows[g] = p.offsets && 32 * g + lane < p.experts ? p.counts[32 * g + lane] : 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (L::kOwnSums && splits > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // this CTA runs
    const uint32_t tmem = *tmem_slot;

    uint32_t amax = 0;
    int s = 0;                      // stage and its phase, of each role
    uint32_t phase = 0, acc_phase = 0;
    uint32_t issued_any = 0, issued_parity = 0;   // producer: the last phase issued on each stage
    bool ok = true, freed = false, first = true;
    auto any_many = [&] {           // whether any expert has rows for a second pass
        int most = rows[0];
#pragma unroll
        for (int g = 1; g < F_GROUPS; ++g) most = max(most, rows[g]);
        return __any_sync(0xFFFFFFFFu, most > TOK) != 0;
    };
    // A pass over a weight tile for up to TOK tokens.  The CTAs of a cluster take the same passes, also after an abort.
    auto pass = [&](int e, int tile, int t0, int stop) {
        const Finish f = finish_at(p, e, (int64_t)tile * F_ROWS + 4 * lane);
        if (!first) {               // the pass before is done with the accumulator and the stages
            tc_fence_before();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (splits == 1) __syncthreads();
            else cluster_sync();
            tc_fence_after();
        }
        const int tokens = min(TOK, stop - t0), boxes = (tokens + 15) / 16;
        if (warp == 0) {
            if (lane == 0) {
                const Source src = source(p, e, tile, t0, tokens);
                for (int kb = kb0; kb < kb1 && ok; ++kb) {
                    if (!mbar_wait(bar_empty + 8 * s, phase ^ 1, abort_flag)) { ok = false; break; }
                    load_stage<TOK>(sbase + s * L::kStage, bar_full + 8 * s, map_w, map_x, src, kb, min(4, steps - kb * 4));
                    issued_any |= 1u << s;
                    issued_parity = (issued_parity & ~(1u << s)) | (phase << s);
                    if (++s == L::kStages) { s = 0; phase ^= 1; }
                }
            }
        } else if (warp == 1) {
            if (lane == 0) {
                const uint32_t idesc = few_idesc(boxes);
                for (int kb = kb0; kb < kb1 && ok; ++kb) {
                    // raised by the scale warps once the stage had landed
                    if (!mbar_wait(bar_sf + 8 * s, phase, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    issue_steps<L::kOffX>(tmem, (sbase + s * L::kStage) >> 4, tmem + L::kSf + s * 32, idesc,
                                          min(4, steps - kb * 4), kb > kb0);
                    tc_commit(bar_empty + 8 * s);
                    if (++s == L::kStages) { s = 0; phase ^= 1; }
                }
                tc_commit(bar_acc);
            }
        } else {
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            for (int kb = kb0; kb < kb1 && ok; ++kb) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * s, phase, abort_flag))) { ok = false; break; }
                scale_stage<TOK>(sbase + s * L::kStage + L::kOffSfw, tmem + lanes + L::kSf + s * 32, t0, lane);
                if (lane == 0) mbar_arrive(bar_sf + 8 * s);
                if (++s == L::kStages) { s = 0; phase ^= 1; }
            }
            (void)mbar_wait(bar_acc, acc_phase, abort_flag);   // run out: the results are wrong and the error word says so
            tc_fence_after();
        }
        acc_phase ^= 1;
        __syncwarp();
        // Shared memory takes the partial sums, [CTA][token][feature], of the tokens that a CTA finishes: all of them, or in
        // a cluster a share.
        int shift = 0;              // a share is 2^shift tokens
        while ((splits << shift) < tokens) ++shift;
        if (splits > 1) {
            // Every CTA of the cluster runs, and its stages (or, with sums of their own, those of the pass before) are free.
            if (L::kOwnSums && first) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            else cluster_sync();
        }
        if (warp >= 2) {
            const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t col = sbase + L::kOffSums + 4 * ((warp & 3) * 32 + lane) + (rank << shift) * F_ROWS * 4;
            for (int b = 0; b < boxes; ++b) {
                uint32_t v[16];
                tc_ld_32x32b_x16(tlane + 16 * b, v);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int t = 16 * b + j;
                    if (t >= tokens) break;
                    const uint32_t at = col + (t & ((1 << shift) - 1)) * F_ROWS * 4;
                    if (splits > 1) store_remote(at, t >> shift, __uint_as_float(v[j]));
                    else asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v[j]) : "memory");
                }
            }
        }
        tc_fence_before();
        if (splits > 1) cluster_sync();
        else __syncthreads();
        if (warp == 1 && !any_many() && !*abort_flag) {   // the only pass: nothing needs tensor memory any more
            freed = true;
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F_TMEM));
        }
        {
            const float4* part = reinterpret_cast<const float4*>(smem + L::kOffSums) + lane;
            const int from = rank << shift, count = min(1 << shift, tokens - from);
            for (int t = warp; t < count; t += F_THREADS / 32) {
                float4 sum = part[t * (F_ROWS / 4)];
                for (int c = 1; c < splits; ++c) {
                    const float4 q = part[((c << shift) + t) * (F_ROWS / 4)];
                    sum.x += q.x;
                    sum.y += q.y;
                    sum.z += q.z;
                    sum.w += q.w;
                }
                finish<ACT>(p, f, t0 + from + t, sum, amax);
            }
        }
        first = false;
    };
    if (own_start < own_stop) pass(own, own_tile, own_start, own_stop);
    // Experts with more rows than one pass takes: their other passes, dealt to all clusters.
    int next = 0;                   // the cluster whose turn it is
#pragma unroll 1
    for (int base = 0; base < (any_many() ? p.experts : 0); base += 32) {
        unsigned more = __ballot_sync(0xFFFFFFFFu, base + lane < p.experts && p.counts[base + lane] > TOK);
        while (more) {
            const int e = base + __ffs(more) - 1;
            more &= more - 1;
            const int start = segment_start(p.offsets, e, p.M), stop = segment_end(p.offsets, p.counts, e, p.M);
            const int64_t count = (int64_t)max((stop - start + TOK - 1) / TOK - 1, 0) * p.tiles;
            for (int64_t i = (unit - next + units) % units; i < count; i += units)
                pass(e, (int)(i % p.tiles), start + (int)(i / p.tiles + 1) * TOK, stop);
            next = (int)((next + count) % units);
        }
    }
    if (p.c_amax) {                 // over the CTA, then one atomic
        __syncwarp();
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, amax);
        if (lane == 0 && m) atomicMax(s_amax, m);
    }
    if (p.offsets && warp >= 2) {
        zero_padding(p, own, own_tile * F_ROWS, own_stop, rank * 4 + warp - 2, splits * 4, lane);
        zero_tail(p, blockIdx.x * 4 + warp - 2, gridDim.x * 4, lane);
    }
    // After an abort, no copy and no MMA may be in flight when memory is released; otherwise every copy was waited for by
    // the scale warps and every MMA by the accumulator's barrier.
    if (*abort_flag) {
        if (warp == 0 && lane == 0) {
            for (int st = 0; st < L::kStages; ++st)
                if (issued_any & (1u << st)) {
                    const unsigned long long w0 = globaltimer();
                    while (!mbar_try(bar_full + 8 * st, (issued_parity >> st) & 1u) && globaltimer() - w0 < kWaitLimitNs) {}
                }
        }
        if (warp == 1 && lane == 0) {
            tc_commit(bar_drain);
            const unsigned long long w0 = globaltimer();
            while (!mbar_try(bar_drain, 0) && globaltimer() - w0 < kWaitLimitNs) {}
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (p.c_amax && threadIdx.x == 0 && *s_amax) atomicMax(p.c_amax, *s_amax);
    if (warp == 1 && !freed) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F_TMEM));
    }
}

// The same where there is enough to do without splitting K: a CTA goes through
// tiles (of features, per expert) one after the other, and the operands of the
// next tiles are on their way while a finished one leaves.  Against a CTA per
// tile: 8 experts of 14336 x 4096 71 -> 56 us, 64 of 2048 x 2048 54 -> 33, 64 of
// 4096 x 1024 75 -> 38, one token through 131072 x 4096 57 -> 50.
// Two accumulators; the epilogue has four warps of its own, each with its 32
// features of 16 tokens at a time turned through 2 KB of shared memory.
constexpr int S_THREADS = 320;
template <int TOK>
struct StreamLayout {
    using L = Layout<TOK>;
    static constexpr int kOffTurn = L::kStages * L::kStage;
    static constexpr int kOffBar = kOffTurn + 4 * 2048;       // full, empty, scales per stage; 2 accumulators full, empty; drain
    static constexpr int kOffMisc = kOffBar + (3 * L::kStages + 5) * 8;
    static constexpr int kBytes = kOffMisc + 16 + 1008;
    static constexpr uint32_t kSf = 2 * TOK;
    static_assert(TOK <= 32 && kSf + L::kStages * 32 <= F_TMEM, "tensor memory");
};

template <int TOK, int ACT>
__global__ void __launch_bounds__(S_THREADS, 2)
gemm_few_stream_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, FewParams p) {
    using L = Layout<TOK>;
    using S = StreamLayout<TOK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + S::kOffBar, bar_empty = bar_full + 8 * L::kStages;
    const uint32_t bar_sf = bar_empty + 8 * L::kStages, bar_acc = bar_sf + 8 * L::kStages;
    const uint32_t bar_free = bar_acc + 16, bar_drain = bar_free + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
    unsigned int* s_amax = reinterpret_cast<unsigned int*>(smem + S::kOffMisc + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = p.tiles * p.experts, stride = gridDim.x;
    const int steps = p.K / 64, blocks = (steps + 3) / 4;

    if (threadIdx.x == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_x);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
            mbar_init(bar_sf + 8 * s, 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc + 8 * b, 1);
            mbar_init(bar_free + 8 * b, 4);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        *s_amax = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(F_TMEM));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    wait_for_stream();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // Every role goes through the same tiles and passes.  A tile's rows are fetched one tile ahead: they are read from
    // global memory, and nothing should wait for that between two tiles.
    auto rows_of = [&](int unit, int& e, int& tile, int& start, int& stop) {
        e = min(unit, units - 1) / p.tiles;
        tile = min(unit, units - 1) - e * p.tiles;
        start = p.offsets ? segment_start(p.offsets, e, p.M) : 0;
        stop = p.offsets ? segment_end(p.offsets, p.counts, e, p.M) : p.M;
    };
    int e1, tile1, start1, stop1;
    rows_of(blockIdx.x, e1, tile1, start1, stop1);
    int s = 0, acc = 0;             // stage and accumulator, and their phases, of each role
    uint32_t phase = 0, acc_phase = 0, amax = 0;
    uint32_t issued_any = 0, issued_parity = 0;   // producer: the last phase issued on each stage
    bool ok = true;
    if (p.offsets && warp >= 6) zero_tail(p, blockIdx.x * 4 + warp - 6, gridDim.x * 4, lane);
    auto pass = [&](int e, int tile, int t0, int stop) {
        Finish f;
        if (warp >= 6) f = finish_at(p, e, tile * F_ROWS + 32 * (warp & 3) + 4 * (lane & 7));
        const int tokens = min(TOK, stop - t0), boxes = (tokens + 15) / 16;
        if (warp == 0) {
            if (lane == 0) {
                const Source src = source(p, e, tile, t0, tokens);
                for (int kb = 0; kb < blocks; ++kb) {
                    if (!mbar_wait(bar_empty + 8 * s, phase ^ 1, abort_flag)) { ok = false; break; }
                    load_stage<TOK>(sbase + s * L::kStage, bar_full + 8 * s, map_w, map_x, src, kb, min(4, steps - kb * 4));
                    issued_any |= 1u << s;
                    issued_parity = (issued_parity & ~(1u << s)) | (phase << s);
                    if (++s == L::kStages) { s = 0; phase ^= 1; }
                }
            }
        } else if (warp == 1) {
            if (lane == 0) {
                ok = mbar_wait(bar_free + 8 * acc, acc_phase ^ 1, abort_flag);
                tc_fence_after();
                const uint32_t idesc = few_idesc(boxes);
                for (int kb = 0; kb < blocks && ok; ++kb) {
                    if (!mbar_wait(bar_sf + 8 * s, phase, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    issue_steps<L::kOffX>(tmem + acc * TOK, (sbase + s * L::kStage) >> 4, tmem + S::kSf + s * 32, idesc,
                                          min(4, steps - kb * 4), kb > 0);
                    tc_commit(bar_empty + 8 * s);
                    if (++s == L::kStages) { s = 0; phase ^= 1; }
                }
                if (ok) tc_commit(bar_acc + 8 * acc);
            }
        } else if (warp < 6) {
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            for (int kb = 0; kb < blocks; ++kb) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * s, phase, abort_flag))) { ok = false; break; }
                scale_stage<TOK>(sbase + s * L::kStage + L::kOffSfw, tmem + lanes + S::kSf + s * 32, t0, lane);
                if (lane == 0) mbar_arrive(bar_sf + 8 * s);
                if (++s == L::kStages) { s = 0; phase ^= 1; }
            }
        } else {
            ok = mbar_wait(bar_acc + 8 * acc, acc_phase, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                tc_fence_after();
                uint32_t v[TOK / 16][16];
#pragma unroll
                for (int b = 0; b < TOK / 16; ++b)
                    tc_ld_32x32b_x16(tmem + acc * TOK + ((uint32_t)((warp & 3) * 32) << 16) + 16 * b, v[b]);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_free + 8 * acc);
                float* turn = reinterpret_cast<float*>(smem + S::kOffTurn) + (warp & 3) * 512;   // [token][feature]
#pragma unroll
                for (int b = 0; b < TOK / 16; ++b) {
                    if (16 * b >= tokens) break;
#pragma unroll
                    for (int j = 0; j < 16; ++j) turn[32 * j + lane] = __uint_as_float(v[b][j]);
                    __syncwarp();
                    for (int t = 16 * b + (lane >> 3); t < min(tokens, 16 * b + 16); t += 4)
                        finish<ACT>(p, f, t0 + t, *reinterpret_cast<const float4*>(turn + 32 * (t - 16 * b) + 4 * (lane & 7)), amax);
                    __syncwarp();
                }
            }
        }
        if (warp < 2) ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    };
    for (int unit = blockIdx.x; unit < units && ok; unit += stride) {
        const int e = e1, tile = tile1, start = start1, stop = stop1;
        rows_of(unit + stride, e1, tile1, start1, stop1);
        if (start < stop) pass(e, tile, start, stop);
        if (p.offsets && warp >= 6) zero_padding(p, e, tile * F_ROWS, stop, warp - 6, 4, lane);
    }
    // Experts with more rows than one pass takes: their other passes, dealt to all CTAs, so that an expert which got most
    // of the tokens does not leave the GPU to a few of them (all of 1024 tokens to one of 64 experts of 2048 x 2048: 125 -> 19 us).
    if (p.offsets) {
        int next = units % stride;      // the CTA whose turn it is
        for (int base = 0; base < p.experts && ok; base += 32) {
            int first = 0, last = 0;
            if (base + lane < p.experts) {
                first = segment_start(p.offsets, base + lane, p.M);
                last = segment_end(p.offsets, p.counts, base + lane, p.M);
            }
            unsigned more = __ballot_sync(0xFFFFFFFFu, last - first > TOK);
            while (more && ok) {
                const int from = __ffs(more) - 1;
                more &= more - 1;
                const int start = __shfl_sync(0xFFFFFFFFu, first, from), stop = __shfl_sync(0xFFFFFFFFu, last, from);
                const int64_t count = (int64_t)((stop - start + TOK - 1) / TOK - 1) * p.tiles;
                for (int64_t i = ((int)blockIdx.x - next + stride) % stride; i < count && ok; i += stride)
                    pass(base + from, (int)(i % p.tiles), start + (int)(i / p.tiles + 1) * TOK, stop);
                next = (int)((next + count) % stride);
            }
        }
    }
    if (p.c_amax && warp >= 6) {
        __syncwarp();
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, amax);
        if (lane == 0 && m) atomicMax(s_amax, m);
    }
    // As above: after an abort, no copy and no MMA may be in flight when memory is released.
    if (*abort_flag) {
        if (warp == 0 && lane == 0) {
            for (int st = 0; st < L::kStages; ++st)
                if (issued_any & (1u << st)) {
                    const unsigned long long w0 = globaltimer();
                    while (!mbar_try(bar_full + 8 * st, (issued_parity >> st) & 1u) && globaltimer() - w0 < kWaitLimitNs) {}
                }
        }
        if (warp == 1 && lane == 0) {
            tc_commit(bar_drain);
            const unsigned long long w0 = globaltimer();
            while (!mbar_try(bar_drain, 0) && globaltimer() - w0 < kWaitLimitNs) {}
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (p.c_amax && threadIdx.x == 0 && *s_amax) atomicMax(p.c_amax, *s_amax);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F_TMEM));
    }
}

typedef void (*FewKernel)(const CUtensorMap, const CUtensorMap, FewParams);

template <int TOK>
FewKernel stream_kernel(int act) {
    switch (act) {
        case ACT_RELU: return gemm_few_stream_kernel<TOK, ACT_RELU>;
        case ACT_RELU2: return gemm_few_stream_kernel<TOK, ACT_RELU2>;
        case ACT_GELU: return gemm_few_stream_kernel<TOK, ACT_GELU>;
        case ACT_GELU_TANH: return gemm_few_stream_kernel<TOK, ACT_GELU_TANH>;
        case ACT_SILU: return gemm_few_stream_kernel<TOK, ACT_SILU>;
        default: return gemm_few_stream_kernel<TOK, ACT_NONE>;
    }
}

template <int TOK>
FewKernel few_kernel(int act) {
    switch (act) {
        case ACT_RELU: return gemm_few_kernel<TOK, ACT_RELU>;
        case ACT_RELU2: return gemm_few_kernel<TOK, ACT_RELU2>;
        case ACT_GELU: return gemm_few_kernel<TOK, ACT_GELU>;
        case ACT_GELU_TANH: return gemm_few_kernel<TOK, ACT_GELU_TANH>;
        case ACT_SILU: return gemm_few_kernel<TOK, ACT_SILU>;
        default: return gemm_few_kernel<TOK, ACT_NONE>;
    }
}

int prepared_sms() {
    static int cached[64];
    static std::mutex mu;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!cached[dev]) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        for (int act = 0; act < kNumActivations; ++act) {
            cudaFuncSetAttribute(few_kernel<16>(act), cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<16>::kBytes);
            cudaFuncSetAttribute(few_kernel<32>(act), cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<32>::kBytes);
            cudaFuncSetAttribute(few_kernel<128>(act), cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<128>::kBytes);
            cudaFuncSetAttribute(stream_kernel<16>(act), cudaFuncAttributeMaxDynamicSharedMemorySize, StreamLayout<16>::kBytes);
            cudaFuncSetAttribute(stream_kernel<32>(act), cudaFuncAttributeMaxDynamicSharedMemorySize, StreamLayout<32>::kBytes);
        }
        cached[dev] = n > 0 ? n : 148;
    }
    return cached[dev];
}

}  // namespace

cudaError_t launch_gemm_few(const GemmExtArgs& g, cudaStream_t s) {
    const int sms = prepared_sms();
    FewParams p{};
    p.sfx = g.sfa;
    p.sfw = g.sfb;
    p.x_gs = g.a_gs;
    p.w_gs = g.b_gs;
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.K = (int)g.K;
    p.chunks_k = (int)mma_chunks_k(g.K);
    p.tiles = (int)ceil_div(g.N, F_ROWS);
    p.sfw_stride = (int64_t)mma_scale_bytes(g.N, g.K);
    p.offsets = g.offsets;
    p.counts = g.counts;
    p.experts = g.offsets ? (int)g.experts : 1;
    p.bias = static_cast<const __nv_bfloat16*>(g.bias);
    p.residual = static_cast<const __nv_bfloat16*>(g.residual);
    p.ldr = g.ldr;
    p.out_bf16 = g.out_bf16;
    p.c = g.c;
    p.ldc = g.ldc;
    p.pre = static_cast<__nv_bfloat16*>(g.pre);
    p.ldp = g.ldp;
    p.c_amax = reinterpret_cast<unsigned int*>(g.c_amax);
    CUtensorMap mw, mx;
    if (!make_code_map(&mw, g.b, p.experts * g.N, g.K, F_ROWS) || !make_code_map(&mx, g.a, g.M, g.K, 16))
        return cudaErrorInvalidValue;
    // The largest cluster whose CTAs are resident together (two to an SM) and have two blocks of K each.
    const int64_t units = (int64_t)p.tiles * p.experts, blocks = ceil_div(g.K, 256);
    int splits = 1;
    while (splits < 8 && units * splits * 2 <= 2 * sms && blocks >= 4 * splits && p.experts <= 32 * F_GROUPS) splits *= 2;
    const int tokens = g.offsets ? (splits > 1 ? 128 : 32) : g.M <= 16 ? 16 : g.M <= 32 ? 32 : 128;
    if (splits == 1 && tokens <= 32) {
        const int grid = (int)(units < 2 * sms ? units : 2 * sms);
        return tokens == 16 ? launch_early(stream_kernel<16>(g.act), grid, S_THREADS, StreamLayout<16>::kBytes, s, 1, mw, mx, p)
                            : launch_early(stream_kernel<32>(g.act), grid, S_THREADS, StreamLayout<32>::kBytes, s, 1, mw, mx, p);
    }
    FewKernel kernel = tokens == 16 ? few_kernel<16>(g.act) : tokens == 32 ? few_kernel<32>(g.act) : few_kernel<128>(g.act);
    const int smem = tokens == 16 ? Layout<16>::kBytes : tokens == 32 ? Layout<32>::kBytes : Layout<128>::kBytes;
    return launch_early(kernel, (unsigned)(units * splits), F_THREADS, smem, s, splits, mw, mx, p);
}

unsigned int* few_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_error_word) == cudaSuccess ? static_cast<unsigned int*>(p) : nullptr;
}

}  // namespace nvfp4
