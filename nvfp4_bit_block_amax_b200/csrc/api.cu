// api.cu -- the C ABI (include/nvfp4.h): argument validation on the host, then
// stream-ordered kernel launches.  Nothing here allocates device memory.
#include <atomic>
#include <cstdint>

#include "../../include/nvfp4.h"
#include "activation.cuh"
#include "internal.h"

using namespace nvfp4;

namespace {

std::atomic<long long> g_launches{0};

static_assert((int)NVFP4_ACT_NONE == ACT_NONE && (int)NVFP4_ACT_RELU == ACT_RELU && (int)NVFP4_ACT_RELU2 == ACT_RELU2 &&
                  (int)NVFP4_ACT_GELU == ACT_GELU && (int)NVFP4_ACT_GELU_TANH == ACT_GELU_TANH &&
                  (int)NVFP4_ACT_SILU == ACT_SILU,
              "the kernels' activations are the header's");

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
// A bf16 matrix: row stride of whole 16-byte units that holds `cols`, base on a 16-byte boundary.
nvfp4_status check_bf16_matrix(const void* p, int64_t ld, int64_t cols) {
    if (!p || ld < cols) return NVFP4_ERR_INVALID_ARG;
    return ld % 8 || !aligned16(p) ? NVFP4_ERR_MISALIGNED : NVFP4_OK;
}

constexpr size_t kWorkspaceBytes = (size_t)kMaxPartials * sizeof(uint32_t);
constexpr int64_t kMaxDim = (int64_t)1 << 31;   // TMA and index arithmetic bound per dimension

nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

nvfp4_status check_quant_common(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose,
                                int rounding, const uint8_t* codes, const uint8_t* scales,
                                const uint8_t* scales_mma, const float* gs, const void* ws, size_t ws_bytes) {
    if (!x || !codes || !gs || (!scales && !scales_mma)) return NVFP4_ERR_INVALID_ARG;
    if (rows < 1 || cols < 1 || ld < cols || rows >= kMaxDim || cols >= kMaxDim) return NVFP4_ERR_INVALID_ARG;
    if ((transpose != 0 && transpose != 1) || (rounding != NVFP4_RNE && rounding != NVFP4_SR))
        return NVFP4_ERR_INVALID_ARG;
    const int64_t qc = transpose ? rows : cols;
    if (qc % 16 != 0 || cols % 8 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (ld % 8 != 0 || !aligned16(x) || !aligned16(codes) || (scales && !aligned16(scales)) ||
        (scales_mma && !aligned16(scales_mma)) || !aligned4(gs))
        return NVFP4_ERR_MISALIGNED;
    if (!ws || ws_bytes < kWorkspaceBytes || !aligned16(ws)) return NVFP4_ERR_WORKSPACE;
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_version(void) { return 101; }

const char* nvfp4_status_string(nvfp4_status s) {
    switch (s) {
        case NVFP4_OK: return "ok";
        case NVFP4_ERR_INVALID_ARG: return "invalid argument";
        case NVFP4_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
        case NVFP4_ERR_MISALIGNED: return "misaligned pointer or stride";
        case NVFP4_ERR_CUDA: return "CUDA error";
        case NVFP4_ERR_TIMEOUT: return "device wait timed out";
        case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
    }
    return "unknown status";
}

size_t nvfp4_workspace_size(int64_t rows, int64_t cols) {
    (void)rows;
    (void)cols;
    return kWorkspaceBytes;
}

size_t nvfp4_mma_scale_bytes(int64_t rows, int64_t k) {
    if (rows < 1 || k < 16 || k % 16) return 0;
    return mma_scale_bytes(rows, k);
}

long long nvfp4_kernel_launches(void) { return g_launches.load(); }

static nvfp4_status quantize_1d_impl(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose, int rht,
                                     uint64_t rht_seed, int rounding, uint64_t sr_seed, uint8_t* codes,
                                     uint8_t* scales, uint8_t* scales_mma, float* global_scale, void* workspace,
                                     size_t ws_bytes, void* stream, const float* given_amax = nullptr,
                                     int rht_order = 16) {
    nvfp4_status st = check_quant_common(x, rows, cols, ld, transpose, rounding, codes, scales, scales_mma,
                                         global_scale, workspace, ws_bytes);
    if (st != NVFP4_OK) return st;
    if (rht) {
        if (rht_order != 16 && rht_order != 32 && rht_order != 64 && rht_order != 128) return NVFP4_ERR_INVALID_ARG;
        if ((transpose ? rows : cols) % rht_order) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    }
    QuantArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.transpose = transpose;
    a.rht = rht;
    a.rht_order = rht_order;
    a.rht_seed = rht_seed;
    a.rounding = rounding;
    a.sr_seed = sr_seed;
    a.codes = codes;
    a.scales = scales;
    a.scales_mma = scales_mma;
    a.global_scale = global_scale;
    a.partials = static_cast<uint32_t*>(workspace);
    a.given_amax = given_amax;
    int n = 0;
    cudaError_t e = launch_quantize_1d(a, static_cast<cudaStream_t>(stream), &n);
    g_launches += n;
    return from_cuda(e);
}

nvfp4_status nvfp4_quantize_1d(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose, int rounding,
                               uint64_t sr_seed, uint8_t* codes, uint8_t* scales, uint8_t* scales_mma,
                               float* global_scale, void* workspace, size_t ws_bytes, void* stream) {
    return quantize_1d_impl(x, rows, cols, ld, transpose, 0, 0, rounding, sr_seed, codes, scales, scales_mma,
                            global_scale, workspace, ws_bytes, stream);
}

nvfp4_status nvfp4_quantize_1d_from_amax(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose,
                                         int rounding, uint64_t sr_seed, const float* amax, uint8_t* codes,
                                         uint8_t* scales, uint8_t* scales_mma, float* global_scale, void* stream) {
    if (!amax) return NVFP4_ERR_INVALID_ARG;
    if (!aligned4(amax)) return NVFP4_ERR_MISALIGNED;
    // no amax pass, so no workspace: the check gets a placeholder it only compares
    return quantize_1d_impl(x, rows, cols, ld, transpose, 0, 0, rounding, sr_seed, codes, scales, scales_mma,
                            global_scale, reinterpret_cast<void*>(uintptr_t(256)), kWorkspaceBytes, stream, amax);
}

nvfp4_status nvfp4_quantize_1d_noalloc(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose,
                                       int rounding, uint64_t sr_seed, uint8_t* codes, uint8_t* scales,
                                       uint8_t* scales_mma, float* global_scale, void* stream) {
    // The argument checks of nvfp4_quantize_1d.  There is no caller workspace
    // here (the scratch is the library's static array), so the workspace check
    // is given a placeholder that is only compared, never dereferenced.
    nvfp4_status st = check_quant_common(x, rows, cols, ld, transpose, rounding, codes, scales, scales_mma,
                                         global_scale, reinterpret_cast<const void*>(uintptr_t(256)),
                                         kWorkspaceBytes);
    if (st != NVFP4_OK) return st;
    QuantArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.transpose = transpose;
    a.rounding = rounding;
    a.sr_seed = sr_seed;
    a.codes = codes;
    a.scales = scales;
    a.scales_mma = scales_mma;
    a.global_scale = global_scale;
    int n = 0;
    bool too_big = false;
    cudaError_t e = launch_quantize_1d_noalloc(a, static_cast<cudaStream_t>(stream), &n, &too_big);
    if (too_big) return NVFP4_ERR_WORKSPACE;
    g_launches += n;
    return from_cuda(e);
}

nvfp4_status nvfp4_rht_quantize_sr(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose,
                                   uint64_t rht_seed, int rounding, uint64_t sr_seed, uint8_t* codes,
                                   uint8_t* scales, uint8_t* scales_mma, float* global_scale, void* workspace,
                                   size_t ws_bytes, void* stream) {
    return quantize_1d_impl(x, rows, cols, ld, transpose, 1, rht_seed, rounding, sr_seed, codes, scales,
                            scales_mma, global_scale, workspace, ws_bytes, stream);
}

nvfp4_status nvfp4_rht_quantize_n(const void* x, int64_t rows, int64_t cols, int64_t ld, int transpose,
                                  int rht_order, uint64_t rht_seed, int rounding, uint64_t sr_seed, uint8_t* codes,
                                  uint8_t* scales, uint8_t* scales_mma, float* global_scale, void* workspace,
                                  size_t ws_bytes, void* stream) {
    return quantize_1d_impl(x, rows, cols, ld, transpose, 1, rht_seed, rounding, sr_seed, codes, scales,
                            scales_mma, global_scale, workspace, ws_bytes, stream, nullptr, rht_order);
}

static nvfp4_status quantize_2d_impl(const void* w, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes_row,
                                     uint8_t* codes_col, uint8_t* scales, uint8_t* scales_mma_row,
                                     uint8_t* scales_mma_col, float* global_scale, void* workspace,
                                     size_t ws_bytes, void* stream, const float* given_amax) {
    if (!w || !codes_row || !global_scale || (!scales && !scales_mma_row && !scales_mma_col))
        return NVFP4_ERR_INVALID_ARG;
    if (rows < 1 || cols < 1 || ld < cols || rows >= kMaxDim || cols >= kMaxDim) return NVFP4_ERR_INVALID_ARG;
    if (rows % 16 || cols % 16) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (ld % 8 || !aligned16(w) || !aligned16(codes_row) || (codes_col && !aligned16(codes_col)) ||
        (scales && !aligned16(scales)) || (scales_mma_row && !aligned16(scales_mma_row)) ||
        (scales_mma_col && !aligned16(scales_mma_col)) || !aligned4(global_scale))
        return NVFP4_ERR_MISALIGNED;
    if (!workspace || ws_bytes < kWorkspaceBytes || !aligned16(workspace)) return NVFP4_ERR_WORKSPACE;
    Quant2dArgs a{};
    a.w = static_cast<const uint16_t*>(w);
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.codes_row = codes_row;
    a.codes_col = codes_col;
    a.scales = scales;
    a.scales_mma_row = scales_mma_row;
    a.scales_mma_col = scales_mma_col;
    a.global_scale = global_scale;
    a.partials = static_cast<uint32_t*>(workspace);
    a.given_amax = given_amax;
    int n = 0;
    cudaError_t e = launch_quantize_2d(a, static_cast<cudaStream_t>(stream), &n);
    g_launches += n;
    return from_cuda(e);
}

nvfp4_status nvfp4_quantize_dual(const void* x, int64_t rows, int64_t cols, int64_t ld, int rounding,
                                 uint64_t sr_seed, uint8_t* codes, uint8_t* scales, uint8_t* scales_mma,
                                 float* global_scale, uint64_t rht_seed, uint64_t sr_seed_t, uint8_t* codes_t,
                                 uint8_t* scales_t, uint8_t* scales_mma_t, float* global_scale_t, void* workspace,
                                 size_t ws_bytes, void* stream) {
    // both halves must pass the single-call checks; the workspace holds two sets of partials
    nvfp4_status st = check_quant_common(x, rows, cols, ld, 0, rounding, codes, scales, scales_mma, global_scale,
                                         workspace, ws_bytes);
    if (st != NVFP4_OK) return st;
    st = check_quant_common(x, rows, cols, ld, 1, rounding, codes_t, scales_t, scales_mma_t, global_scale_t,
                            workspace, ws_bytes);
    if (st != NVFP4_OK) return st;
    if (ws_bytes < 2 * kWorkspaceBytes) return NVFP4_ERR_WORKSPACE;
    QuantArgs r{}, t{};
    r.x = t.x = static_cast<const uint16_t*>(x);
    r.rows = t.rows = rows;
    r.cols = t.cols = cols;
    r.ld = t.ld = ld;
    r.rounding = t.rounding = rounding;
    r.sr_seed = sr_seed;
    r.codes = codes;
    r.scales = scales;
    r.scales_mma = scales_mma;
    r.global_scale = global_scale;
    r.partials = static_cast<uint32_t*>(workspace) + kMaxPartials;
    t.transpose = 1;
    t.rht = 1;
    t.rht_seed = rht_seed;
    t.sr_seed = sr_seed_t;
    t.codes = codes_t;
    t.scales = scales_t;
    t.scales_mma = scales_mma_t;
    t.global_scale = global_scale_t;
    t.partials = static_cast<uint32_t*>(workspace);
    int n = 0;
    cudaError_t e = launch_quantize_dual(r, t, static_cast<cudaStream_t>(stream), &n);
    g_launches += n;
    return from_cuda(e);
}

nvfp4_status nvfp4_quantize_2d(const void* w, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes_row,
                               uint8_t* codes_col, uint8_t* scales, uint8_t* scales_mma_row,
                               uint8_t* scales_mma_col, float* global_scale, void* workspace, size_t ws_bytes,
                               void* stream) {
    return quantize_2d_impl(w, rows, cols, ld, codes_row, codes_col, scales, scales_mma_row, scales_mma_col,
                            global_scale, workspace, ws_bytes, stream, nullptr);
}

nvfp4_status nvfp4_quantize_2d_from_amax(const void* w, int64_t rows, int64_t cols, int64_t ld, const float* amax,
                                         uint8_t* codes_row, uint8_t* codes_col, uint8_t* scales,
                                         uint8_t* scales_mma_row, uint8_t* scales_mma_col, float* global_scale,
                                         void* stream) {
    if (!amax) return NVFP4_ERR_INVALID_ARG;
    if (!aligned4(amax)) return NVFP4_ERR_MISALIGNED;
    return quantize_2d_impl(w, rows, cols, ld, codes_row, codes_col, scales, scales_mma_row, scales_mma_col,
                            global_scale, reinterpret_cast<void*>(uintptr_t(256)), kWorkspaceBytes, stream, amax);
}

nvfp4_status nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int scale_mode,
                              const float* global_scale, int64_t rows, int64_t cols, int out_dtype, void* out,
                              void* stream) {
    if (!codes || !scales || !global_scale || !out) return NVFP4_ERR_INVALID_ARG;
    if (scale_mode != NVFP4_SCALE_1D && scale_mode != NVFP4_SCALE_2D) return NVFP4_ERR_INVALID_ARG;
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (rows < 1 || cols < 1 || rows >= kMaxDim || cols >= kMaxDim) return NVFP4_ERR_INVALID_ARG;
    if (cols % 16 || (scale_mode == NVFP4_SCALE_2D && rows % 16)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(codes) || !aligned16(out) || !aligned4(global_scale)) return NVFP4_ERR_MISALIGNED;
    cudaError_t e = launch_dequantize(codes, scales, scale_mode, global_scale, rows, cols,
                                      out_dtype == NVFP4_OUT_BF16, out, static_cast<cudaStream_t>(stream));
    g_launches += 1;
    return from_cuda(e);
}

static nvfp4_status gemm_impl(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                              const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs, int64_t M,
                              int64_t N, int64_t K, int out_dtype, void* c, int64_t ldc, float* c_amax,
                              void* stream, int mx = 0) {
    if (!a_codes || !a_scales_mma || !b_codes || !b_scales_mma || !c) return NVFP4_ERR_INVALID_ARG;
    if (!mx && (!a_gs || !b_gs)) return NVFP4_ERR_INVALID_ARG;
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (M < 1 || N < 1 || K < 1 || ldc < N || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
        return NVFP4_ERR_INVALID_ARG;
    if (K % 64) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(a_codes) || !aligned16(b_codes) || !aligned16(a_scales_mma) || !aligned16(b_scales_mma) ||
        !aligned16(c) || ldc % 8 || (!mx && (!aligned4(a_gs) || !aligned4(b_gs))))
        return NVFP4_ERR_MISALIGNED;
    GemmArgs g{};
    g.a = a_codes;
    g.sfa = a_scales_mma;
    g.a_gs = a_gs;
    g.b = b_codes;
    g.sfb = b_scales_mma;
    g.b_gs = b_gs;
    g.M = M;
    g.N = N;
    g.K = K;
    g.out_bf16 = out_dtype == NVFP4_OUT_BF16;
    g.c = c;
    g.ldc = ldc;
    g.c_amax = c_amax;
    g.mx = mx;
    if (c_amax) {
        cudaError_t z = cudaMemsetAsync(c_amax, 0, sizeof(float), static_cast<cudaStream_t>(stream));
        if (z != cudaSuccess) return NVFP4_ERR_CUDA;
    }
    cudaError_t e = launch_gemm(g, static_cast<cudaStream_t>(stream));
    g_launches += 1;
    return from_cuda(e);
}

nvfp4_status nvfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                        const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs, int64_t M,
                        int64_t N, int64_t K, int out_dtype, void* c, int64_t ldc, void* stream) {
    return gemm_impl(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, out_dtype, c, ldc, nullptr,
                     stream);
}

nvfp4_status nvfp4_gemm_amax(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                             const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs, int64_t M,
                             int64_t N, int64_t K, int out_dtype, void* c, int64_t ldc, float* c_amax,
                             void* stream) {
    if (!c_amax) return NVFP4_ERR_INVALID_ARG;
    if (!aligned4(c_amax)) return NVFP4_ERR_MISALIGNED;
    return gemm_impl(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, out_dtype, c, ldc, c_amax,
                     stream);
}

nvfp4_status nvfp4_mxfp4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                  uint8_t* scales, uint8_t* scales_mma, void* stream) {
    if (!x || !codes || (!scales && !scales_mma)) return NVFP4_ERR_INVALID_ARG;
    if (rows < 1 || cols < 1 || ld < cols || rows >= kMaxDim || cols >= kMaxDim) return NVFP4_ERR_INVALID_ARG;
    if (cols % 32) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (ld % 8 || !aligned16(x) || !aligned16(codes) || (scales_mma && !aligned16(scales_mma)))
        return NVFP4_ERR_MISALIGNED;
    cudaError_t e = launch_mx_quantize(static_cast<const uint16_t*>(x), rows, cols, ld, codes, scales, scales_mma,
                                       static_cast<cudaStream_t>(stream));
    g_launches += 1;
    return from_cuda(e);
}

nvfp4_status nvfp4_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                    int out_dtype, void* out, void* stream) {
    if (!codes || !scales || !out) return NVFP4_ERR_INVALID_ARG;
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (rows < 1 || cols < 1 || rows >= kMaxDim || cols >= kMaxDim) return NVFP4_ERR_INVALID_ARG;
    if (cols % 32) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(codes) || !aligned16(out)) return NVFP4_ERR_MISALIGNED;
    cudaError_t e = launch_mx_dequantize(codes, scales, rows, cols, out_dtype == NVFP4_OUT_BF16, out,
                                         static_cast<cudaStream_t>(stream));
    g_launches += 1;
    return from_cuda(e);
}

nvfp4_status nvfp4_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales_mma, const uint8_t* b_codes,
                              const uint8_t* b_scales_mma, int64_t M, int64_t N, int64_t K, int out_dtype, void* c,
                              int64_t ldc, void* stream) {
    return gemm_impl(a_codes, a_scales_mma, nullptr, b_codes, b_scales_mma, nullptr, M, N, K, out_dtype, c, ldc,
                     nullptr, stream, 1);
}

// Whether the product for few rows is the faster one (us, it against the large product, on one B200):
//   M x 14336 x 4096     64: 13.8 / 15.8   96: 16.1 / 16.0   128: 17.2 / 16.1   192: 27 / 16
//   M x 28672 x 8192     64: 31.0 / 38.3                     128: 36.8 / 39.3   192: 65 / 40
//   M x 4096 x 14336     64: 14.0 / 31.1                     128: 18.4 / 31.4   192: 28 / 31
//   M x 1024 x 1024      64:  7.5 /  9.4   96:  9.9 /  9.5   128: 10.9 /  9.7   192: 17 / 10
// so up to 128 rows.  How many rows each expert has is not known here, but segments are padded to 128: with
// nvfp4_moe_rows, M / experts is about 127 more than the mean.  Weights with tiles for every CTA, passes of 32 rows;
// mean 16, 32, 40 rows, the same two times:
//   8 experts of 14336 x 4096    58 / 70   59 / 70   97 / 70
//   64 experts of 2048 x 2048    35 / 47   37 / 47   67 / 47
//   64 experts of 4096 x 1024    40 / 65   44 / 66   74 / 66
//   16 experts of 4096 x 4096    33 / 44   35 / 44   56 / 44
// so up to a mean of 32, one pass.  Few and small weights, K split over a cluster, passes of 128; mean 32, 64, 128:
//   1 expert of 14336 x 4096     14 / 17   16 / 18   18 / 18
//   1 expert of 4096 x 1024       8 / 10    9 / 10   11 / 10
//   3 experts of 2048 x 2048      8 / 11    9 / 11   13 / 11
//   8 experts of 1024 x 4096     11 / 15   12 / 15   15 / 15
// so where the rounding of M hides the mean (one expert's 2 to 129 rows are all M = 256), little is lost.
// What M cannot tell: 128 rows an expert are the capacity of up to one copy each (64 experts of 2048 x 2048: 34 / 46),
// but also a caller's own for segments that he knows to be full (97 / 46).  The first is every small batch; the second
// can ask for the large product by a capacity beyond this limit (see nvfp4.h).
static bool few_rows(const GemmExtArgs& g) { return g.experts ? g.M <= (127 + 32) * g.experts + 127 : g.M <= 128; }

static nvfp4_status gemm_ext(GemmExtArgs g, int out_dtype, void* stream) {
    if (!g.a || !g.sfa || !g.a_gs || !g.b || !g.sfb || !g.b_gs || !g.c) return NVFP4_ERR_INVALID_ARG;
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (g.act < 0 || g.act >= kNumActivations) return NVFP4_ERR_INVALID_ARG;
    if (g.M < 1 || g.N < 1 || g.K < 1 || g.ldc < g.N || g.M >= kMaxDim || g.N >= kMaxDim || g.K >= kMaxDim)
        return NVFP4_ERR_INVALID_ARG;
    if ((g.residual && g.ldr < g.N) || (g.pre && g.ldp < g.N)) return NVFP4_ERR_INVALID_ARG;
    if (g.experts && (!g.offsets || !g.counts || g.experts < 1 || g.experts > kMaxExpertsArg ||
                      g.experts * g.N >= kMaxDim || (g.wgrad && g.experts * g.M >= kMaxDim)))
        return NVFP4_ERR_INVALID_ARG;
    if (g.experts && !g.wgrad && g.M > kMaxSortedRows) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (g.K % 64 || (g.experts && (g.wgrad ? g.K : g.M) % 128)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(g.a) || !aligned16(g.b) || !aligned16(g.sfa) || !aligned16(g.sfb) || !aligned16(g.c) || g.ldc % 8 ||
        !aligned4(g.a_gs) || !aligned4(g.b_gs) || !aligned2(g.bias) || !aligned4(g.c_amax) || !aligned4(g.offsets) ||
        !aligned4(g.counts) || (g.residual && (!aligned16(g.residual) || g.ldr % 8)) ||
        (g.pre && (!aligned16(g.pre) || g.ldp % 8)))
        return NVFP4_ERR_MISALIGNED;
    g.out_bf16 = out_dtype == NVFP4_OUT_BF16;
    if (zero_word(g.c_amax, static_cast<cudaStream_t>(stream)) != cudaSuccess) return NVFP4_ERR_CUDA;
    const bool few = !g.wgrad && few_rows(g);
    cudaError_t e = (few ? launch_gemm_few : launch_gemm_ext)(g, static_cast<cudaStream_t>(stream));
    g_launches += g.c_amax ? 2 : 1;
    return from_cuda(e);
}

static GemmExtArgs operands(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                            const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs, int64_t M,
                            int64_t N, int64_t K, void* c, int64_t ldc) {
    GemmExtArgs g{};
    g.a = a_codes;
    g.sfa = a_scales_mma;
    g.a_gs = a_gs;
    g.b = b_codes;
    g.sfb = b_scales_mma;
    g.b_gs = b_gs;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.ldc = ldc;
    return g;
}

nvfp4_status nvfp4_gemm_epilogue(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                                 const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs, int64_t M,
                                 int64_t N, int64_t K, const void* bias, int activation, const void* residual,
                                 int64_t ldr, int out_dtype, void* c, int64_t ldc, void* pre, int64_t ldp,
                                 float* c_amax, void* stream) {
    GemmExtArgs g = operands(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, c, ldc);
    g.bias = bias;
    g.act = activation;
    g.residual = residual;
    g.ldr = ldr;
    g.pre = pre;
    g.ldp = ldp;
    g.c_amax = c_amax;
    return gemm_ext(g, out_dtype, stream);
}

nvfp4_status nvfp4_gemm_grouped(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                                const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs,
                                const int32_t* offsets, const int32_t* counts, int64_t experts, int64_t M, int64_t N,
                                int64_t K, const void* bias, int activation, const void* residual, int64_t ldr,
                                int out_dtype, void* c, int64_t ldc, void* pre, int64_t ldp, float* c_amax,
                                void* stream) {
    if (experts < 1) return NVFP4_ERR_INVALID_ARG;
    GemmExtArgs g = operands(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, c, ldc);
    g.offsets = offsets;
    g.counts = counts;
    g.experts = experts;
    g.bias = bias;
    g.act = activation;
    g.residual = residual;
    g.ldr = ldr;
    g.pre = pre;
    g.ldp = ldp;
    g.c_amax = c_amax;
    return gemm_ext(g, out_dtype, stream);
}

nvfp4_status nvfp4_gemm_grouped_wgrad(const uint8_t* a_codes, const uint8_t* a_scales_mma, const float* a_gs,
                                      const uint8_t* b_codes, const uint8_t* b_scales_mma, const float* b_gs,
                                      const int32_t* offsets, const int32_t* counts, int64_t experts, int64_t M,
                                      int64_t N, int64_t K, int out_dtype, void* c, int64_t ldc, void* stream) {
    if (experts < 1) return NVFP4_ERR_INVALID_ARG;
    GemmExtArgs g = operands(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, c, ldc);
    g.offsets = offsets;
    g.counts = counts;
    g.experts = experts;
    g.wgrad = 1;
    return gemm_ext(g, out_dtype, stream);
}

size_t nvfp4_act_grad_workspace_size(int64_t M, int64_t N) {
    return M < 1 || N < 1 || M >= kMaxDim || N >= kMaxDim ? 0 : act_grad_workspace(M, N);
}

nvfp4_status nvfp4_act_grad(const void* dy, int64_t ldy, const void* z, int64_t ldz, int64_t M, int64_t N,
                            int activation, const int32_t* offsets, const int32_t* counts, int64_t experts, void* dz,
                            int64_t lddz, float* dbias, float* amax, void* workspace, size_t ws_bytes,
                            void* stream) {
    if (activation < 0 || activation >= kNumActivations) return NVFP4_ERR_INVALID_ARG;
    if (M < 1 || N < 1 || M >= kMaxDim || N >= kMaxDim || ceil_div(M, 128) * ceil_div(N, 256) >= kMaxDim)
        return NVFP4_ERR_INVALID_ARG;
    if (experts < 0 || experts > kMaxExpertsArg || (experts && (!offsets || !counts))) return NVFP4_ERR_INVALID_ARG;
    if (experts && M % 128) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    nvfp4_status st = check_bf16_matrix(dy, ldy, N);
    if (st == NVFP4_OK) st = check_bf16_matrix(dz, lddz, N);
    if (st == NVFP4_OK && activation != NVFP4_ACT_NONE) st = check_bf16_matrix(z, ldz, N);
    if (st != NVFP4_OK) return st;
    if (!aligned4(dbias) || !aligned4(amax) || (experts && (!aligned4(offsets) || !aligned4(counts))))
        return NVFP4_ERR_MISALIGNED;
    if (dbias && (!workspace || ws_bytes < nvfp4_act_grad_workspace_size(M, N) || !aligned16(workspace)))
        return NVFP4_ERR_WORKSPACE;
    ActGradArgs a{};
    a.dy = dy;
    a.ldy = ldy;
    a.z = z;
    a.ldz = ldz;
    a.M = M;
    a.N = N;
    a.act = activation;
    a.offsets = experts ? offsets : nullptr;
    a.counts = counts;
    a.experts = experts;
    a.dz = dz;
    a.lddz = lddz;
    a.dbias = dbias;
    a.amax = amax;
    a.workspace = static_cast<float*>(workspace);
    int n = 0;
    cudaError_t e = launch_act_grad(a, static_cast<cudaStream_t>(stream), &n);
    g_launches += n;
    return from_cuda(e);
}

int64_t nvfp4_moe_rows(int64_t copies, int64_t experts) {
    if (copies < 1 || experts < 1 || copies >= kMaxDim || experts > kMaxExpertsArg) return 0;
    return ceil_div(copies + 127 * (copies < experts ? copies : experts), 128) * 128;
}

size_t nvfp4_moe_workspace_size(int64_t copies, int64_t experts) {
    if (copies < 1 || experts < 1 || copies >= kMaxDim || experts > kMaxExpertsArg) return 0;
    return moe_sort_workspace(copies, experts);
}

nvfp4_status nvfp4_moe_sort(const int32_t* expert_ids, int64_t copies, int64_t experts, int64_t rows,
                            int32_t* offsets, int32_t* counts, int32_t* row_copy, int32_t* copy_row, void* workspace,
                            size_t ws_bytes, void* stream) {
    if (!expert_ids || !offsets || !counts || !row_copy || !copy_row) return NVFP4_ERR_INVALID_ARG;
    if (copies < 1 || experts < 1 || rows < 1 || experts > kMaxExpertsArg || copies >= kMaxDim || rows >= kMaxDim ||
        nvfp4_moe_rows(copies, experts) >= kMaxDim)
        return NVFP4_ERR_INVALID_ARG;
    if (rows % 128) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned4(expert_ids) || !aligned4(offsets) || !aligned4(counts) || !aligned4(row_copy) || !aligned4(copy_row))
        return NVFP4_ERR_MISALIGNED;
    if (!workspace || ws_bytes < moe_sort_workspace(copies, experts) || !aligned16(workspace))
        return NVFP4_ERR_WORKSPACE;
    SortArgs a{};
    a.ids = expert_ids;
    a.n = copies;
    a.experts = experts;
    a.rows = rows;
    a.offsets = offsets;
    a.counts = counts;
    a.row_copy = row_copy;
    a.copy_row = copy_row;
    a.workspace = static_cast<int32_t*>(workspace);
    int n = 0;
    cudaError_t e = launch_moe_sort(a, static_cast<cudaStream_t>(stream), &n);
    g_launches += n;
    return from_cuda(e);
}

// Shapes and index arrays of the row movements.
static nvfp4_status check_move(const MoveArgs& a) {
    if (!a.copy_row || a.tokens < 1 || a.topk < 1 || a.rows < 1 || a.cols < 1) return NVFP4_ERR_INVALID_ARG;
    if (a.tokens >= kMaxDim || a.topk >= kMaxDim || a.rows >= kMaxDim || a.cols >= kMaxDim ||
        a.tokens * a.topk >= kMaxDim)
        return NVFP4_ERR_INVALID_ARG;
    if (a.cols % 8) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned4(a.copy_row) || !aligned4(a.row_copy) || !aligned4(a.weights) || !aligned4(a.dweights) ||
        !aligned4(a.amax))
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

static nvfp4_status move_done(cudaError_t e, int launches) {
    g_launches += launches;
    return from_cuda(e);
}

nvfp4_status nvfp4_moe_gather(const void* x, int64_t ldx, int64_t tokens, int64_t topk, int64_t cols,
                              const int32_t* copy_row, const int32_t* row_copy, int64_t rows, void* y, int64_t ldy,
                              float* amax, void* stream) {
    MoveArgs a{};
    a.src = x;
    a.lds = ldx;
    a.dst = y;
    a.ldd = ldy;
    a.copy_row = copy_row;
    a.row_copy = row_copy;
    a.amax = amax;
    a.tokens = tokens;
    a.topk = topk;
    a.rows = rows;
    a.cols = cols;
    if (!row_copy) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status st = check_move(a);
    if (st == NVFP4_OK) st = check_bf16_matrix(x, ldx, cols);
    if (st == NVFP4_OK) st = check_bf16_matrix(y, ldy, cols);
    if (st != NVFP4_OK) return st;
    int n = 0;
    cudaError_t e = launch_moe_gather(a, static_cast<cudaStream_t>(stream), &n);
    return move_done(e, n);
}

nvfp4_status nvfp4_moe_combine(const void* y, int64_t ldy, int64_t rows, int64_t cols, const int32_t* copy_row,
                               const float* weights, const void* residual, int64_t ldr, int64_t tokens, int64_t topk,
                               void* out, int64_t ldo, void* stream) {
    MoveArgs a{};
    a.src = y;
    a.lds = ldy;
    a.other = residual;
    a.ldo = ldr;
    a.dst = out;
    a.ldd = ldo;
    a.copy_row = copy_row;
    a.weights = weights;
    a.tokens = tokens;
    a.topk = topk;
    a.rows = rows;
    a.cols = cols;
    nvfp4_status st = check_move(a);
    if (st == NVFP4_OK) st = check_bf16_matrix(y, ldy, cols);
    if (st == NVFP4_OK) st = check_bf16_matrix(out, ldo, cols);
    if (st == NVFP4_OK && residual) st = check_bf16_matrix(residual, ldr, cols);
    if (st != NVFP4_OK) return st;
    int n = 0;
    cudaError_t e = launch_moe_combine(a, static_cast<cudaStream_t>(stream), &n);
    return move_done(e, n);
}

nvfp4_status nvfp4_moe_combine_grad(const void* dout, int64_t ldo, const void* y, int64_t ldy, int64_t tokens,
                                    int64_t topk, int64_t cols, const int32_t* copy_row, const int32_t* row_copy,
                                    int64_t rows, const float* weights, void* dy, int64_t lddy, float* dweights,
                                    float* amax, void* stream) {
    MoveArgs a{};
    a.src = dout;
    a.lds = ldo;
    a.other = y;
    a.ldo = ldy;
    a.dst = dy;
    a.ldd = lddy;
    a.copy_row = copy_row;
    a.row_copy = row_copy;
    a.weights = weights;
    a.dweights = dweights;
    a.amax = amax;
    a.tokens = tokens;
    a.topk = topk;
    a.rows = rows;
    a.cols = cols;
    if (!row_copy) return NVFP4_ERR_INVALID_ARG;
    nvfp4_status st = check_move(a);
    if (st == NVFP4_OK) st = check_bf16_matrix(dout, ldo, cols);
    if (st == NVFP4_OK) st = check_bf16_matrix(dy, lddy, cols);
    if (st == NVFP4_OK && dweights) st = check_bf16_matrix(y, ldy, cols);
    if (st != NVFP4_OK) return st;
    int n = 0;
    cudaError_t e = launch_moe_combine_grad(a, static_cast<cudaStream_t>(stream), &n);
    return move_done(e, n);
}

nvfp4_status nvfp4_scales_to_mma(const uint8_t* scales, int scale_mode, int64_t rows, int64_t k,
                                 uint8_t* scales_mma, void* stream) {
    if (!scales || !scales_mma) return NVFP4_ERR_INVALID_ARG;
    if (scale_mode != NVFP4_SCALE_1D && scale_mode != NVFP4_SCALE_2D) return NVFP4_ERR_INVALID_ARG;
    if (rows < 1 || k < 16 || rows >= kMaxDim || k >= kMaxDim) return NVFP4_ERR_INVALID_ARG;
    if (k % 16 || (scale_mode == NVFP4_SCALE_2D && rows % 16)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    cudaError_t e = launch_scales_to_mma(scales, scale_mode, rows, k, scales_mma, static_cast<cudaStream_t>(stream));
    g_launches += 1;
    return from_cuda(e);
}

nvfp4_status nvfp4_selftest_wait_timeout(uint64_t limit_ns, void* stream) {
    if (limit_ns < 1000 || limit_ns > 2000000000ull) return NVFP4_ERR_INVALID_ARG;
    g_launches.fetch_add(1);
    return launch_wait_selftest((unsigned long long)limit_ns, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_get_error(void* stream) {
    cudaError_t err = cudaSuccess;
    const unsigned int w = read_and_clear_error_word(static_cast<cudaStream_t>(stream), &err);
    if (err != cudaSuccess) return NVFP4_ERR_CUDA;
    return w ? NVFP4_ERR_TIMEOUT : NVFP4_OK;
}

}  // extern "C"
