// capi.cu — the extern "C" boundary declared in include/fp4.h: host-side
// validation of every argument, then stream-ordered launches.  No entry point
// allocates or frees device memory or synchronizes the host (except
// fp4_check_device_status, which is documented to).
#include <math.h>

#include <atomic>

#include "kv.cuh"

namespace fp4 {
cudaError_t launch_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld, int fmt,
                            int hk, float ck, int round_away, int mx_floor, int mse, int gscale_given,
                            uint8_t *q, uint8_t *s, float *gscale, int sms, cudaStream_t st, bool pdl,
                            uint32_t *res);
cudaError_t launch_dequantize(const uint8_t *q, const uint8_t *s, const float *gscale, int64_t rows,
                              int64_t cols, int fmt, int hk, float ck, int bf16out, void *out,
                              int sms, cudaStream_t st, const uint32_t *res);
cudaError_t launch_gemm(const uint8_t *Aq, const uint8_t *As, const float *gA, const uint8_t *Wq,
                        const uint8_t *Ws, const float *gW, int64_t M, int64_t N, int64_t K,
                        int fmt, int bf16out, void *C, int64_t ldc, void *ws, size_t ws_bytes,
                        int sms, cudaStream_t st, int *timeout_flag_out, bool pdl, unsigned *counters,
                        bool w_before_wait);
cudaError_t launch_act_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld, int fmt, int hk, float ck,
                                int round_away, int mx_floor, int gscale_given, uint8_t *q, uint8_t *s, float *gscale,
                                unsigned *zero, int nzero, int early, cudaStream_t st);
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt, int sms);
cudaError_t launch_gemm_quantized(const uint8_t *Aq, const uint8_t *As, const float *gA, const uint8_t *Wq,
                                  const uint8_t *Ws, const float *gW, int64_t M, int64_t N, int64_t K, int fmt,
                                  int out_fmt, int round_away, int mx_floor, const float *gC, uint8_t *Cq, uint8_t *Cs,
                                  int sms, cudaStream_t st);
cudaError_t launch_mx_to_nv_scales(const uint8_t *s_mx, int64_t rows, int64_t cols, uint8_t *s_nv, float *gscale,
                                   int sms, cudaStream_t st);
size_t nv_refine_workspace_bytes(int64_t rows, int64_t cols);
cudaError_t launch_nv_refine(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld, int hk, float ck,
                             int round_away, int rounds, uint8_t *q, uint8_t *s, void *ws, float *gscale, int sms,
                             cudaStream_t st);
cudaError_t launch_linear_fused(const uint16_t *x, int64_t ldx, int64_t M, int64_t K, int fmt, int hk, float ck,
                                int round_away, int mx_floor, const float *gA, const uint8_t *Wq, const uint8_t *Ws,
                                const float *gW, int64_t N, int bf16out, void *C, int64_t ldc, int sms, cudaStream_t st,
                                bool w_before_wait, bool residual, bool *taken);
cudaError_t launch_kv_append(const KvView &c, int dim, int fmt, int hk, float ck, const uint16_t *k, int64_t k_tok,
                             int64_t k_head, const uint16_t *v, int64_t v_tok, int64_t v_head, const int64_t *slots,
                             int64_t tokens, int round_away, int mx_floor, int sms, cudaStream_t st, bool *too_many);
cudaError_t launch_kv_gather(const KvView &c, int dim, int fmt, int hk, float ck, const int64_t *slots, int64_t tokens,
                             int bf16out, void *k, void *v, int sms, cudaStream_t st, bool *too_many);
size_t paged_attention_workspace_bytes(int64_t batch, int q_heads, int kv_heads, int dim, int64_t max_len, int64_t window,
                                       int sms);
cudaError_t launch_paged_attention(const KvView &c, int dim, int fmt, int hk, float ck, const uint16_t *q, int64_t batch,
                                   int q_heads, int64_t q_b, int64_t q_h, const int32_t *table, int64_t table_b,
                                   int64_t table_cols, const int32_t *lens, int64_t max_len, float scale, int64_t window,
                                   int bf16out, void *out, float *lse, void *ws, int sms, cudaStream_t st);
cudaError_t launch_linear_w4a16(const uint16_t *x, int64_t ldx, int64_t M, int64_t K, int fmt, int hk, float ck,
                                const uint8_t *Wq, const uint8_t *Ws, const float *gW, int64_t N, int bf16out, void *C,
                                int64_t ldc, int w_early, void *ws, int sms, cudaStream_t st);
size_t linear_w4a16_workspace_bytes(int64_t M, int64_t N, int64_t K, int cols, bool rotated, int sms);
cudaError_t read_and_clear_device_errors(cudaStream_t st, unsigned int *err);
static std::atomic<uint64_t> g_launches{0};
void count_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }
}  // namespace fp4

namespace {

int sm_count()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Format and block pairs of the quantizer; FP4_MXFP4 with block 16 is
// FP4_MXFP4_16 (norm_fmt).
bool valid_fmt(int fmt, int block)
{
    return (fmt == FP4_MXFP4 && (block == 32 || block == 16)) || (fmt == FP4_NVFP4 && block == 16) ||
           (fmt == FP4_MXFP4_16 && block == 16);
}

int norm_fmt(int fmt, int block) { return (fmt == FP4_MXFP4 && block == 16) ? FP4_MXFP4_16 : fmt; }

// Formats of the product (the block size follows from the format).
bool valid_gemm_fmt(int fmt) { return fmt == FP4_MXFP4 || fmt == FP4_NVFP4 || fmt == FP4_MXFP4_16; }

bool valid_k(int k) { return k == 0 || k == 16 || k == 32 || k == 64 || k == 128; }

// The streaming kernels index 32-element units with 32-bit integers: 2^32
// units are 2^37 elements, more than device memory holds as bf16.
bool too_many_units(int64_t rows, int64_t cols) { return cols > 0 && rows > ((int64_t(1) << 32) - 1) / (cols / 32 > 0 ? cols / 32 : 1); }

// RN_fp32(1/sqrt(k)): the double quotient is within 2^-52 relative of the
// exact value, far inside half an fp32 ulp, so rounding it once to fp32 gives
// the correctly rounded constant.
float hadamard_constant(int k) { return k ? (float)(1.0 / sqrt((double)k)) : 1.0f; }

// Sizes of a paged cache that the kernels take.
fp4_status kv_geometry(int64_t num_pages, int page_size, int kv_heads, int head_dim, int fmt, int hadamard_k)
{
    if (num_pages < 0 || kv_heads < 1) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt) || !valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
        return FP4_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP4_ERR_UNSUPPORTED;
    if (hadamard_k && head_dim % hadamard_k) return FP4_ERR_UNSUPPORTED;
    if (kv_heads > 65535 || num_pages > (int64_t(1) << 31) - 1) return FP4_ERR_UNSUPPORTED;
    // head rows have 32-bit numbers: 2^32 of the smallest are more than device memory holds
    if (num_pages * kv_heads > ((int64_t(1) << 32) - 1) / page_size) return FP4_ERR_UNSUPPORTED;
    return FP4_OK;
}

// The kernels' view of a cache.
fp4_status kv_view(const fp4_kv_cache *cache, fp4::KvView &c)
{
    if (!cache) return FP4_ERR_INVALID_ARG;
    const fp4_status st = kv_geometry(cache->num_pages, cache->page_size, cache->kv_heads, cache->head_dim, cache->fmt,
                                      cache->hadamard_k);
    if (st != FP4_OK) return st;
    if (!cache->kq || !cache->ks || !cache->vq || !cache->vs) return FP4_ERR_INVALID_ARG;
    if (cache->fmt == FP4_NVFP4 && (!cache->gk || !cache->gv)) return FP4_ERR_INVALID_ARG;
    if (!aligned(cache->kq, 16) || !aligned(cache->ks, 16) || !aligned(cache->vq, 16) || !aligned(cache->vs, 16) ||
        !aligned(cache->gk, 4) || !aligned(cache->gv, 4))
        return FP4_ERR_ALIGNMENT;
    int shift = 4;
    while ((1 << shift) < cache->page_size) shift++;
    c = {cache->kq, cache->ks, cache->vq, cache->vs, cache->gk, cache->gv, cache->num_pages, shift, cache->kv_heads};
    return FP4_OK;
}

fp4_status attention_sizes(int64_t batch, int q_heads, int kv_heads, int head_dim, int64_t max_seq_len, int64_t window)
{
    if (batch < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || max_seq_len < 1 || window < 0)
        return FP4_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP4_ERR_UNSUPPORTED;
    if (batch > 65535 || q_heads > 65535 || max_seq_len > (1 << 30)) return FP4_ERR_UNSUPPORTED;
    return FP4_OK;
}

}  // namespace

extern "C" {

const char *fp4_status_string(fp4_status st)
{
    switch (st) {
    case FP4_OK: return "FP4_OK";
    case FP4_ERR_INVALID_ARG: return "FP4_ERR_INVALID_ARG: invalid argument";
    case FP4_ERR_UNSUPPORTED: return "FP4_ERR_UNSUPPORTED: shape or format not supported";
    case FP4_ERR_ALIGNMENT: return "FP4_ERR_ALIGNMENT: pointer or stride misaligned";
    case FP4_ERR_CUDA: return "FP4_ERR_CUDA: CUDA runtime error";
    case FP4_ERR_TIMEOUT: return "FP4_ERR_TIMEOUT: a kernel gave up a bounded wait";
    }
    return "unknown fp4_status";
}

fp4_status fp4_quantize_sizes(int64_t rows, int64_t cols, int fmt, int block, size_t *q_bytes,
                              size_t *s_bytes)
{
    if (rows < 0 || cols < 0 || !q_bytes || !s_bytes) return FP4_ERR_INVALID_ARG;
    if (!valid_fmt(fmt, block)) return FP4_ERR_UNSUPPORTED;
    if (cols % block) return FP4_ERR_UNSUPPORTED;
    // byte counts must fit in 63 bits: rows * cols/2 and the padded scale tile
    if (rows > 0 && cols / 2 > (INT64_MAX - 127) / rows) return FP4_ERR_INVALID_ARG;
    const int64_t nkb = cols / block;
    if ((rows + 127) / 128 * 128 > 0 && (nkb + 3) / 4 * 4 > INT64_MAX / ((rows + 127) / 128 * 128))
        return FP4_ERR_INVALID_ARG;
    *q_bytes = (size_t)(rows * (cols / 2));
    *s_bytes = (size_t)(((rows + 127) / 128 * 128) * ((nkb + 3) / 4 * 4));
    return FP4_OK;
}

static fp4_status quantize_impl(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int fmt, int block,
                                int hadamard_k, const fp4_opts *opts, uint8_t *q, uint8_t *s, float *gscale,
                                uint32_t *res, bool with_res, void *stream)
{
    fp4_opts o = {FP4_ROUND_EVEN, FP4_MX_SCALE_CEIL, 0, FP4_SCALE_ABSMAX, 0};
    if (opts) o = *opts;
    if (rows < 0 || cols < 0 || ld_x < cols) return FP4_ERR_INVALID_ARG;
    if (o.round != FP4_ROUND_EVEN && o.round != FP4_ROUND_AWAY) return FP4_ERR_INVALID_ARG;
    if (o.mx_scale_rule != FP4_MX_SCALE_CEIL && o.mx_scale_rule != FP4_MX_SCALE_FLOOR)
        return FP4_ERR_INVALID_ARG;
    if (o.scale_search != FP4_SCALE_ABSMAX && o.scale_search != FP4_SCALE_MSE) return FP4_ERR_INVALID_ARG;
    if (with_res && o.scale_search != FP4_SCALE_ABSMAX) return FP4_ERR_UNSUPPORTED;
    if (!valid_fmt(fmt, block) || !valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    fmt = norm_fmt(fmt, block);
    if (cols % 32 || (hadamard_k && cols % hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (too_many_units(rows, cols)) return FP4_ERR_UNSUPPORTED;
    const bool empty = rows == 0 || cols == 0;
    if (fmt == FP4_NVFP4 && !gscale) return FP4_ERR_INVALID_ARG;
    if (!empty && (!x || !q || !s || (with_res && !res))) return FP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x % 8) || !aligned(q, 16) || !aligned(s, 16)) return FP4_ERR_ALIGNMENT;
    if ((gscale && !aligned(gscale, 4)) || (res && !aligned(res, 4))) return FP4_ERR_ALIGNMENT;
    if (empty && fmt != FP4_NVFP4) return FP4_OK;
    cudaError_t e = fp4::launch_quantize(static_cast<const uint16_t *>(x), rows, cols, ld_x, fmt,
                                         hadamard_k, hadamard_constant(hadamard_k),
                                         o.round == FP4_ROUND_AWAY, o.mx_scale_rule == FP4_MX_SCALE_FLOOR,
                                         o.scale_search == FP4_SCALE_MSE, o.gscale_given, q, s, gscale, sm_count(),
                                         static_cast<cudaStream_t>(stream), true, with_res ? res : nullptr);
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int fmt, int block,
                        int hadamard_k, const fp4_opts *opts, uint8_t *q, uint8_t *s, float *gscale,
                        void *stream)
{
    return quantize_impl(x, rows, cols, ld_x, fmt, block, hadamard_k, opts, q, s, gscale, nullptr, false, stream);
}

fp4_status fp4_quantize_residual(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int fmt, int block,
                                 int hadamard_k, const fp4_opts *opts, uint8_t *q, uint8_t *s, float *gscale,
                                 uint32_t *res, void *stream)
{
    return quantize_impl(x, rows, cols, ld_x, fmt, block, hadamard_k, opts, q, s, gscale, res, true, stream);
}

static fp4_status dequantize_impl(const uint8_t *q, const uint8_t *s, const float *gscale, const uint32_t *res,
                                  bool with_res, int64_t rows, int64_t cols, int fmt, int block, int hadamard_k,
                                  int out_dtype, void *out, void *stream)
{
    if (rows < 0 || cols < 0) return FP4_ERR_INVALID_ARG;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (!valid_fmt(fmt, block) || !valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    fmt = norm_fmt(fmt, block);
    if (cols % 32 || (hadamard_k && cols % hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (too_many_units(rows, cols)) return FP4_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return FP4_OK;
    if (!q || !s || !out || (fmt == FP4_NVFP4 && !gscale) || (with_res && !res)) return FP4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(s, 16) || !aligned(out, 16) || (res && !aligned(res, 4)))
        return FP4_ERR_ALIGNMENT;
    cudaError_t e = fp4::launch_dequantize(q, s, gscale, rows, cols, fmt, hadamard_k,
                                           hadamard_constant(hadamard_k), out_dtype == FP4_OUT_BF16,
                                           out, sm_count(), static_cast<cudaStream_t>(stream),
                                           with_res ? res : nullptr);
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_dequantize(const uint8_t *q, const uint8_t *s, const float *gscale, int64_t rows,
                          int64_t cols, int fmt, int block, int hadamard_k, int out_dtype, void *out,
                          void *stream)
{
    return dequantize_impl(q, s, gscale, nullptr, false, rows, cols, fmt, block, hadamard_k, out_dtype, out,
                           stream);
}

fp4_status fp4_dequantize_residual(const uint8_t *q, const uint8_t *s, const float *gscale, const uint32_t *res,
                                   int64_t rows, int64_t cols, int fmt, int block, int hadamard_k, int out_dtype,
                                   void *out, void *stream)
{
    return dequantize_impl(q, s, gscale, res, true, rows, cols, fmt, block, hadamard_k, out_dtype, out, stream);
}

fp4_status fp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int fmt, size_t *bytes)
{
    if (M < 0 || N < 0 || K < 0 || !bytes) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;  // as fp4_gemm
    *bytes = fp4::gemm_workspace_bytes(M, N, K, fmt, sm_count());
    return FP4_OK;
}

fp4_status fp4_gemm(const uint8_t *Aq, const uint8_t *As, const float *gA, const uint8_t *Wq,
                    const uint8_t *Ws, const float *gW, int64_t M, int64_t N, int64_t K, int fmt,
                    int out_dtype, void *C, int64_t ldc, void *workspace, size_t ws_bytes, void *stream)
{
    if (M < 0 || N < 0 || K < 0 || ldc < N) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (K % 32) return FP4_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP4_OK;
    if (!Aq || !As || !Wq || !Ws || !C) return FP4_ERR_INVALID_ARG;
    if (fmt == FP4_NVFP4 && (!gA || !gW)) return FP4_ERR_INVALID_ARG;
    if (!aligned(Aq, 16) || !aligned(Wq, 16) || !aligned(As, 16) || !aligned(Ws, 16) || !aligned(C, 16))
        return FP4_ERR_ALIGNMENT;
    const int sms = sm_count();
    const size_t need = fp4::gemm_workspace_bytes(M, N, K, fmt, sms);
    if (need > 0 && (!workspace || ws_bytes < need)) return FP4_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 16)) return FP4_ERR_ALIGNMENT;
    int bad = 0;
    cudaError_t e = fp4::launch_gemm(Aq, As, gA, Wq, Ws, gW, M, N, K, fmt, out_dtype == FP4_OUT_BF16,
                                     C, ldc, workspace, ws_bytes, sms,
                                     static_cast<cudaStream_t>(stream), &bad, true, nullptr, false);
    if (bad) return FP4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // extern "C"

namespace {
struct LinearLayout {
    size_t aq, as, ga, gemm, counters, total;
};

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

LinearLayout linear_layout(int64_t M, int64_t N, int64_t K, int fmt, int sms)
{
    LinearLayout L;
    const int64_t nkb = K / (fmt == FP4_MXFP4 ? 32 : 16);
    L.aq = 0;
    L.as = round256((size_t)(M * (K / 2)));
    L.ga = L.as + round256((size_t)(((M + 127) / 128 * 128) * ((nkb + 3) / 4 * 4)));
    L.gemm = L.ga + 256;
    L.counters = L.gemm + round256(fp4::gemm_workspace_bytes(M, N, K, fmt, sms));
    // per-tile arrival counters of the decode kernel's fused reduction
    L.total = L.counters + round256((size_t)((N + 127) / 128) * sizeof(unsigned));
    return L;
}
}  // namespace

extern "C" {

fp4_status fp4_linear_workspace_size(int64_t M, int64_t N, int64_t K, int fmt, size_t *bytes)
{
    if (M < 0 || N < 0 || K < 0 || !bytes) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;  // as fp4_gemm
    *bytes = linear_layout(M, N, K, fmt, sm_count()).total;
    return FP4_OK;
}

fp4_status fp4_linear(const void *x, int64_t M, int64_t K, int64_t ld_x, int fmt, int hadamard_k,
                      const fp4_opts *opts, const float *gA, const uint8_t *Wq, const uint8_t *Ws,
                      const float *gW, int64_t N, int out_dtype, void *C, int64_t ldc,
                      void *workspace, size_t ws_bytes, void *stream)
{
    fp4_opts o = {FP4_ROUND_EVEN, FP4_MX_SCALE_CEIL, 0, FP4_SCALE_ABSMAX, 0};
    if (opts) o = *opts;
    if (M < 0 || N < 0 || K < 0 || ld_x < K || ldc < N) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (o.round != FP4_ROUND_EVEN && o.round != FP4_ROUND_AWAY) return FP4_ERR_INVALID_ARG;
    if (o.mx_scale_rule != FP4_MX_SCALE_CEIL && o.mx_scale_rule != FP4_MX_SCALE_FLOOR) return FP4_ERR_INVALID_ARG;
    if (o.scale_search != FP4_SCALE_ABSMAX) return FP4_ERR_UNSUPPORTED;  // absmax scales only
    if (o.weights_static != 0 && o.weights_static != 1) return FP4_ERR_INVALID_ARG;
    if (!valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (K % 32 || (hadamard_k && K % hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (too_many_units(M, K)) return FP4_ERR_UNSUPPORTED;
    if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;  // as fp4_gemm
    if (M == 0 || N == 0) return FP4_OK;
    if (!x || !Wq || !Ws || !C || !workspace) return FP4_ERR_INVALID_ARG;
    if (fmt == FP4_NVFP4 && !gW) return FP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x % 8) || !aligned(Wq, 16) || !aligned(Ws, 16) || !aligned(C, 16) ||
        !aligned(workspace, 256))
        return FP4_ERR_ALIGNMENT;
    const int sms = sm_count();
    const LinearLayout L = linear_layout(M, N, K, fmt, sms);
    if (ws_bytes < L.total) return FP4_ERR_INVALID_ARG;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    uint8_t *aq = base + L.aq, *as = base + L.as;
    float *ga = (fmt == FP4_NVFP4 && gA) ? const_cast<float *>(gA) : reinterpret_cast<float *>(base + L.ga);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool decode = M <= 16;
    unsigned *counters = decode ? reinterpret_cast<unsigned *>(base + L.counters) : nullptr;
    cudaError_t e;
    if (decode) {
        // one launch: the decode kernel quantizes the activations itself
        // (whole-tile and cluster work splits)
        bool taken = false;
        e = fp4::launch_linear_fused(static_cast<const uint16_t *>(x), ld_x, M, K, fmt, hadamard_k,
                                     hadamard_constant(hadamard_k), o.round == FP4_ROUND_AWAY,
                                     o.mx_scale_rule == FP4_MX_SCALE_FLOOR, fmt == FP4_NVFP4 ? gA : nullptr, Wq, Ws, gW,
                                     N, out_dtype == FP4_OUT_BF16, C, ldc, sms, st, o.weights_static != 0, false,
                                     &taken);
        if (taken) return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
        // otherwise two launches: one cluster quantizes the activations (and
        // zeroes the tile counters); the split-K kernel streams W meanwhile
        // and reduces.
        e = fp4::launch_act_quantize(static_cast<const uint16_t *>(x), M, K, ld_x, fmt, hadamard_k,
                                     hadamard_constant(hadamard_k), o.round == FP4_ROUND_AWAY,
                                     o.mx_scale_rule == FP4_MX_SCALE_FLOOR, gA != nullptr, aq, as, ga, counters,
                                     (int)((N + 127) / 128), o.weights_static != 0, st);
    } else {
        e = fp4::launch_quantize(static_cast<const uint16_t *>(x), M, K, ld_x, fmt, hadamard_k,
                                 hadamard_constant(hadamard_k), o.round == FP4_ROUND_AWAY,
                                 o.mx_scale_rule == FP4_MX_SCALE_FLOOR, 0, gA != nullptr, aq, as, ga, sms, st, true,
                                 nullptr);
    }
    if (e != cudaSuccess) return FP4_ERR_CUDA;
    int bad = 0;
    e = fp4::launch_gemm(aq, as, ga, Wq, Ws, gW, M, N, K, fmt, out_dtype == FP4_OUT_BF16, C, ldc, base + L.gemm,
                         L.counters - L.gemm, sms, st, &bad, true, counters, decode);
    if (bad) return FP4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_linear_residual(const void *x, int64_t M, int64_t K, int64_t ld_x, int fmt, int hadamard_k,
                               const fp4_opts *opts, const float *gA, const uint8_t *Wq, const uint8_t *Ws,
                               const float *gW, int64_t N, int out_dtype, void *C, int64_t ldc, void *stream)
{
    fp4_opts o = {FP4_ROUND_EVEN, FP4_MX_SCALE_CEIL, 0, FP4_SCALE_ABSMAX, 0};
    if (opts) o = *opts;
    if (M < 0 || N < 0 || K < 0 || ld_x < K || ldc < N) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (o.round != FP4_ROUND_EVEN && o.round != FP4_ROUND_AWAY) return FP4_ERR_INVALID_ARG;
    if (o.mx_scale_rule != FP4_MX_SCALE_CEIL && o.mx_scale_rule != FP4_MX_SCALE_FLOOR) return FP4_ERR_INVALID_ARG;
    if (o.scale_search != FP4_SCALE_ABSMAX) return FP4_ERR_UNSUPPORTED;
    if (o.weights_static != 0 && o.weights_static != 1) return FP4_ERR_INVALID_ARG;
    if (!valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (K % 32 || (hadamard_k && K % hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (M > 16 || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;  // the decode product only
    if (M == 0 || N == 0) return FP4_OK;
    if (K == 0) return FP4_ERR_UNSUPPORTED;
    if (!x || !Wq || !Ws || !C) return FP4_ERR_INVALID_ARG;
    if (fmt == FP4_NVFP4 && !gW) return FP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x % 8) || !aligned(Wq, 16) || !aligned(Ws, 16) || !aligned(C, 16))
        return FP4_ERR_ALIGNMENT;
    if (gA && !aligned(gA, 4)) return FP4_ERR_ALIGNMENT;
    bool taken = false;
    const cudaError_t e = fp4::launch_linear_fused(
        static_cast<const uint16_t *>(x), ld_x, M, K, fmt, hadamard_k, hadamard_constant(hadamard_k),
        o.round == FP4_ROUND_AWAY, o.mx_scale_rule == FP4_MX_SCALE_FLOOR, fmt == FP4_NVFP4 ? gA : nullptr, Wq, Ws, gW,
        N, out_dtype == FP4_OUT_BF16, C, ldc, sm_count(), static_cast<cudaStream_t>(stream), o.weights_static != 0, true,
        &taken);
    if (!taken) return FP4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_gemm_quantized(const uint8_t *Aq, const uint8_t *As, const float *gA, const uint8_t *Wq,
                              const uint8_t *Ws, const float *gW, int64_t M, int64_t N, int64_t K, int fmt,
                              int out_fmt, const fp4_opts *opts, const float *gC, uint8_t *Cq, uint8_t *Cs,
                              void *stream)
{
    fp4_opts o = {FP4_ROUND_EVEN, FP4_MX_SCALE_CEIL, 0, FP4_SCALE_ABSMAX, 0};
    if (opts) o = *opts;
    if (M < 0 || N < 0 || K < 0) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (out_fmt != FP4_MXFP4 && out_fmt != FP4_NVFP4) return FP4_ERR_UNSUPPORTED;
    if (o.round != FP4_ROUND_EVEN && o.round != FP4_ROUND_AWAY) return FP4_ERR_INVALID_ARG;
    if (o.mx_scale_rule != FP4_MX_SCALE_CEIL && o.mx_scale_rule != FP4_MX_SCALE_FLOOR) return FP4_ERR_INVALID_ARG;
    if (o.scale_search != FP4_SCALE_ABSMAX) return FP4_ERR_UNSUPPORTED;  // absmax scales only
    if (M <= 16 || K % 32 || N % 128) return FP4_ERR_UNSUPPORTED;
    if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;
    if (!Aq || !As || !Wq || !Ws || !Cq || !Cs) return FP4_ERR_INVALID_ARG;
    if (fmt == FP4_NVFP4 && (!gA || !gW)) return FP4_ERR_INVALID_ARG;
    if (out_fmt == FP4_NVFP4 && !gC) return FP4_ERR_INVALID_ARG;
    if (!aligned(Aq, 16) || !aligned(Wq, 16) || !aligned(As, 16) || !aligned(Ws, 16) || !aligned(Cq, 16) ||
        !aligned(Cs, 16))
        return FP4_ERR_ALIGNMENT;
    if (gC && !aligned(gC, 4)) return FP4_ERR_ALIGNMENT;
    cudaError_t e = fp4::launch_gemm_quantized(Aq, As, gA, Wq, Ws, gW, M, N, K, fmt, out_fmt,
                                               o.round == FP4_ROUND_AWAY, o.mx_scale_rule == FP4_MX_SCALE_FLOOR,
                                               gC, Cq, Cs, sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_mx_to_nv_scales(const uint8_t *s_mx, int64_t rows, int64_t cols, uint8_t *s_nv, float *gscale,
                               void *stream)
{
    if (rows < 0 || cols < 0 || !gscale) return FP4_ERR_INVALID_ARG;
    if (cols % 32) return FP4_ERR_UNSUPPORTED;
    if (too_many_units(rows, cols)) return FP4_ERR_UNSUPPORTED;
    if (rows > 0 && cols > 0 && (!s_mx || !s_nv)) return FP4_ERR_INVALID_ARG;
    if (!aligned(gscale, 4)) return FP4_ERR_ALIGNMENT;
    cudaError_t e = fp4::launch_mx_to_nv_scales(s_mx, rows, cols, s_nv, gscale, sm_count(),
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_nv_refine_gscale_workspace_size(int64_t rows, int64_t cols, size_t *bytes)
{
    if (rows < 0 || cols < 0 || !bytes) return FP4_ERR_INVALID_ARG;
    if (cols % 32) return FP4_ERR_UNSUPPORTED;
    *bytes = fp4::nv_refine_workspace_bytes(rows, cols);
    return FP4_OK;
}

fp4_status fp4_nv_refine_gscale(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int hadamard_k,
                                const fp4_opts *opts, int rounds, uint8_t *q, uint8_t *s, void *workspace,
                                size_t ws_bytes, float *gscale, void *stream)
{
    fp4_opts o = {FP4_ROUND_EVEN, FP4_MX_SCALE_CEIL, 0, FP4_SCALE_ABSMAX, 0};
    if (opts) o = *opts;
    if (rows < 0 || cols < 0 || ld_x < cols || rounds < 1 || rounds > 64) return FP4_ERR_INVALID_ARG;
    if (o.round != FP4_ROUND_EVEN && o.round != FP4_ROUND_AWAY) return FP4_ERR_INVALID_ARG;
    if (!valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (cols % 32 || (hadamard_k && cols % hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (too_many_units(rows, cols)) return FP4_ERR_UNSUPPORTED;
    if (!gscale || !workspace) return FP4_ERR_INVALID_ARG;
    if (rows > 0 && cols > 0 && (!x || !q || !s)) return FP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x % 8) || !aligned(q, 16) || !aligned(s, 16) || !aligned(workspace, 256) ||
        !aligned(gscale, 4))
        return FP4_ERR_ALIGNMENT;
    if (ws_bytes < fp4::nv_refine_workspace_bytes(rows, cols)) return FP4_ERR_INVALID_ARG;
    cudaError_t e = fp4::launch_nv_refine(static_cast<const uint16_t *>(x), rows, cols, ld_x, hadamard_k,
                                          hadamard_constant(hadamard_k), o.round == FP4_ROUND_AWAY, rounds, q, s,
                                          workspace, gscale, sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_kv_cache_sizes(int64_t num_pages, int page_size, int kv_heads, int head_dim, int fmt, size_t *q_bytes,
                              size_t *s_bytes)
{
    if (!q_bytes || !s_bytes) return FP4_ERR_INVALID_ARG;
    const fp4_status st = kv_geometry(num_pages, page_size, kv_heads, head_dim, fmt, 0);
    if (st != FP4_OK) return st;
    const size_t rows = (size_t)num_pages * (size_t)kv_heads * (size_t)page_size;
    *q_bytes = rows * (size_t)(head_dim / 2);
    *s_bytes = rows * (size_t)(head_dim / (fmt == FP4_MXFP4 ? 32 : 16));
    return FP4_OK;
}

fp4_status fp4_kv_append(const fp4_kv_cache *cache, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                         const void *v, int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                         int64_t tokens, const fp4_opts *opts, void *stream)
{
    fp4_opts o = {FP4_ROUND_EVEN, FP4_MX_SCALE_CEIL, 0, FP4_SCALE_ABSMAX, 0};
    if (opts) o = *opts;
    fp4::KvView c;
    fp4_status st = kv_view(cache, c);
    if (st != FP4_OK) return st;
    if (tokens < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
        return FP4_ERR_INVALID_ARG;
    if (o.round != FP4_ROUND_EVEN && o.round != FP4_ROUND_AWAY) return FP4_ERR_INVALID_ARG;
    if (o.mx_scale_rule != FP4_MX_SCALE_CEIL && o.mx_scale_rule != FP4_MX_SCALE_FLOOR) return FP4_ERR_INVALID_ARG;
    if (o.scale_search != FP4_SCALE_ABSMAX) return FP4_ERR_UNSUPPORTED;
    if (tokens == 0) return FP4_OK;
    if (!k || !v || !slots) return FP4_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 ||
        v_head_stride % 8 || !aligned(slots, 8))
        return FP4_ERR_ALIGNMENT;
    bool too_many = false;
    const cudaError_t e = fp4::launch_kv_append(
        c, cache->head_dim, cache->fmt, cache->hadamard_k, hadamard_constant(cache->hadamard_k),
        static_cast<const uint16_t *>(k), k_token_stride, k_head_stride, static_cast<const uint16_t *>(v), v_token_stride,
        v_head_stride, slots, tokens, o.round == FP4_ROUND_AWAY, o.mx_scale_rule == FP4_MX_SCALE_FLOOR,
        sm_count(), static_cast<cudaStream_t>(stream), &too_many);
    if (too_many) return FP4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_kv_gather(const fp4_kv_cache *cache, const int64_t *slots, int64_t tokens, int out_dtype, void *k_out,
                         void *v_out, void *stream)
{
    fp4::KvView c;
    fp4_status st = kv_view(cache, c);
    if (st != FP4_OK) return st;
    if (tokens < 0) return FP4_ERR_INVALID_ARG;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (tokens == 0) return FP4_OK;
    if (!slots || !k_out || !v_out) return FP4_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(k_out, 32) || !aligned(v_out, 32)) return FP4_ERR_ALIGNMENT;
    bool too_many = false;
    const cudaError_t e = fp4::launch_kv_gather(c, cache->head_dim, cache->fmt, cache->hadamard_k,
                                                hadamard_constant(cache->hadamard_k), slots, tokens,
                                                out_dtype == FP4_OUT_BF16, k_out, v_out, sm_count(),
                                                static_cast<cudaStream_t>(stream), &too_many);
    if (too_many) return FP4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_paged_attention_workspace_size(int64_t batch, int q_heads, int kv_heads, int head_dim,
                                              int64_t max_seq_len, int64_t window, size_t *bytes)
{
    if (!bytes) return FP4_ERR_INVALID_ARG;
    const fp4_status st = attention_sizes(batch, q_heads, kv_heads, head_dim, max_seq_len, window);
    if (st != FP4_OK) return st;
    *bytes = fp4::paged_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_seq_len, window, sm_count());
    return FP4_OK;
}

fp4_status fp4_paged_attention(const fp4_kv_cache *cache, const void *q, int64_t batch, int q_heads,
                               int64_t q_batch_stride, int64_t q_head_stride, const int32_t *page_table,
                               int64_t table_stride, int64_t table_cols, const int32_t *seq_lens, int64_t max_seq_len,
                               float scale, int64_t window, int out_dtype, void *out, float *lse, void *workspace,
                               size_t ws_bytes, void *stream)
{
    fp4::KvView c;
    fp4_status st = kv_view(cache, c);
    if (st != FP4_OK) return st;
    st = attention_sizes(batch, q_heads, cache->kv_heads, cache->head_dim, max_seq_len, window);
    if (st != FP4_OK) return st;
    if (q_batch_stride < 0 || q_head_stride < 0 || table_cols < 0 || table_stride < 0) return FP4_ERR_INVALID_ARG;
    if (table_cols > (1 << 30)) return FP4_ERR_UNSUPPORTED;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return FP4_ERR_INVALID_ARG;  // NaN or infinite
    if (batch == 0) return FP4_OK;
    if (!q || !seq_lens || !out || (table_cols > 0 && !page_table)) return FP4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_batch_stride % 8 || q_head_stride % 8 || !aligned(out, 16) || !aligned(page_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(lse, 4))
        return FP4_ERR_ALIGNMENT;
    const int sms = sm_count();
    const size_t need = fp4::paged_attention_workspace_bytes(batch, q_heads, cache->kv_heads, cache->head_dim, max_seq_len,
                                                             window, sms);
    if (need > 0 && (!workspace || ws_bytes < need)) return FP4_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 16)) return FP4_ERR_ALIGNMENT;
    const cudaError_t e = fp4::launch_paged_attention(
        c, cache->head_dim, cache->fmt, cache->hadamard_k, hadamard_constant(cache->hadamard_k),
        static_cast<const uint16_t *>(q), batch, q_heads, q_batch_stride, q_head_stride, page_table, table_stride,
        table_cols, seq_lens, max_seq_len, scale, window, out_dtype == FP4_OUT_BF16, out, lse, workspace, sms,
        static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fp4_linear_w4a16_workspace_size(int64_t M, int64_t N, int64_t K, int fmt, size_t *bytes)
{
    if (M < 0 || N < 0 || K < 0 || !bytes) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (M > 16 || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;  // as fp4_linear_w4a16
    const int sms = sm_count();
    *bytes = 0;  // the most that any rotation and output type takes
    for (int rot = 0; rot < 2; rot++)
        for (int two = 0; two <= rot; two++) {
            const size_t need = fp4::linear_w4a16_workspace_bytes(M, N, K, (int)(two ? 2 * M : M), rot != 0, sms);
            if (need > *bytes) *bytes = need;
        }
    return FP4_OK;
}

fp4_status fp4_linear_w4a16(const void *x, int64_t M, int64_t K, int64_t ld_x, int fmt, int hadamard_k,
                            const fp4_opts *opts, const uint8_t *Wq, const uint8_t *Ws, const float *gW, int64_t N,
                            int out_dtype, void *C, int64_t ldc, void *workspace, size_t ws_bytes, void *stream)
{
    const int w_static = opts ? opts->weights_static : 0;
    if (M < 0 || N < 0 || K < 0 || ld_x < K || ldc < N) return FP4_ERR_INVALID_ARG;
    if (!valid_gemm_fmt(fmt)) return FP4_ERR_UNSUPPORTED;
    if (out_dtype != FP4_OUT_F32 && out_dtype != FP4_OUT_BF16) return FP4_ERR_INVALID_ARG;
    if (w_static != 0 && w_static != 1) return FP4_ERR_INVALID_ARG;
    if (!valid_k(hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (K % 32 || (hadamard_k && K % hadamard_k)) return FP4_ERR_UNSUPPORTED;
    if (M > 16 || N > (1 << 30) || K > (1 << 30)) return FP4_ERR_UNSUPPORTED;  // the decode product only
    if (M == 0 || N == 0) return FP4_OK;
    if (K == 0) return FP4_ERR_UNSUPPORTED;
    if (!x || !Wq || !Ws || !C) return FP4_ERR_INVALID_ARG;
    if (fmt == FP4_NVFP4 && !gW) return FP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x % 8) || !aligned(Wq, 16) || !aligned(Ws, 16) || !aligned(C, 16) || !aligned(gW, 4))
        return FP4_ERR_ALIGNMENT;
    const int sms = sm_count(), cols = (int)(hadamard_k && out_dtype == FP4_OUT_F32 ? 2 * M : M);
    const size_t need = fp4::linear_w4a16_workspace_bytes(M, N, K, cols, hadamard_k != 0, sms);
    if (need > 0 && (!workspace || ws_bytes < need)) return FP4_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return FP4_ERR_ALIGNMENT;
    const cudaError_t e = fp4::launch_linear_w4a16(
        static_cast<const uint16_t *>(x), ld_x, M, K, fmt, hadamard_k, hadamard_constant(hadamard_k), Wq, Ws, gW, N,
        out_dtype == FP4_OUT_BF16, C, ldc, w_static, workspace, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

uint64_t fp4_kernel_launches(void) { return fp4::g_launches.load(std::memory_order_relaxed); }

fp4_status fp4_check_device_status(void *stream)
{
    unsigned int err = 0;
    if (fp4::read_and_clear_device_errors(static_cast<cudaStream_t>(stream), &err) != cudaSuccess)
        return FP4_ERR_CUDA;
    return err ? FP4_ERR_TIMEOUT : FP4_OK;
}

}  // extern "C"
