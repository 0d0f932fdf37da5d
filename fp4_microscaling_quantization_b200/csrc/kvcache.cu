// kvcache.cu — the paged FP4 key-value cache: quantization of new keys and
// values into their slots as they arrive (fp4_kv_append), and tokens read
// back by their slots (fp4_kv_gather).
//
// Method: fp4_quantize's and fp4_dequantize's, unit by unit, with the same
// encoder and the same bits: TransFP4 §1.1 Eq.(1) with absmax block scales,
// after the rotation H_k of every head row; x^ = RN(RN(s_g s_b) q) and H_k
// again on the way back.  The NVFP4 tensor scales are given: they belong to
// the cache, not to one call's tokens.
//
// Work decomposition: one thread owns one 32-element unit of a head row
// (64 bytes of bf16, 16 bytes of nibbles, 1 or 2 scale bytes).  A warp owns
// 32 / (dim / 32) consecutive tokens of one head of K or of V: with
// consecutive slots its nibbles are 512 contiguous bytes of a page, and its
// bf16 rows are whole 2 * dim byte segments.  Bound: HBM for prompts, the
// launch and two dependent loads (slot, then data) for a decode step.
#include "kv.cuh"
#include "sm100.cuh"

namespace fp4 {

struct KvAppendArgs {
    KvView c;
    const uint16_t *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;  // strides, elements
    const int64_t *slots;
    int64_t tokens;
    int64_t num_slots;
    int upr_shift;  // log2 of the units in a head row (1, 2, 3)
    float ck;
    int round_away, mx_floor;
    uint32_t warps;  // 2 * heads * token groups
    FastDiv heads_div;
};

// The token, head and tensor (0 = K, 1 = V) of a warp, and its lane's unit.
struct KvWork {
    int64_t token;
    int head, kv, unit;
};

FP4_DEV KvWork kv_work(uint32_t warp, int lane, int upr_shift, const FastDiv &heads_div)
{
    KvWork w;
    w.kv = warp & 1;
    const uint32_t th = warp >> 1;
    const uint32_t group = fastdiv(th, heads_div);
    w.head = (int)(th - group * heads_div.d);
    w.unit = lane & ((1 << upr_shift) - 1);
    w.token = (int64_t)group * (32 >> upr_shift) + (lane >> upr_shift);
    return w;
}

template <int FMT, int HK>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    const uint32_t warp = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (warp >= a.warps) return;
    const int lane = threadIdx.x & 31;
    const KvWork w = kv_work(warp, lane, a.upr_shift, a.heads_div);
    const int64_t slot = w.token < a.tokens ? __ldg(a.slots + w.token) : -1;
    const bool live = slot >= 0 && slot < a.num_slots;  // others are dropped
    float sg = 1.0f, six_sg = 6.0f;
    if (FMT == FP4_NVFP4) {
        sg = __ldg(w.kv ? a.c.gv : a.c.gk);
        six_sg = __fmul_rn(6.0f, sg);
    }
    uint4 raw[4] = {};
    if (live) {
        const uint16_t *row = w.kv ? a.v + w.token * a.v_tok + w.head * a.v_head : a.k + w.token * a.k_tok + w.head * a.k_head;
        const uint4 *p = reinterpret_cast<const uint4 *>(row + w.unit * 32);
#pragma unroll
        for (int i = 0; i < 4; i++) raw[i] = __ldg(p + i);
    }
    float v[32];
    unpack_unit(raw, v);
    if (HK) fwht_unit<HK>(v, a.ck, lane);  // every lane: chunks of 64 and 128 exchange values
    uint4 out;
    const uint32_t sb = encode_unit<FMT>(v, sg, six_sg, a.round_away, a.mx_floor, out);
    if (!live) return;
    const int64_t unit = (kv_row(slot, w.head, a.c) << a.upr_shift) + w.unit;
    reinterpret_cast<uint4 *>(w.kv ? a.c.vq : a.c.kq)[unit] = out;
    uint8_t *s = w.kv ? a.c.vs : a.c.ks;
    if (FMT == FP4_MXFP4)
        s[unit] = (uint8_t)sb;
    else
        reinterpret_cast<uint16_t *>(s)[unit] = (uint16_t)sb;
}

struct KvGatherArgs {
    KvView c;
    const int64_t *slots;
    int64_t tokens;
    int64_t num_slots;
    int upr_shift;
    float ck;
    void *k, *v;  // (tokens, heads, dim)
    uint32_t warps;
    FastDiv heads_div;
};

template <int FMT, int HK, int BF16OUT>
__global__ void __launch_bounds__(256) kv_gather_kernel(KvGatherArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    const uint32_t warp = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (warp >= a.warps) return;
    const int lane = threadIdx.x & 31;
    const KvWork w = kv_work(warp, lane, a.upr_shift, a.heads_div);
    const bool live = w.token < a.tokens;
    const int64_t slot = live ? __ldg(a.slots + w.token) : -1;
    const float sg = (FMT == FP4_NVFP4) ? __ldg(w.kv ? a.c.gv : a.c.gk) : 1.0f;
    uint4 raw = make_uint4(0, 0, 0, 0);
    uint32_t sb = 0;
    const bool held = slot >= 0 && slot < a.num_slots;  // others read as zeros
    if (held) {
        const int64_t unit = (kv_row(slot, w.head, a.c) << a.upr_shift) + w.unit;
        raw = __ldg(reinterpret_cast<const uint4 *>(w.kv ? a.c.vq : a.c.kq) + unit);
        const uint8_t *s = w.kv ? a.c.vs : a.c.ks;
        sb = (FMT == FP4_MXFP4) ? (uint32_t)__ldg(s + unit) : (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(s) + unit);
    }
    const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
    float d0, d1, v[32];
    unit_decode_factors<FMT>(sb, sg, d0, d1);
    if (!held) d0 = d1 = 0.0f;  // a tensor scale that is not finite reaches no zero
#pragma unroll
    for (int c = 0; c < 4; c++) {
#pragma unroll
        for (int b = 0; b < 4; b++) {
            float lo, hi;
            e2m1x2_to_f32((words[c] >> (8 * b)) & 0xFF, lo, hi);
            v[8 * c + 2 * b] = __fmul_rn(c < 2 ? d0 : d1, lo);
            v[8 * c + 2 * b + 1] = __fmul_rn(c < 2 ? d0 : d1, hi);
        }
    }
    if (HK) fwht_unit<HK>(v, a.ck, lane);
    if (!live) return;
    // 32-byte stores: whole sectors from each lane, so no staging for the
    // write side is needed
    const int64_t unit = ((w.token * a.c.heads + w.head) << a.upr_shift) + w.unit;
    if (BF16OUT) {
        uint8_t *p = static_cast<uint8_t *>(w.kv ? a.v : a.k) + unit * 64;
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            h[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        st_global_v8(p, h);
        st_global_v8(p + 32, h + 8);
    } else {
        uint8_t *p = static_cast<uint8_t *>(w.kv ? a.v : a.k) + unit * 128;
#pragma unroll
        for (int i = 0; i < 4; i++) st_global_v8(p + 32 * i, reinterpret_cast<const uint32_t *>(v) + 8 * i);
    }
}

// ---------------------------------------------------------------------------
// Host launchers (called from capi.cu after validation).
template <int FMT>
static void (*append_for(int hk))(KvAppendArgs)
{
    switch (hk) {
    case 16: return kv_append_kernel<FMT, 16>;
    case 32: return kv_append_kernel<FMT, 32>;
    case 64: return kv_append_kernel<FMT, 64>;
    case 128: return kv_append_kernel<FMT, 128>;
    default: return kv_append_kernel<FMT, 0>;
    }
}

template <int FMT, int BF16OUT>
static void (*gather_for(int hk))(KvGatherArgs)
{
    switch (hk) {
    case 16: return kv_gather_kernel<FMT, 16, BF16OUT>;
    case 32: return kv_gather_kernel<FMT, 32, BF16OUT>;
    case 64: return kv_gather_kernel<FMT, 64, BF16OUT>;
    case 128: return kv_gather_kernel<FMT, 128, BF16OUT>;
    default: return kv_gather_kernel<FMT, 0, BF16OUT>;
    }
}

// Warps of a call (0 if they do not fit the kernels' 32-bit index).
static uint32_t kv_warps(int64_t tokens, int heads, int upr_shift)
{
    const int64_t groups = (tokens + (32 >> upr_shift) - 1) / (32 >> upr_shift);
    if (groups > (int64_t(1) << 31) / (2 * (int64_t)heads)) return 0;
    return (uint32_t)(2 * heads * groups);
}

static int upr_shift_of(int dim) { return dim == 64 ? 1 : dim == 128 ? 2 : 3; }

cudaError_t launch_kv_append(const KvView &c, int dim, int fmt, int hk, float ck, const uint16_t *k, int64_t k_tok,
                             int64_t k_head, const uint16_t *v, int64_t v_tok, int64_t v_head, const int64_t *slots,
                             int64_t tokens, int round_away, int mx_floor, cudaStream_t st, bool *too_many)
{
    KvAppendArgs a = {};
    a.c = c;
    a.k = k;
    a.v = v;
    a.k_tok = k_tok;
    a.k_head = k_head;
    a.v_tok = v_tok;
    a.v_head = v_head;
    a.slots = slots;
    a.tokens = tokens;
    a.num_slots = c.num_pages << c.page_shift;
    a.upr_shift = upr_shift_of(dim);
    a.ck = ck;
    a.round_away = round_away;
    a.mx_floor = mx_floor;
    a.warps = kv_warps(tokens, c.heads, a.upr_shift);
    a.heads_div = make_fastdiv((uint32_t)c.heads);
    *too_many = a.warps == 0;
    if (*too_many) return cudaSuccess;
    auto kern = fmt == FP4_MXFP4 ? append_for<FP4_MXFP4>(hk) : fmt == FP4_NVFP4 ? append_for<FP4_NVFP4>(hk) : append_for<FP4_MXFP4_16>(hk);
    return launch_k(kern, dim3((a.warps + 7) / 8), dim3(256), 0, st, true, a);
}

cudaError_t launch_kv_gather(const KvView &c, int dim, int fmt, int hk, float ck, const int64_t *slots, int64_t tokens,
                             int bf16out, void *k, void *v, cudaStream_t st, bool *too_many)
{
    KvGatherArgs a = {};
    a.c = c;
    a.slots = slots;
    a.tokens = tokens;
    a.num_slots = c.num_pages << c.page_shift;
    a.upr_shift = upr_shift_of(dim);
    a.ck = ck;
    a.k = k;
    a.v = v;
    a.warps = kv_warps(tokens, c.heads, a.upr_shift);
    a.heads_div = make_fastdiv((uint32_t)c.heads);
    *too_many = a.warps == 0;
    if (*too_many) return cudaSuccess;
    void (*kern)(KvGatherArgs);
    if (bf16out)
        kern = fmt == FP4_MXFP4 ? gather_for<FP4_MXFP4, 1>(hk) : fmt == FP4_NVFP4 ? gather_for<FP4_NVFP4, 1>(hk) : gather_for<FP4_MXFP4_16, 1>(hk);
    else
        kern = fmt == FP4_MXFP4 ? gather_for<FP4_MXFP4, 0>(hk) : fmt == FP4_NVFP4 ? gather_for<FP4_NVFP4, 0>(hk) : gather_for<FP4_MXFP4_16, 0>(hk);
    return launch_k(kern, dim3((a.warps + 7) / 8), dim3(256), 0, st, true, a);
}

}  // namespace fp4
