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
// (64 bytes of bf16, 16 bytes of nibbles, 1 or 2 scale bytes) of K and the
// same of V, both loads ahead of the first use; calls that do not fill the GPU
// give K and V to different warps (61 tokens: append and gather 4.0 us, by one
// warp 5.1).  A warp owns 32 / (dim / 32)
// consecutive tokens of one head: with consecutive slots its nibbles are 512
// contiguous bytes of a page, and its bf16 rows are whole 2 * dim byte
// segments, read and written 32 bytes a lane.  Bound: HBM for prompts (100003
// tokens read back at 99 % of the measured copy rate); with H_64 68 %, where
// most of a warp's time is the wait for its loads (long_scoreboard 2.9 and 3.3
// per issue at 7 warps per scheduler, 0.65 of the issue slots used): a thread
// loads, computes and stores once.  The launch and two dependent loads (slot,
// then data) for a decode step.
#include "frag.cuh"
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
    int wide;       // rows are 32-byte aligned: 32-byte loads
    uint32_t warps;  // heads * token groups (of a grid row)
    FastDiv heads_div;
};

// The head of a warp, its lane's token and unit of the head row.
struct KvWork {
    int64_t token;
    int head, unit;
};

FP4_DEV KvWork kv_work(uint32_t warp, int lane, int upr_shift, const FastDiv &heads_div)
{
    KvWork w;
    const uint32_t group = fastdiv(warp, heads_div);
    w.head = (int)(warp - group * heads_div.d);
    w.unit = lane & ((1 << upr_shift) - 1);
    w.token = (int64_t)group * (32 >> upr_shift) + (lane >> upr_shift);
    return w;
}

// Plain loads here and below: a launch may begin before the one before it has
// ended, and no wait orders reads as constant data (ld.global.nc) of what that
// one wrote.
FP4_DEV void ld_v8(const void *p, uint4 &a, uint4 &b)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
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
    const int only = gridDim.y == 2 ? (int)blockIdx.y : -1;  // K or V alone
    const int64_t slot = w.token < a.tokens ? a.slots[w.token] : -1;
    const bool live = slot >= 0 && slot < a.num_slots;  // others are dropped
    uint4 raw[2][4] = {};
    if (live) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (i + only == 1) continue;
            const uint16_t *row = i ? a.v + w.token * a.v_tok + w.head * a.v_head : a.k + w.token * a.k_tok + w.head * a.k_head;
            const uint4 *p = reinterpret_cast<const uint4 *>(row + w.unit * 32);
            if (a.wide) {
                ld_v8(p, raw[i][0], raw[i][1]);
                ld_v8(p + 2, raw[i][2], raw[i][3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) raw[i][e] = p[e];
            }
        }
    }
    const int64_t unit = live ? (kv_row(slot, w.head, a.c) << a.upr_shift) + w.unit : 0;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (i + only == 1) continue;
        float sg = 1.0f, six_sg = 6.0f;
        if (FMT == FP4_NVFP4) {
            sg = *(i ? a.c.gv : a.c.gk);
            six_sg = __fmul_rn(6.0f, sg);
        }
        float v[32];
        unpack_unit(raw[i], v);
        if (HK) fwht_unit<HK>(v, a.ck, lane);  // every lane: chunks of 64 and 128 exchange values
        uint4 out;
        const uint32_t sb = encode_unit<FMT>(v, sg, six_sg, a.round_away, a.mx_floor, out);
        if (!live) continue;
        reinterpret_cast<uint4 *>(i ? a.c.vq : a.c.kq)[unit] = out;
        uint8_t *s = i ? a.c.vs : a.c.ks;
        if (FMT == FP4_MXFP4)
            s[unit] = (uint8_t)sb;
        else
            reinterpret_cast<uint16_t *>(s)[unit] = (uint16_t)sb;
    }
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
    const int only = gridDim.y == 2 ? (int)blockIdx.y : -1;  // K or V alone
    const int64_t slot = live ? a.slots[w.token] : -1;
    uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    uint32_t sb[2] = {0, 0};
    const bool held = slot >= 0 && slot < a.num_slots;  // others read as zeros
    if (held) {
        const int64_t unit = (kv_row(slot, w.head, a.c) << a.upr_shift) + w.unit;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (i + only == 1) continue;
            raw[i] = reinterpret_cast<const uint4 *>(i ? a.c.vq : a.c.kq)[unit];
            const uint8_t *s = i ? a.c.vs : a.c.ks;
            sb[i] = (FMT == FP4_MXFP4) ? (uint32_t)s[unit] : (uint32_t)reinterpret_cast<const uint16_t *>(s)[unit];
        }
    }
    const int64_t unit = ((w.token * a.c.heads + w.head) << a.upr_shift) + w.unit;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (i + only == 1) continue;
        const float sg = (FMT == FP4_NVFP4) ? *(i ? a.c.gv : a.c.gk) : 1.0f;
        const uint32_t words[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float d0, d1, v[32];
        unit_decode_factors<FMT>(sb[i], sg, d0, d1);
        if (!held) d0 = d1 = 0.0f;  // a tensor scale that is not finite reaches no zero
#pragma unroll
        for (int c = 0; c < 4; c++) {
            uint32_t h[4];
            e2m1x8_to_f16(words[c], h);
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[b]));
                v[8 * c + 2 * b] = t.x;
                v[8 * c + 2 * b + 1] = t.y;
            }
        }
        // RN(d q): the scale times an exact value, each rounded on its own
#pragma unroll
        for (int e = 0; e < 32; e++) v[e] = __fmul_rn(e < 16 ? d0 : d1, v[e]);
        if (HK) fwht_unit<HK>(v, a.ck, lane);
        if (!live) continue;
        // 32-byte stores: whole sectors from each lane, so no staging for the
        // write side is needed
        if (BF16OUT) {
            uint8_t *p = static_cast<uint8_t *>(i ? a.v : a.k) + unit * 64;
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 16; e++) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                h[e] = *reinterpret_cast<const uint32_t *>(&t);
            }
            st_global_v8(p, h);
            st_global_v8(p + 32, h + 8);
        } else {
            uint8_t *p = static_cast<uint8_t *>(i ? a.v : a.k) + unit * 128;
#pragma unroll
            for (int e = 0; e < 4; e++) st_global_v8(p + 32 * e, reinterpret_cast<const uint32_t *>(v) + 8 * e);
        }
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
    if (groups > (int64_t(1) << 31) / heads) return 0;
    return (uint32_t)(heads * groups);
}

// Eight warps to a CTA; a second row of CTAs for V up to one round of 24 warps per SM.
static dim3 kv_grid(uint32_t warps, int sms) { return dim3((warps + 7) / 8, warps <= (uint32_t)sms * 12 ? 2 : 1); }

static int upr_shift_of(int dim) { return dim == 64 ? 1 : dim == 128 ? 2 : 3; }

cudaError_t launch_kv_append(const KvView &c, int dim, int fmt, int hk, float ck, const uint16_t *k, int64_t k_tok,
                             int64_t k_head, const uint16_t *v, int64_t v_tok, int64_t v_head, const int64_t *slots,
                             int64_t tokens, int round_away, int mx_floor, int sms, cudaStream_t st, bool *too_many)
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
    a.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0) && (k_tok | k_head | v_tok | v_head) % 16 == 0;
    a.warps = kv_warps(tokens, c.heads, a.upr_shift);
    a.heads_div = make_fastdiv((uint32_t)c.heads);
    *too_many = a.warps == 0;
    if (*too_many) return cudaSuccess;
    auto kern = fmt == FP4_MXFP4 ? append_for<FP4_MXFP4>(hk) : fmt == FP4_NVFP4 ? append_for<FP4_NVFP4>(hk) : append_for<FP4_MXFP4_16>(hk);
    return launch_k(kern, kv_grid(a.warps, sms), dim3(256), 0, st, true, a);
}

cudaError_t launch_kv_gather(const KvView &c, int dim, int fmt, int hk, float ck, const int64_t *slots, int64_t tokens,
                             int bf16out, void *k, void *v, int sms, cudaStream_t st, bool *too_many)
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
    return launch_k(kern, kv_grid(a.warps, sms), dim3(256), 0, st, true, a);
}

}  // namespace fp4
