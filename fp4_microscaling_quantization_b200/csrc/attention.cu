// attention.cu — attention of one new token per sequence over the paged FP4
// key-value cache (fp4_paged_attention).
//
// Mathematics.  For query head h with key-value head h / group,
//   x_t = scale * (H q_h) . k~_t,   w_t = exp(x_t),   o = H (sum_t w_t v~_t) / sum_t w_t,
// over the live tokens t (inside the length, the window and a held page);
// k~, v~ are the cache's dequantized values in the rotated domain, where
// (H q) . (H k) = q . k, so the cache is never rotated back: q is rotated
// once, and o once at the end.  One pass: running maximum m, sum l and
// unnormalised o are rescaled when m grows.
//
// What bounds it: the cache is read once, 2 * dim * (1/2 + 1/block) bytes per
// token and head, and every element has to become a 16-bit operand first: the
// issue slots of that conversion come next after HBM.  Per 32 tokens of a head
// of 128 (4608 bytes, 198 clocks of an SM's share of HBM) a warp issues about
// 630 instructions, 128 of them conversions (64 a clock and SM) and 128 scale
// multiplies, and at 16 warps per SM about 0.6 slots of a clock are used: 66 %
// of the measured copy rate for one sequence of 262143 tokens (MXFP4, 66.0 us
// in a graph of calls, as all times here), 62 % for 64 of 1 to 8192 (NVFP4,
// 76.2 us).  So:
//   * The products run on mma.sync m16n8k16 (f16 in, fp32 sums) from registers.
//     tcgen05 would need the dequantized tile written to shared or tensor
//     memory first, at four times the packed bytes; its rate is not what
//     is short here (up to 8 query rows per key head).
//   * The order of a product's inner index is free, so each lane's operand
//     elements are whole consecutive bytes of a token's row.  K is the row
//     operand of the scores (a lane holds dim/4 consecutive elements of two
//     tokens), q the 8 columns; V transposed is the row operand of the output
//     (a lane holds dim/8 consecutive elements of 4 tokens), the weights the
//     columns.  A byte of K is a register pair after one conversion; two
//     tokens' V bytes are merged nibble by nibble first.  The scores' result
//     becomes the next product's operand by one 8 x 8 transpose of registers.
//     (K as the column operand needs no transpose, but half of its rows are
//     padding: 98.7 us instead of 87.4 for the batch above, at that stage.)
//   * E2M1 times its block scale is exact in f16: for NVFP4 the E4M3 scale
//     itself (6 significant bits, 2^-10 .. 2688), for E8M0 a power of two
//     relative to the largest scale that the warp has met so far.
//   * q in f16 as a power of two times hi: exact for a bf16 q, and hi + lo (a
//     second product) after a rotation.  Weights w_t are rounded to f16 (11
//     bits, scaled by 2^15 so that they stay normal down to 2^-29 of the
//     largest; below, to steps of 2^-39), and for fp32 output are split into
//     hi + lo as well.
//   * Every warp streams its own steps of 16, 32 or 64 tokens through its own
//     two stages of asynchronous copies: no barrier among warps until their
//     results are joined.  (Three or four stages, and scores computed beside
//     the values of the step before, were no faster: 86.0 and 86.3 against 84.3,
//     when that was the time of the batch above.)
// Long sequences are cut into chunks of tokens over CTAs; a second kernel
// joins the chunks.  The cut depends on the call's sizes only, and every sum
// has a fixed order, so results repeat bit for bit.
#include <math.h>

#include <algorithm>

#include "frag.cuh"
#include "kv.cuh"
#include "sm100.cuh"

namespace fp4 {
namespace attn {

constexpr int NW = 4;           // warps per CTA, each on its own tokens
constexpr int HT = 8;           // query heads per CTA
constexpr float kPShift = 15.0f;  // weights are 2^15 w / w_max, inside f16's range
constexpr float kUnit = 32768.0f; // 2^kPShift: so are their sums; E8M0 outputs leave the warps without it
// Scores (in units of log 2) from which fp32 has steps of 1: the largest
// weight is then 2^kPShift only up to a factor of 2.
constexpr float kFar = 8388608.0f;
constexpr int kAlign = 64;      // chunks start at multiples of the longest step
constexpr int kMaxChunks = 1024;
constexpr int kJoin = 256;      // threads of join_kernel
constexpr float kTiny = 1.17549435e-38f;  // the least normal number

struct Args {
    KvView c;
    const uint16_t *q;
    int64_t q_b, q_h;  // strides, elements
    const int32_t *table;
    int64_t table_b;       // row stride of the page table
    int table_tokens;      // tokens that a row of the table reaches (at most 2^30: lengths fit 31 bits)
    const int32_t *lens;
    int max_len;
    int window;            // 0 = none
    int group, head_tiles, q_heads;
    float scale;           // times log2(e)
    float ck;
    int hk;
    int chunk;             // tokens per chunk, a multiple of kAlign
    int chunks;
    void *out;
    float *lse;
    float *part_o;         // [batch][q_heads][chunks][dim]
    float2 *part_ml;       // [batch][q_heads][chunks] (m, l)
};

template <int FMT, int D>
struct Shape {
    static constexpr int SB = D / (FMT == FP4_MXFP4 ? 32 : 16);  // scale bytes per row
    static constexpr int QB = D / 2;                             // element bytes per row
    static constexpr int TS = D == 64 ? 64 : D == 128 ? 32 : 16; // tokens per step
    static constexpr int STAGE = 2 * TS * (QB + SB);             // bytes: K, V elements, K, V scales
    static constexpr int ST = 2;                                 // stages per warp
    static constexpr int RING = NW * ST * STAGE;
    static constexpr int JOIN = NW * HT * D * 4;                 // the warps' results, over the ring
    static constexpr int QF = 2 * HT * D * 2;                    // hi and lo of q
    // q lies in warp 0's last stage, which its first loop trip fills, where it
    // fits (dims 64, 128), else behind the ring
    static constexpr int BODY = RING > JOIN ? RING : JOIN;
    static constexpr int QAT = QF <= STAGE ? (ST - 1) * STAGE : BODY;
    static constexpr int SMEM = QF <= STAGE ? BODY : BODY + QF;
};

FP4_DEV float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The transpose of an 8 x 8 matrix of 16-bit values held as a product's result
// is (row lane / 4, columns 2 (lane % 4) and the next).
FP4_DEV uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The bits of a where m is set, of b elsewhere: one instruction (written out,
// the compiler moves the masks before the shifts and needs two).
FP4_DEV uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
    return r;
}

// The token of column n in a tile of 8 (an involution).  Columns 2m and 2m+1
// are tokens of opposite parity, for K's 16-byte loads; even columns are
// tokens 0, 3, 4, 7, for V's: both then touch every bank once.
__host__ __device__ constexpr int tau(int n) { return n ^ ((n >> 1) & 1); }

// Byte offset of 16-byte piece j of row t in the K and V element arrays of a
// stage: as in the cache for dims 64 and 128 (V's loads then meet two rows in
// a bank, which costs less than the addresses of a swizzle: they are immediate
// offsets of one register); swizzled for dim 256, where it would be four.
template <int D>
FP4_DEV uint32_t k_piece(int t, int j)
{
    return (uint32_t)(D == 256 ? t * 128 + (j ^ ((t & 1) << 2)) * 16 : t * (D / 2) + j * 16);
}
template <int D>
FP4_DEV uint32_t v_piece(int t, int j)
{
    return (uint32_t)(D == 256 ? t * 128 + (j ^ (((t & 1) | (((t >> 2) & 1) << 1)) << 1)) * 16 : t * (D / 2) + j * 16);
}

// e8m0_rel of two scale bytes, one in each half.
FP4_DEV uint32_t e8m0_rel2(uint32_t e0, uint32_t e1, uint32_t ref)
{
    const int t0 = (int)e0 - (int)ref + 23, t1 = (int)e1 - (int)ref + 23;
    return ((uint32_t)(t0 > 0 ? t0 : 0) << 10) | ((uint32_t)(t1 > 0 ? t1 : 0) << 26);
}

// The live range of a sequence's tokens, and where its chunks start.
struct Range {
    int begin, end, base;
};
FP4_DEV Range live_range(const Args &a, int b)
{
    Range r;
    r.end = max(min(a.lens[b], min(a.max_len, a.table_tokens)), 0);
    r.begin = a.window > 0 && r.end > a.window ? r.end - a.window : 0;
    r.base = r.begin & ~(kAlign - 1);
    return r;
}

template <int BF16OUT>
FP4_DEV void store_out(void *out, int64_t i, float v)
{
    if (BF16OUT)
        static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(out)[i] = v;
}

// The result rows o[h][0 .. D) in shared memory (normalised) -> out, through
// H_k where the cache is rotated.  Called by all threads; nt is their number.
template <int D, int BF16OUT>
FP4_DEV void write_rows(const float *o, int rows, int64_t out_row, const Args &a, int nt)
{
    constexpr int UPR = D / 32;
    if (a.hk) {
        for (int i = threadIdx.x; i < (rows * UPR + 31) / 32 * 32; i += nt) {
            float v[32];
            const bool live = i < rows * UPR;
#pragma unroll
            for (int e = 0; e < 32; e++) v[e] = live ? o[i * 32 + e] : 0.0f;
            rotate_unit(v, a.hk, a.ck, threadIdx.x & 31);
            if (live) {
#pragma unroll
                for (int e = 0; e < 32; e++) store_out<BF16OUT>(a.out, out_row * D + i * 32 + e, v[e]);
            }
        }
    } else {
        for (int i = threadIdx.x; i < rows * D / 4; i += nt) {
            const float4 v = reinterpret_cast<const float4 *>(o)[i];
            if (BF16OUT) {
                const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
                reinterpret_cast<uint2 *>(a.out)[out_row * (D / 4) + i] =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
            } else {
                reinterpret_cast<float4 *>(a.out)[out_row * (D / 4) + i] = v;
            }
        }
    }
}

// What a warp has to give for the join, worked out value by value in fp32 from
// the cache itself: its maxima, sums and unnormalised outputs of the CTA's heads
// over its steps of TS tokens.  For what a warp's loop leaves out, at no
// cost where it does not occur (a look at the scale bytes in the loop cost 4 to
// 7 % at dim 64 by the registers it took), and slowly where it does:
//   * an E8M0 scale of 0xFF, which the loop takes for a largest scale, is NaN
//     (of a key: its score, so all; of a value: its block's channels);
//   * scores from kFar on: the difference to the maximum, taken after the
//     score's rounding, is 0 for the maximum itself, whatever fp32's steps.
// A lane holds D / 32 consecutive channels.
template <int FMT, int D, int TS>
__device__ __noinline__ void plain_warp(const Args &a, float *so, float *sm_m, float *sm_l)
{
    constexpr int E = D / 32, BLOCK = FMT == FP4_MXFP4 ? 32 : 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d0 = lane * E;
    const int b = blockIdx.z, kvh = blockIdx.y, chunk = blockIdx.x / a.head_tiles, ht = blockIdx.x - chunk * a.head_tiles;
    const int h0 = kvh * a.group + ht * HT, nh = min(HT, a.group - ht * HT);
    const Range r = live_range(a, b);
    const int cs = r.base + chunk * a.chunk, ce = min(cs + a.chunk, r.end);
    const auto values = [&](const uint8_t *q, const uint8_t *s, int64_t row, float *v) {
        const uint32_t byte = s[row * (D / BLOCK) + d0 / BLOCK];
        const float f = FMT == FP4_NVFP4 ? e4m3_to_f32(byte) : e8m0_to_f32(byte);
        for (int e = 0; e < E; e += 2) {
            e2m1x2_to_f32(q[row * (D / 2) + (d0 + e) / 2], v[e], v[e + 1]);
            v[e] = __fmul_rn(v[e], f);
            v[e + 1] = __fmul_rn(v[e + 1], f);
        }
    };
    const float gk = FMT == FP4_NVFP4 ? *a.c.gk : 1.0f;  // (values: with the normalisation, as from the loop)
    for (int h = 0; h < nh; h++) {
        float q[E], o[E] = {}, m = -kFltMax, l = 0.0f;
        for (int e = 0; e < E; e++) q[e] = bf16lo(a.q[b * a.q_b + (int64_t)(h0 + h) * a.q_h + d0 + e]);
        if (a.hk) {
            for (int s = 1; s < a.hk; s <<= 1) {
                float t[E];
                for (int e = 0; e < E; e++) {
                    const bool up = ((d0 + e) & s) != 0;
                    float other = s >= E ? __shfl_xor_sync(0xFFFFFFFFu, q[e], s / E) : 0.0f;
                    for (int k = 0; s < E && k < E; k++)
                        if (k == (e ^ s)) other = q[k];
                    t[e] = up ? __fsub_rn(other, q[e]) : __fadd_rn(q[e], other);
                }
                for (int e = 0; e < E; e++) q[e] = t[e];
            }
            for (int e = 0; e < E; e++) q[e] = __fmul_rn(q[e], a.ck);
        }
        for (int t = cs; t < ce; t++) {
            if ((t - cs) / TS % NW != warp || t < r.begin) continue;
            const int page = a.table[b * a.table_b + (t >> a.c.page_shift)];
            if ((uint32_t)page >= (uint32_t)a.c.num_pages) continue;
            const int64_t row = kv_row(((int64_t)page << a.c.page_shift) + (t & ((1 << a.c.page_shift) - 1)), kvh, a.c);
            float v[E], x = 0.0f;
            values(a.c.kq, a.c.ks, row, v);
            for (int e = 0; e < E; e++) x = __fmaf_rn(q[e], v[e], x);
            for (int s = 1; s < 32; s <<= 1) x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, s));
            x = __fmul_rn(__fmul_rn(x, gk), a.scale);
            const float top = fmaxf(m, x), alpha = ex2(__fsub_rn(m, top)), p = ex2(__fsub_rn(x, top));
            m = top;
            l = __fmaf_rn(l, alpha, p);
            values(a.c.vq, a.c.vs, row, v);
            for (int e = 0; e < E; e++) o[e] = __fmaf_rn(o[e], alpha, __fmul_rn(p, v[e]));
        }
        if (lane == 0) {
            sm_m[h] = m;
            sm_l[h] = __fmul_rn(l, kUnit);
        }
        for (int e = 0; e < E; e++) so[h * D + d0 + e] = FMT == FP4_NVFP4 ? __fmul_rn(o[e], kUnit) : o[e];
    }
}

// ROT: the cache is rotated, so q has more than f16's 11 bits and its lo rows
// are not zero (a bf16 q is exact in the hi rows alone).
template <int FMT, int D, int BF16OUT, bool ROT>
__global__ void __launch_bounds__(NW * 32, D == 256 ? (ROT ? 2 : 3) : 4) paged_kernel(const __grid_constant__ Args a)
{
    using S = Shape<FMT, D>;
    constexpr int WPT = D / 32;       // words of a lane's K row part
    constexpr int VW = D / 64;        // words of a lane's V row part
    constexpr int NT = S::TS / 8;     // token tiles per step
    constexpr int MT = D / 16;        // output tiles
    constexpr int PIECES = S::QB / 16;
    constexpr int HALVES = S::TS / 16;
    constexpr bool NV = FMT == FP4_NVFP4;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sm_m[NW][HT], sm_l[NW][HT], q_exp[HT];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int b = blockIdx.z, kvh = blockIdx.y;
    const int chunk = blockIdx.x / a.head_tiles, ht = blockIdx.x - chunk * a.head_tiles;
    const int h0 = kvh * a.group + ht * HT;  // first query head
    const int nh = min(HT, a.group - ht * HT);
    // (plain loads: what launches before this one wrote may not be read as
    // constant data, which no wait orders)
    // this thread's pieces of q, asked for before anything else: the page
    // numbers and the first pages wait for the lengths
    constexpr int QP = D / 8, QI = (HT * QP + NW * 32 - 1) / (NW * 32);
    uint4 q_raw[QI];
#pragma unroll
    for (int i = 0; i < QI; i++) {
        const int p = i * NW * 32 + threadIdx.x, h = p / QP;
        q_raw[i] = make_uint4(0, 0, 0, 0);
        if (h < nh) q_raw[i] = reinterpret_cast<const uint4 *>(a.q + b * a.q_b + (int64_t)(h0 + h) * a.q_h)[p % QP];
    }
    const Range r = live_range(a, b);
    const int cs = r.base + chunk * a.chunk;  // below 2^31: the chunks cover max_len and less than one more
    const int ce = min(cs + a.chunk, r.end);
    if (cs >= r.end && a.chunks > 1) return;  // the join reads no chunk past the length

    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * S::ST * S::STAGE);
    const int32_t *table = a.table + b * a.table_b;
    const uint32_t pm = (1u << a.c.page_shift) - 1u;  // tokens of a page, less one

    // ---- the stream of this warp's steps ----
    // The cache rows (page, head, position) of 32 half steps at a time, one per
    // lane, whose pages are loaded 32 ahead.  Rows are 32-bit: 2^32 of them are
    // more than device memory holds.
    const int first = cs + warp * S::TS;
    constexpr int PAGED = 32 / HALVES;  // steps per batch
    auto token_at = [&](int step) { return first + (step + lane / HALVES) * (NW * S::TS) + 16 * (lane % HALVES); };
    auto page_at = [&](int t) -> int { return t < ce ? table[t >> a.c.page_shift] : -1; };
    uint32_t row_now, bad_now;
    auto rows_of = [&](int page, int t) {
        const bool live = (uint32_t)page < (uint32_t)a.c.num_pages;  // num_pages < 2^31
        bad_now = __ballot_sync(0xFFFFFFFFu, !live);
        row_now = live ? (((uint32_t)page * (uint32_t)a.c.heads + kvh) << a.c.page_shift) + ((uint32_t)t & pm) : 0u;
    };
    int page_next = page_at(token_at(0));
    rows_of(page_next, token_at(0));
    page_next = page_at(token_at(PAGED));
    // this lane's pieces of a row's 16 tokens
    const uint8_t *kq_lane = a.c.kq + lane * 16, *vq_lane = a.c.vq + lane * 16;
    const uint8_t *s_lane = (lane < 16 ? a.c.ks : a.c.vs) + (lane & 15) * 16;
    uint32_t k_dst[D == 256 ? PIECES / 2 : 1], v_dst[D == 256 ? PIECES / 2 : 1];  // dim 256: swizzled
#pragma unroll
    for (int i = 0; i < (D == 256 ? PIECES / 2 : 1); i++) {
        const int p = i * 32 + lane, t = p / PIECES, j = p % PIECES;
        k_dst[i] = ring + k_piece<D>(t, j);
        v_dst[i] = ring + S::TS * S::QB + v_piece<D>(t, j);
    }
    const uint32_t s_dst = ring + 2 * S::TS * S::QB + (lane < 16 ? 0 : S::TS * S::SB) + (lane & 15) * 16;
    uint32_t holes = 0;  // bit 4 * stage + half: no page
    auto fetch = [&](int step, int stage) {
        const int i0 = step % PAGED;
        if (i0 == 0 && step) {
            rows_of(page_next, token_at(step));
            page_next = page_at(token_at(step + PAGED));
        }
        const uint32_t bad = (bad_now >> (i0 * HALVES)) & ((1u << HALVES) - 1u);
        holes = (holes & ~(15u << (4 * stage))) | (bad << (4 * stage));
        const uint32_t so = (uint32_t)(stage * S::STAGE);
#pragma unroll
        for (int h = 0; h < HALVES; h++) {
            const uint32_t row = __shfl_sync(0xFFFFFFFFu, row_now, i0 * HALVES + h);
            const uint8_t *kq = kq_lane + (uint64_t)row * S::QB, *vq = vq_lane + (uint64_t)row * S::QB;
            const bool live = !((bad >> h) & 1u);
#pragma unroll
            for (int i = 0; i < PIECES / 2; i++) {
                cp_async16((D == 256 ? k_dst[i] : k_dst[0] + i * 512) + so + h * 16 * S::QB, kq + i * 512, live);
                cp_async16((D == 256 ? v_dst[i] : k_dst[0] + S::TS * S::QB + i * 512) + so + h * 16 * S::QB, vq + i * 512, live);
            }
            if ((lane & 15) < S::SB)  // 16 rows' scales: SB pieces of K by the lower lanes, of V by the upper
                cp_async16(s_dst + so + h * 16 * S::SB, s_lane + (uint64_t)row * S::SB, live);
        }
    };
#pragma unroll
    for (int i = 0; i < S::ST - 1; i++) {
        if (first + i * NW * S::TS < ce) fetch(i, i);
        cp_async_commit();
    }

    // ---- q: rotated, times a power of two that puts its largest value in
    // [2^14, 2^15), as f16 hi + lo in 16 rows of shared memory ----
    uint16_t *qs = reinterpret_cast<uint16_t *>(smem + S::QAT);
#pragma unroll
    for (int i = 0; i < QI; i++) {
        const int p = i * NW * 32 + threadIdx.x, h = p / QP;  // D / 8 lanes to a head: whole warps
        if (p >= HT * QP) break;
        float v[8] = {bf16lo(q_raw[i].x), bf16hi(q_raw[i].x), bf16lo(q_raw[i].y), bf16hi(q_raw[i].y),
                      bf16lo(q_raw[i].z), bf16hi(q_raw[i].z), bf16lo(q_raw[i].w), bf16hi(q_raw[i].w)};
        if (ROT) {  // H_k: stages 1, 2, 4 here, 8 .. k / 2 between lanes, in that order
#pragma unroll
            for (int st = 1; st < 8; st <<= 1) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    if (e & st) continue;
                    const float x = v[e], y = v[e + st];
                    v[e] = __fadd_rn(x, y);
                    v[e + st] = __fsub_rn(x, y);
                }
            }
            for (int m = 1; 8 * m < a.hk; m <<= 1) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float o = __shfl_xor_sync(0xFFFFFFFFu, v[e], m);
                    v[e] = (lane & m) ? __fsub_rn(o, v[e]) : __fadd_rn(v[e], o);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = __fmul_rn(v[e], a.ck);
        }
        float amax = absmax_tree<8>(v);
#pragma unroll
        for (int m = 1; m < QP; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
        int e = amax > 0.0f ? (int)((__float_as_uint(amax) >> 23) & 0xFF) - 127 - 14 : 0;
        e = e < -126 ? -126 : e;  // 2^-e stays finite
        const float down = a.scale < 0.0f ? -exp2i(-e) : exp2i(-e);  // scores times a positive factor: their order holds
        if (p % QP == 0) q_exp[h] = exp2i(e);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float x0 = __fmul_rn(v[2 * j], down), x1 = __fmul_rn(v[2 * j + 1], down);
            hi[j] = pack_f16(x0, x1);
            const __half2 hh = *reinterpret_cast<const __half2 *>(&hi[j]);
            if (ROT) lo[j] = pack_f16(__fsub_rn(x0, __low2float(hh)), __fsub_rn(x1, __high2float(hh)));
        }
        reinterpret_cast<uint4 *>(qs)[p] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (ROT) reinterpret_cast<uint4 *>(qs)[HT * QP + p] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();
    uint32_t qf[2 * WPT][ROT ? 4 : 2];  // B operand, column g: hi, then lo
#pragma unroll
    for (int s = 0; s < 2 * WPT; s++) {
        const int w = s >> 1;
        const int e = (D == 256 ? ((w >> 2) * 4 + c) * 32 + (w & 3) * 8 : c * (D / 4) + w * 8) + (s & 1) * 4;
        const uint2 hi = *reinterpret_cast<const uint2 *>(qs + g * D + e);
        qf[s][0] = hi.x;
        qf[s][1] = hi.y;
        if (ROT) {
            const uint2 lo = *reinterpret_cast<const uint2 *>(qs + (HT + g) * D + e);
            qf[s][ROT ? 2 : 0] = lo.x;
            qf[s][ROT ? 3 : 1] = lo.y;
        }
    }
    __syncthreads();  // q's place becomes a stage
    // Scores in units of log 2 are s * xs: xs > 0, so that a score of -inf stays one.
    float xscale[2], xs[2];  // of heads 2c and 2c + 1
#pragma unroll
    for (int i = 0; i < 2; i++) {
        xscale[i] = __fmul_rn(__fmul_rn(fabsf(a.scale), q_exp[2 * c + i]), NV ? *a.c.gk : 0.00390625f);  // (E8M0: e8m0_rel's 2^8)
        xs[i] = fmaxf(xscale[i], kTiny);
    }

    // where this lane's operands lie in a stage: tokens of other tiles follow at fixed distances
    const uint32_t k_at = k_piece<D>(tau(g), D == 64 ? c >> 1 : c) + (D == 64 ? (c & 1) * 8 : 0);
    const uint32_t k_at1 = D == 256 ? k_piece<D>(tau(g), 4 + c) : 0;
    const uint32_t ks_at = 2 * S::TS * S::QB + tau(g) * S::SB + (FMT == FP4_MXFP4 ? (D == 64 ? c >> 1 : c) : D == 64 ? c : 2 * c);
    const int vj = D == 64 ? g >> 2 : D == 128 ? g >> 1 : g, vb = D == 64 ? (g & 3) * 4 : D == 128 ? (g & 1) * 8 : 0;
    const int vsj = FMT == FP4_MXFP4 ? vj : D == 64 ? g >> 1 : D == 128 ? g : 2 * g;
    uint32_t v_at[2], vs_at[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        v_at[i] = S::TS * S::QB + v_piece<D>(tau(2 * c + i), vj) + vb;
        vs_at[i] = 2 * S::TS * S::QB + S::TS * S::SB + tau(2 * c + i) * S::SB + vsj;
    }

    // no score yet: the least finite number, so that differences stay numbers
    float m_run[2] = {-kFltMax, -kFltMax}, l_run[2] = {0.0f, 0.0f};
    uint32_t k_ref = 0, v_ref = 1;  // E8M0: the largest scale bytes so far
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; i++) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;

    float x[NT / 2][4];  // 16 tokens: rows g and g + 8, heads 2c and 2c + 1 of each
    uint32_t ph[NT], pl[NT];
    constexpr int LW = (S::TS + 31) / 32;
    uint32_t live[LW], ref_new = 1;  // a bit per token of the step, if not all take part
    bool all = true;

    // Before a step's scores: which of its tokens take part; E8M0: the largest
    // scales so far (of V: to be taken up with the step's own weights).
    auto look = [&](int t0, int stage) {
        const uint32_t at = ring + (uint32_t)(stage * S::STAGE);
        const uint32_t hole = (holes >> (4 * stage)) & 15u;
        all = t0 + S::TS <= ce && t0 >= r.begin && !hole;
        if (!all) {
#pragma unroll
            for (int i = 0; i < LW; i++) {
                const int lo = r.begin - t0 - 32 * i, hi = ce - t0 - 32 * i;  // live from lo to hi
                uint32_t v = hi >= 32 ? 0xFFFFFFFFu : hi > 0 ? (1u << hi) - 1u : 0u;
                if (lo > 0) v = lo < 32 ? v & (0xFFFFFFFFu << lo) : 0u;
                if ((hole >> (2 * i)) & 1u) v &= 0xFFFF0000u;
                if ((hole >> (2 * i)) & 2u) v &= 0x0000FFFFu;
                live[i] = v;
                // whatever scales the others have (NaN among them) becomes 0
                if (lane + 32 * i < S::TS && !((v >> lane) & 1u)) {
                    const uint32_t ks = at + 2 * S::TS * S::QB + (lane + 32 * i) * S::SB;
#pragma unroll
                    for (int k = 0; k < S::SB; k += 2) {
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(ks + k), "h"((uint16_t)0) : "memory");
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(ks + S::TS * S::SB + k), "h"((uint16_t)0) : "memory");
                    }
                }
            }
            __syncwarp();
        }
        if (!NV) {
            // bytes as pairs of 16-bit lanes; the rows of K, then those of V
            constexpr int W = S::TS * S::SB / 4;  // words of each
            static_assert(W % 32 == 0, "a warp's words belong to K or to V");
            uint32_t ek = 0, ev = 0;
#pragma unroll
            for (int i = 0; i < 2 * W / 32; i++) {
                uint32_t q;
                lds(at + 2 * S::TS * S::QB + (i * 32 + lane) * 4, &q, 1);
                const uint32_t e = __vmaxu2(q & 0x00FF00FFu, (q >> 8) & 0x00FF00FFu);
                if (i * 32 < W) ek = __vmaxu2(ek, e);
                else ev = __vmaxu2(ev, e);
            }
            const uint32_t k2 = k_ref * 0x10001u, v2 = ref_new * 0x10001u;
            if (__any_sync(0xFFFFFFFFu, __vmaxu2(ek, k2) != k2 || __vmaxu2(ev, v2) != v2)) {
                k_ref = max(k_ref, __reduce_max_sync(0xFFFFFFFFu, max(ek & 0xFFFFu, ek >> 16)));
                ref_new = max(ref_new, __reduce_max_sync(0xFFFFFFFFu, max(ev & 0xFFFFu, ev >> 16)));
#pragma unroll
                for (int i = 0; i < 2; i++) xs[i] = fmaxf(__fmul_rn(xscale[i], exp2i((int)k_ref - 127)), kTiny);
            }
        }

    };

    // x = q . k of a step's tokens
    auto scores = [&](int stage) {
        const uint32_t at = ring + (uint32_t)(stage * S::STAGE);
#pragma unroll
        for (int j = 0; j < NT / 2; j++) {
            uint32_t w[2][WPT], sc[2][(WPT + 1) / 2];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const int n = 2 * j + r;
                lds(at + k_at + n * 8 * S::QB, w[r], D == 64 ? 2 : 4);
                if (D == 256) lds(at + k_at1 + n * 8 * S::QB, w[r] + WPT / 2, 4);
                const uint32_t ks = at + ks_at + n * 8 * S::SB;
                if (FMT == FP4_MXFP4) {  // one scale per 4 words (dim 64: shared by two lanes)
#pragma unroll
                    for (int p = 0; p < (D == 256 ? 2 : 1); p++) {
                        const uint32_t f = e8m0_rel(lds8(ks + 4 * p), k_ref);
#pragma unroll
                        for (int i = 0; i < (D == 64 ? 1 : 2); i++) sc[r][2 * p + i] = f;
                    }
                } else if (D == 64) {
                    const uint32_t e = lds8(ks);
                    sc[r][0] = NV ? e4m3x2_to_f16x2(e * 0x101u) : e8m0_rel(e, k_ref);
                } else {
#pragma unroll
                    for (int p = 0; p < D / 128; p++) {
                        const uint32_t e = lds16(ks + 8 * p);
                        if (NV) {
                            const uint32_t f = e4m3x2_to_f16x2(e);
                            sc[r][2 * p] = __byte_perm(f, 0, 0x1010);
                            sc[r][2 * p + 1] = __byte_perm(f, 0, 0x3232);
                        } else {
                            sc[r][2 * p] = e8m0_rel(e & 0xFF, k_ref);
                            sc[r][2 * p + 1] = e8m0_rel(e >> 8, k_ref);
                        }
                    }
                }
            }
            x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < WPT; i++) {
                uint32_t h0[4], h1[4];
                e2m1x8_to_f16(w[0][i], h0);
                e2m1x8_to_f16(w[1][i], h1);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    h0[k] = mul_f16x2(h0[k], sc[0][i >> 1]);
                    h1[k] = mul_f16x2(h1[k], sc[1][i >> 1]);
                }
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    mma_f16(x[j], h0[2 * k], h1[2 * k], h0[2 * k + 1], h1[2 * k + 1], qf[2 * i + k][0], qf[2 * i + k][1]);
                    if (ROT)
                        mma_f16(x[j], h0[2 * k], h1[2 * k], h0[2 * k + 1], h1[2 * k + 1], qf[2 * i + k][ROT ? 2 : 0],
                                qf[2 * i + k][ROT ? 3 : 1]);
                }
            }
        }
    };

    // the step's weights, with everything so far on the new maxima
    auto weights = [&]() {
        if (!all) {
#pragma unroll
            for (int j = 0; j < NT / 2; j++) {
                const uint32_t v = live[j / 2] >> (16 * (j & 1) + tau(g));
                if (!(v & 1u)) x[j][0] = x[j][1] = -INFINITY;
                if (!(v & 0x100u)) x[j][2] = x[j][3] = -INFINITY;
            }
        }
        float m_new[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            float mx = fmaxf(x[0][i], x[0][2 + i]);
#pragma unroll
            for (int j = 1; j < NT / 2; j++) mx = fmaxf(mx, fmaxf(x[j][i], x[j][2 + i]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
            m_new[i] = fmaxf(m_run[i], __fmul_rn(mx, xs[i]));
        }
        if (__any_sync(0xFFFFFFFFu, m_new[0] > m_run[0] || m_new[1] > m_run[1]) || (!NV && ref_new != v_ref)) {
            const float f = NV ? 1.0f : exp2i(max((int)v_ref - (int)ref_new, -127));
            float alpha[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                alpha[i] = m_new[i] > m_run[i] ? ex2(__fsub_rn(m_run[i], m_new[i])) : 1.0f;  // 0 at first
                l_run[i] = __fmul_rn(l_run[i], alpha[i]);
                alpha[i] = __fmul_rn(alpha[i], f);
                m_run[i] = m_new[i];
            }
#pragma unroll
            for (int i = 0; i < MT; i++) {
                acc[i][0] = __fmul_rn(acc[i][0], alpha[0]);
                acc[i][1] = __fmul_rn(acc[i][1], alpha[1]);
                acc[i][2] = __fmul_rn(acc[i][2], alpha[0]);
                acc[i][3] = __fmul_rn(acc[i][3], alpha[1]);
            }
            v_ref = ref_new;
        }
        const float off0 = __fsub_rn(kPShift, m_run[0]), off1 = __fsub_rn(kPShift, m_run[1]);
#pragma unroll
        for (int j = 0; j < NT / 2; j++) {
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float p0 = ex2(__fmaf_rn(x[j][2 * r], xs[0], off0)), p1 = ex2(__fmaf_rn(x[j][2 * r + 1], xs[1], off1));
                l_run[0] = __fadd_rn(l_run[0], p0);
                l_run[1] = __fadd_rn(l_run[1], p1);
                const uint32_t h = pack_f16(p0, p1);
                ph[2 * j + r] = transpose_8x8(h);  // head g, tokens of rows 2c and 2c + 1: V's B operand
                if (!BF16OUT) {
                    const __half2 hh = *reinterpret_cast<const __half2 *>(&h);
                    pl[2 * j + r] = transpose_8x8(pack_f16(__fsub_rn(p0, __low2float(hh)), __fsub_rn(p1, __high2float(hh))));
                }
            }
        }
    };

    auto values = [&](int stage) {
        const uint32_t at = ring + (uint32_t)(stage * S::STAGE);
#pragma unroll
        for (int j = 0; j < NT / 2; j++) {
            uint32_t w[4][VW], s01[(VW + 1) / 2], s23[(VW + 1) / 2], e[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                lds(at + v_at[i & 1] + (16 * j + 8 * (i >> 1)) * S::QB, w[i], VW);
                const uint32_t vs = at + vs_at[i & 1] + (16 * j + 8 * (i >> 1)) * S::SB;
                e[i] = FMT != FP4_MXFP4 && D == 256 ? lds16(vs) : lds8(vs);
            }
#pragma unroll
            for (int k = 0; k < (VW + 1) / 2; k++) {
                const int sh = FMT == FP4_MXFP4 ? 0 : 8 * k;  // dim 256: both scales of a 16-bit load
                if (NV && D == 256) {
                    s01[k] = e4m3x2_to_f16x2(__byte_perm(e[0], e[1], k ? 0x0051 : 0x0040));
                    s23[k] = e4m3x2_to_f16x2(__byte_perm(e[2], e[3], k ? 0x0051 : 0x0040));
                } else if (NV) {
                    s01[k] = e4m3x2_to_f16x2(e[0] | (e[1] << 8));
                    s23[k] = e4m3x2_to_f16x2(e[2] | (e[3] << 8));
                } else {
                    s01[k] = e8m0_rel2((e[0] >> sh) & 0xFF, (e[1] >> sh) & 0xFF, v_ref);
                    s23[k] = e8m0_rel2((e[2] >> sh) & 0xFF, (e[3] >> sh) & 0xFF, v_ref);
                }
            }
#pragma unroll
            for (int i = 0; i < VW; i++) {
                const uint32_t M = 0x0F0F0F0Fu;
                uint32_t a0[4], a1[4], a2[4], a3[4];
                e2m1x8_to_f16(select_bits(w[0][i], w[1][i] << 4, M), a0);
                e2m1x8_to_f16(select_bits(w[0][i] >> 4, w[1][i], M), a1);
                e2m1x8_to_f16(select_bits(w[2][i], w[3][i] << 4, M), a2);
                e2m1x8_to_f16(select_bits(w[2][i] >> 4, w[3][i], M), a3);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    a0[k] = mul_f16x2(a0[k], s01[i >> 1]);
                    a1[k] = mul_f16x2(a1[k], s01[i >> 1]);
                    a2[k] = mul_f16x2(a2[k], s23[i >> 1]);
                    a3[k] = mul_f16x2(a3[k], s23[i >> 1]);
                    mma_f16(acc[4 * i + k], a0[k], a1[k], a2[k], a3[k], ph[2 * j], ph[2 * j + 1]);
                    if (!BF16OUT) mma_f16(acc[4 * i + k], a0[k], a1[k], a2[k], a3[k], pl[2 * j], pl[2 * j + 1]);
                }
            }
        }
    };

    // two steps to a trip: stages are then constants in all addresses
    static_assert(S::ST == 2, "one stage is read while the other is filled");
    auto advance = [&](int t0, int step, int stage) {
        cp_async_wait<0>();
        __syncwarp();
        // into the stage of the step before this one, which all lanes have left
        if (t0 + NW * S::TS < ce) fetch(step + 1, stage ^ 1);
        cp_async_commit();
        look(t0, stage);
        scores(stage);
        weights();
        values(stage);
    };
    for (int t0 = first, step = 0; t0 < ce; t0 += 2 * NW * S::TS, step += 2) {
        advance(t0, step, 0);
        if (t0 + NW * S::TS < ce) advance(t0 + NW * S::TS, step + 1, 1);
    }

    // ---- join the warps ----
    // Whether plain_warp has to work this out: a NaN scale; a maximum from kFar
    // on; one that was passed later, whose weights past f16's range have left no
    // finite outputs, though there is a sum (of queries that are NaN there is
    // none, and the result is right).
    bool plain = !NV && max(k_ref, v_ref) == 255;
#pragma unroll
    for (int i = 0; i < 2; i++)
        plain |= (fabsf(m_run[i]) >= kFar && fabsf(m_run[i]) < kFltMax) || (l_run[i] > 0.0f && !(fabsf(acc[0][i]) <= kFltMax));
    const bool any_plain = __any_sync(0xFFFFFFFFu, plain);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l_run[i] = __fadd_rn(l_run[i], __shfl_xor_sync(0xFFFFFFFFu, l_run[i], d));
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with the ring
    float *so = reinterpret_cast<float *>(smem) + warp * HT * D;
    if (g == 0) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            sm_m[warp][2 * c + i] = m_run[i];
            sm_l[warp][2 * c + i] = l_run[i];
        }
    }
    // E8M0: without 2^15 and e8m0_rel's 2^8, so that scales up to the largest have
    // finite sums (from 2^-126 on the factor is exact)
    const float vf = NV ? 1.0f : __fmul_rn(exp2i((int)v_ref - 127), 1.0f / (256.0f * kUnit));
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int d = g * (D / 8) + 2 * i;
        *reinterpret_cast<float2 *>(so + (2 * c) * D + d) = make_float2(__fmul_rn(acc[i][0], vf), __fmul_rn(acc[i][2], vf));
        *reinterpret_cast<float2 *>(so + (2 * c + 1) * D + d) = make_float2(__fmul_rn(acc[i][1], vf), __fmul_rn(acc[i][3], vf));
    }
    if (__builtin_expect(any_plain, 0)) {
        __syncwarp();  // over what was stored just now
        plain_warp<FMT, D, S::TS>(a, so, sm_m[warp], sm_l[warp]);
    }
    __syncthreads();
    if (threadIdx.x < nh) {  // the rows' factors, per warp
        const int h = threadIdx.x;
        float m = sm_m[0][h], l = 0.0f, f[NW];
#pragma unroll
        for (int w = 1; w < NW; w++) m = fmaxf(m, sm_m[w][h]);
#pragma unroll
        for (int w = 0; w < NW; w++) {
            f[w] = ex2(__fsub_rn(sm_m[w][h], m));  // without a score l is 0
            l = __fmaf_rn(f[w], sm_l[w][h], l);
        }
        const int64_t row = (int64_t)b * a.q_heads + h0 + h;
        float norm = 1.0f;
        if (a.chunks > 1) {
            a.part_ml[row * a.chunks + chunk] = make_float2(m, l);
        } else {
            norm = l == 0.0f ? 0.0f : __fdiv_rn(NV ? *a.c.gv : kUnit, l);
            if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fsub_rn(m, kPShift), log2f(l)), 0.693147180559945f);
        }
#pragma unroll
        for (int w = 0; w < NW; w++) sm_m[w][h] = __fmul_rn(f[w], norm);
    }
    __syncthreads();
    float4 *o4 = reinterpret_cast<float4 *>(smem);
    for (int i = threadIdx.x; i < nh * D / 4; i += NW * 32) {
        const int h = i / (D / 4);
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float4 p = o4[w * (HT * D / 4) + i];
            const float f = sm_m[w][h];
            t.x = __fmaf_rn(f, p.x, t.x);
            t.y = __fmaf_rn(f, p.y, t.y);
            t.z = __fmaf_rn(f, p.z, t.z);
            t.w = __fmaf_rn(f, p.w, t.w);
        }
        if (a.chunks > 1)
            reinterpret_cast<float4 *>(a.part_o)[(((int64_t)b * a.q_heads + h0 + h) * a.chunks + chunk) * (D / 4) + i % (D / 4)] = t;
        else
            o4[i] = t;  // this thread's own element of warp 0's part
    }
    if (a.chunks > 1) return;
    __syncthreads();
    write_rows<D, BF16OUT>(reinterpret_cast<const float *>(smem), nh, (int64_t)b * a.q_heads + h0, a, NW * 32);
}

// Joins a row's chunks: o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c.
template <int FMT, int D, int BF16OUT>
__global__ void __launch_bounds__(kJoin) join_kernel(const __grid_constant__ Args a)
{
    constexpr int LANES = D / 4, GROUPS = kJoin / LANES;
    __shared__ float f[kMaxChunks];
    __shared__ float red[2][kJoin / 32];
    __shared__ __align__(16) float o[GROUPS][D];
    grid_dep_launch();
    grid_dep_wait();
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)b * a.q_heads + blockIdx.x;
    const Range r = live_range(a, b);
    const int n = r.end > r.base ? (int)((r.end - r.base + a.chunk - 1) / a.chunk) : 0;
    const float2 *ml = a.part_ml + row * a.chunks;
    float m = -kFltMax;
    for (int i = threadIdx.x; i < n; i += kJoin) {
        f[i] = ml[i].x;
        m = fmaxf(m, f[i]);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoin / 32; i++) m = fmaxf(m, red[0][i]);
    float l = 0.0f;
    for (int i = threadIdx.x; i < n; i += kJoin) {
        f[i] = ex2(__fsub_rn(f[i], m));
        l = __fmaf_rn(f[i], ml[i].y, l);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xFFFFFFFFu, l, s));
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    l = red[1][0];
#pragma unroll
    for (int i = 1; i < kJoin / 32; i++) l = __fadd_rn(l, red[1][i]);
    const int d4 = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + row * a.chunks * D) + d4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = grp; i < n; i += GROUPS) {
        const float4 t = po[(int64_t)i * LANES];
        const float w = f[i];
        s.x = __fmaf_rn(w, t.x, s.x);
        s.y = __fmaf_rn(w, t.y, s.y);
        s.z = __fmaf_rn(w, t.z, s.z);
        s.w = __fmaf_rn(w, t.w, s.w);
    }
    *reinterpret_cast<float4 *>(&o[grp][4 * d4]) = s;
    __syncthreads();
    const float gv = FMT == FP4_NVFP4 ? *a.c.gv : 1.0f, unit = FMT == FP4_NVFP4 ? l : __fmul_rn(l, 1.0f / kUnit);
    for (int d = threadIdx.x; d < D; d += kJoin) {
        float t = o[0][d];
#pragma unroll
        for (int k = 1; k < GROUPS; k++) t = __fadd_rn(t, o[k][d]);
        o[0][d] = l == 0.0f ? 0.0f : __fmul_rn(__fdiv_rn(t, unit), gv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row] = l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fsub_rn(m, kPShift), log2f(l)), 0.693147180559945f);
    __syncthreads();
    write_rows<D, BF16OUT>(o[0], 1, row, a, kJoin);
}

// The same, a warp to a row: for up to 4 chunks, or very many rows, where a CTA
// to a row is mostly its start (4096 rows of up to 4 chunks: the whole call 76.6
// us, with 128 threads a row 80.2, with 256 85.4).  For 8 chunks of 512 rows it
// is the other way round (48.0 and 46.2 us): a warp reads them one by one.
constexpr int kJoinRows = 2;
template <int FMT, int D, int BF16OUT>
__global__ void __launch_bounds__(32 * kJoinRows) join_rows_kernel(const __grid_constant__ Args a, int64_t rows)
{
    constexpr int P = (D + 127) / 128;  // 16-byte pieces of a lane
    __shared__ __align__(16) float o[kJoinRows][D];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * kJoinRows, row = row0 + warp;
    if (row < rows) {
        const Range r = live_range(a, (int)(row / a.q_heads));
        const int n = r.end > r.base ? (int)((r.end - r.base + a.chunk - 1) / a.chunk) : 0;
        const float2 *ml = a.part_ml + row * a.chunks;
        float m = -kFltMax, l = 0.0f;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, ml[i].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        float4 s[P] = {};
        const float4 *po = reinterpret_cast<const float4 *>(a.part_o + row * a.chunks * D) + lane;
#pragma unroll 4
        for (int i = 0; i < n; i++) {
            const float2 t = ml[i];
            const float w = ex2(__fsub_rn(t.x, m));
            l = __fmaf_rn(w, t.y, l);
#pragma unroll
            for (int k = 0; k < P; k++) {
                if (D < 128 && lane >= D / 4) continue;
                const float4 v = po[(int64_t)i * (D / 4) + 32 * k];
                s[k].x = __fmaf_rn(w, v.x, s[k].x);
                s[k].y = __fmaf_rn(w, v.y, s[k].y);
                s[k].z = __fmaf_rn(w, v.z, s[k].z);
                s[k].w = __fmaf_rn(w, v.w, s[k].w);
            }
        }
        const float norm = l == 0.0f ? 0.0f : __fdiv_rn(FMT == FP4_NVFP4 ? *a.c.gv : kUnit, l);
        if (a.lse && lane == 0)
            a.lse[row] = l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fsub_rn(m, kPShift), log2f(l)), 0.693147180559945f);
#pragma unroll
        for (int k = 0; k < P; k++)
            if (D >= 128 || lane < D / 4)
                *reinterpret_cast<float4 *>(&o[warp][4 * (lane + 32 * k)]) =
                    make_float4(__fmul_rn(s[k].x, norm), __fmul_rn(s[k].y, norm), __fmul_rn(s[k].z, norm), __fmul_rn(s[k].w, norm));
    }
    __syncthreads();
    write_rows<D, BF16OUT>(o[0], (int)(rows - row0 < kJoinRows ? rows - row0 : kJoinRows), row0, a, 32 * kJoinRows);
}

// ---------------------------------------------------------------------------
// How a call is cut: tokens per chunk (a multiple of kAlign) and chunks per
// sequence, from its sizes alone (lengths live on the device).
struct Plan {
    int64_t chunk;
    int chunks;
};

// The cheapest number of chunks by a model fitted to sweeps of chunk sizes on
// the B200 (batch 1 x 262143 tokens to 64 x 8192, dims 64, 128, 256; time in
// units of a warp's step): a CTA costs its warps' steps and 2.1 for its start
// and end; whole rounds of the SMs' resident CTAs cost that each, a last round
// that is partly filled 0.3 to 1 of it, a first one 0.6 to 1; joining n chunks
// 0.6 + 0.02 n; in a batch, whose lengths differ as a rule, half a CTA more
// (64 sequences of 1 to 8192 tokens: 4096 a chunk 98 us, 2048 88, 1024 88).
// (One exact round for the long sequence: 75 us; 1.7 rounds of
// half the chunk 79 us, 1.2 rounds 87 us.)
static Plan search(int64_t batch, int kv_heads, int head_tiles, int dim, int64_t tokens, int sms)
{
    const int64_t rows = batch * kv_heads * head_tiles, slots = (int64_t)sms * (dim == 256 ? 2 : 4);
    const int64_t step = NW * (dim == 64 ? 64 : dim == 128 ? 32 : 16);
    Plan best = {};
    double least = 0.0;
    const auto consider = [&](int64_t n) {
        const int64_t chunk = ((tokens + n - 1) / n + kAlign - 1) / kAlign * kAlign;
        n = (tokens + chunk - 1) / chunk;
        const double t = 2.1 + (double)((chunk + step - 1) / step), rounds = (double)(rows * n) / (double)slots;
        const double whole = floor(rounds), part = rounds - whole;
        const double cost = t * ((rounds < 1.0 ? 0.6 + 0.4 * rounds : whole + (part > 0.0 ? 0.3 + 0.7 * part : 0.0)) + (batch > 1 ? 0.5 : 0.0)) +
                            (n > 1 ? 0.6 + 0.02 * (double)n : 0.0);
        if (best.chunks == 0 || cost < least) {
            least = cost;
            best = {chunk, (int)n};
        }
        return chunk > kAlign;
    };
    for (int64_t n = 1; n <= kMaxChunks && consider(n); n += 1 + n / 32) {
    }
    for (int64_t r = 1; r <= 2; r++)  // whole rounds
        if (r * slots / rows >= 1 && r * slots / rows <= kMaxChunks) consider(r * slots / rows);
    return best;
}

// The last search of this thread is kept: a decode loop asks for the same sizes
// again and again, and a search takes longer than a launch.
static Plan plan(int64_t batch, int kv_heads, int head_tiles, int dim, int64_t tokens, int sms)
{
    struct Last {
        int64_t key[6];
        Plan p;
    };
    static thread_local Last last = {{-1, -1, -1, -1, -1, -1}, {}};
    const int64_t key[6] = {batch, kv_heads, head_tiles, dim, tokens, sms};
    if (!std::equal(key, key + 6, last.key)) {
        last.p = search(batch, kv_heads, head_tiles, dim, tokens, sms);
        std::copy(key, key + 6, last.key);
    }
    return last.p;
}

// Tokens that a sequence's chunks have to cover: its live range from the last
// multiple of kAlign before it.
static int64_t span(int64_t max_len, int64_t window)
{
    return window > 0 && max_len > window ? window + kAlign - 1 : max_len;
}

template <int FMT, int D, int BF16OUT>
static cudaError_t launch_t(const Args &a, int64_t batch, int kv_heads, cudaStream_t st)
{
    using S = Shape<FMT, D>;
    auto kern = a.hk ? paged_kernel<FMT, D, BF16OUT, true> : paged_kernel<FMT, D, BF16OUT, false>;
    static std::atomic<uint64_t> done[2];
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), S::SMEM, done[a.hk ? 1 : 0]);
    if (e != cudaSuccess) return e;
    e = launch_k(kern, dim3((unsigned)(a.chunks * a.head_tiles), (unsigned)kv_heads, (unsigned)batch), dim3(NW * 32), S::SMEM, st, true, a);
    if (e != cudaSuccess || a.chunks == 1) return e;
    const int64_t rows = batch * a.q_heads;
    if (a.chunks <= 4 || rows >= 2048)
        return launch_k(join_rows_kernel<FMT, D, BF16OUT>, dim3((unsigned)((rows + kJoinRows - 1) / kJoinRows)), dim3(32 * kJoinRows), 0, st, true, a, rows);
    return launch_k(join_kernel<FMT, D, BF16OUT>, dim3((unsigned)a.q_heads, (unsigned)batch), dim3(kJoin), 0, st, true, a);
}

template <int FMT>
static cudaError_t launch_f(const Args &a, int dim, int bf16out, int64_t batch, int kv_heads, cudaStream_t st)
{
    if (bf16out)
        return dim == 64    ? launch_t<FMT, 64, 1>(a, batch, kv_heads, st)
               : dim == 128 ? launch_t<FMT, 128, 1>(a, batch, kv_heads, st)
                            : launch_t<FMT, 256, 1>(a, batch, kv_heads, st);
    return dim == 64    ? launch_t<FMT, 64, 0>(a, batch, kv_heads, st)
           : dim == 128 ? launch_t<FMT, 128, 0>(a, batch, kv_heads, st)
                        : launch_t<FMT, 256, 0>(a, batch, kv_heads, st);
}

}  // namespace attn

size_t paged_attention_workspace_bytes(int64_t batch, int q_heads, int kv_heads, int dim, int64_t max_len, int64_t window, int sms)
{
    const int tiles = (q_heads / kv_heads + attn::HT - 1) / attn::HT;
    const attn::Plan p = attn::plan(batch > 0 ? batch : 1, kv_heads, tiles, dim, attn::span(max_len, window), sms);
    if (p.chunks == 1) return 0;
    return (size_t)batch * q_heads * p.chunks * ((size_t)dim + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const KvView &c, int dim, int fmt, int hk, float ck, const uint16_t *q, int64_t batch,
                                   int q_heads, int64_t q_b, int64_t q_h, const int32_t *table, int64_t table_b,
                                   int64_t table_cols, const int32_t *lens, int64_t max_len, float scale, int64_t window,
                                   int bf16out, void *out, float *lse, void *ws, int sms, cudaStream_t st)
{
    attn::Args a = {};
    a.c = c;
    a.q = q;
    a.q_b = q_b;
    a.q_h = q_h;
    a.table = table;
    a.table_b = table_b;
    a.table_tokens = (int)std::min<int64_t>(table_cols << c.page_shift, int64_t(1) << 30);
    a.lens = lens;
    a.max_len = (int)max_len;
    a.window = (int)std::min<int64_t>(window, int64_t(1) << 30);
    a.group = q_heads / c.heads;
    a.head_tiles = (a.group + attn::HT - 1) / attn::HT;
    a.q_heads = q_heads;
    a.scale = (float)((double)scale * 1.4426950408889634);
    a.ck = ck;
    a.hk = hk;
    const attn::Plan p = attn::plan(batch, c.heads, a.head_tiles, dim, attn::span(max_len, window), sms);
    a.chunk = (int)p.chunk;
    a.chunks = p.chunks;
    a.out = out;
    a.lse = lse;
    a.part_o = static_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (p.chunks > 1 ? (size_t)batch * q_heads * p.chunks * dim : 0));
    if (fmt == FP4_MXFP4) return attn::launch_f<FP4_MXFP4>(a, dim, bf16out, batch, c.heads, st);
    if (fmt == FP4_NVFP4) return attn::launch_f<FP4_NVFP4>(a, dim, bf16out, batch, c.heads, st);
    return attn::launch_f<FP4_MXFP4_16>(a, dim, bf16out, batch, c.heads, st);
}

}  // namespace fp4
