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
// token and head, and every element has to become a 16-bit operand first:
// the issue slots of that conversion come next after HBM.  So:
//   * The products run on mma.sync m16n8k16 (f16 in, fp32 sums) from registers.
//     tcgen05 would need the dequantized tile written to shared or tensor
//     memory first, at four times the packed bytes; its rate is not what
//     is short here (up to 8 query rows per key head).
//   * The order of a product's inner index is free, so each lane's operand
//     elements are whole consecutive bytes of a token's row: K is the B operand
//     (8 tokens a tile, a lane holds dim/4 consecutive elements of one token),
//     V the A operand (a lane holds dim/8 consecutive elements of 4 tokens).
//     A byte of K is a register pair after one conversion; two tokens' V
//     bytes are merged nibble by nibble first.  The scores' result registers
//     are then the next product's B operand as they are: nothing is exchanged.
//   * E2M1 times its block scale is exact in f16: for NVFP4 the E4M3 scale
//     itself (6 significant bits, 2^-10 .. 2688), for E8M0 a power of two
//     relative to the row's (K) or the running (V) largest scale.
//   * q in f16 as a power of two times hi + lo: query rows 0-7 of the product
//     hold hi and rows 8-15 lo, so 22 bits cost nothing for groups of up to 8.
//     Weights w_t are rounded to f16 (11 bits, scaled by 2^15 so that they
//     stay normal down to 2^-29 of the largest; below, to steps of 2^-39), and
//     for fp32 output are split into hi + lo as well, a second product.
//   * Every warp streams its own steps of 16 or 32 tokens through its own ring
//     of cp.async stages: no barrier among warps until their results are
//     joined.  Rows lie swizzled, so all operand loads are free of bank conflicts.
// Long sequences are cut into chunks of tokens over CTAs; a second kernel
// joins the chunks.  The cut depends on the call's sizes only, and every sum
// has a fixed order, so results repeat bit for bit.
#include <math.h>

#include "frag.cuh"
#include "kv.cuh"
#include "sm100.cuh"

namespace fp4 {
namespace attn {

constexpr int NW = 4;           // warps per CTA, each on its own tokens
constexpr int HT = 8;           // query heads per CTA
constexpr float kPShift = 15.0f;  // weights are 2^15 w / w_max, inside f16's range
constexpr int kMaxChunks = 1024;

struct Args {
    KvView c;
    const uint16_t *q;
    int64_t q_b, q_h;  // strides, elements
    const int32_t *table;
    int64_t table_b;       // row stride of the page table
    int64_t table_tokens;  // tokens that a row of the table reaches
    const int32_t *lens;
    int64_t max_len;
    int64_t window;        // 0 = none
    int group, head_tiles, q_heads;
    float scale;           // times log2(e)
    float ck;
    int hk;
    int64_t chunk;         // tokens per chunk, a multiple of 32
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
    static constexpr int TS = D == 256 ? 16 : 32;                // tokens per step
    static constexpr int STAGE = 2 * TS * (QB + SB);             // bytes: K, V elements, K, V scales
    static constexpr int ST = D == 64 ? 4 : 3;                   // stages per warp
    static constexpr int RING = NW * ST * STAGE;
    static constexpr int JOIN = NW * HT * D * 4;                 // the warps' results, over the ring
    static constexpr int QF = 2 * HT * D * 2;                    // hi and lo of q
    static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + QF;
};

FP4_DEV float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes global -> shared, or 16 zero bytes.
FP4_DEV void cp_async16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
FP4_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
FP4_DEV void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

FP4_DEV void lds(uint32_t a, uint32_t *w, int n)
{
    if (n == 1)
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(a));
    else if (n == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
    else
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
}
FP4_DEV uint32_t lds8(uint32_t a)
{
    uint16_t v;
    asm volatile("{\n\t.reg .u8 t;\n\tld.shared.u8 t, [%1];\n\tcvt.u16.u8 %0, t;\n\t}" : "=h"(v) : "r"(a));
    return v;
}
FP4_DEV uint32_t lds16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

// The token of column n in a tile of 8 (an involution).  Columns 2m and 2m+1
// are tokens of opposite parity, for K's 16-byte loads; even columns are
// tokens 0, 3, 4, 7, for V's: both then touch every bank once.
__host__ __device__ constexpr int tau(int n) { return n ^ ((n >> 1) & 1); }

// Byte offset of 16-byte piece j of row t in the K and V element arrays of a stage.
template <int D>
FP4_DEV uint32_t k_piece(int t, int j)
{
    if (D == 64) return (uint32_t)((t ^ ((t >> 2) & 1)) * 32 + j * 16);
    if (D == 128) return (uint32_t)(t * 64 + j * 16);
    return (uint32_t)(t * 128 + (j ^ ((t & 1) << 2)) * 16);
}
template <int D>
FP4_DEV uint32_t v_piece(int t, int j)
{
    if (D == 64) return (uint32_t)((t ^ ((t >> 2) & 1)) * 32 + j * 16);
    if (D == 128) return (uint32_t)(t * 64 + (j ^ (((t >> 2) & 1) << 1)) * 16);
    return (uint32_t)(t * 128 + (j ^ (((t & 1) | (((t >> 2) & 1) << 1)) << 1)) * 16);
}

// the same for two bytes, one in each half
FP4_DEV uint32_t e8m0_rel2(uint32_t e0, uint32_t e1, uint32_t ref)
{
    const int t0 = (int)e0 - (int)ref + 23, t1 = (int)e1 - (int)ref + 23;
    return ((uint32_t)(t0 > 0 ? t0 : 0) << 10) | ((uint32_t)(t1 > 0 ? t1 : 0) << 26);
}

// The live range of a sequence's tokens, and where its chunks start.
struct Range {
    int64_t begin, end, base;
};
FP4_DEV Range live_range(const Args &a, int b)
{
    Range r;
    int64_t n = a.lens[b];
    n = n < a.max_len ? n : a.max_len;
    n = n < a.table_tokens ? n : a.table_tokens;
    r.end = n > 0 ? n : 0;
    r.begin = a.window > 0 && r.end > a.window ? r.end - a.window : 0;
    r.base = r.begin & ~(int64_t)31;
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
        for (int i = threadIdx.x; i < rows * D; i += nt) store_out<BF16OUT>(a.out, out_row * D + i, o[i]);
    }
}

template <int FMT, int D, int BF16OUT>
__global__ void __launch_bounds__(NW * 32, D == 256 ? 2 : 4) paged_kernel(const __grid_constant__ Args a)
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
    const Range r = live_range(a, b);
    const int64_t cs = r.base + chunk * a.chunk;
    const int64_t ce = min(cs + a.chunk, r.end);
    if (cs >= r.end && a.chunks > 1) return;  // the join reads no chunk past the length

    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * S::ST * S::STAGE);
    const int32_t *table = a.table + b * a.table_b;
    const int pm = (1 << a.c.page_shift) - 1;

    // ---- the stream of this warp's steps ----
    const int64_t first = cs + warp * S::TS;
    auto page_at = [&](int64_t t) -> int { return t < ce ? __ldg(table + (t >> a.c.page_shift)) : -1; };
    int next_page[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; h++) next_page[h] = page_at(first + 16 * h);
    uint32_t holes = 0;  // bit 2 * stage + half: no page
    auto fetch = [&](int64_t t0, int stage) {
        const uint32_t dst = ring + (uint32_t)(stage * S::STAGE);
#pragma unroll
        for (int h = 0; h < HALVES; h++) {
            const int page = next_page[h];
            const bool live = (uint64_t)(int64_t)page < (uint64_t)a.c.num_pages;
            holes = (holes & ~(1u << (2 * stage + h))) | ((live ? 0u : 1u) << (2 * stage + h));
            next_page[h] = page_at(t0 + NW * S::TS + 16 * h);
            const int64_t row = live ? ((((int64_t)page * a.c.heads + kvh) << a.c.page_shift) + ((t0 + 16 * h) & pm)) : 0;
            const uint8_t *kq = a.c.kq + row * S::QB, *vq = a.c.vq + row * S::QB;
#pragma unroll
            for (int i = 0; i < PIECES / 2; i++) {
                const int p = i * 32 + lane, t = p / PIECES, j = p % PIECES;
                cp_async16(dst + k_piece<D>(16 * h + t, j), kq + p * 16, live);
                cp_async16(dst + S::TS * S::QB + v_piece<D>(16 * h + t, j), vq + p * 16, live);
            }
            if ((lane & 15) < S::SB) {  // 16 rows' scales: SB pieces of K by the lower lanes, of V by the upper
                const uint8_t *s = (lane < 16 ? a.c.ks : a.c.vs) + row * S::SB;
                cp_async16(dst + 2 * S::TS * S::QB + (lane < 16 ? 0 : S::TS * S::SB) + h * 16 * S::SB + (lane & 15) * 16,
                           s + (lane & 15) * 16, live);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < S::ST - 1; i++) {
        if (first + (int64_t)i * NW * S::TS < ce) fetch(first + (int64_t)i * NW * S::TS, i);
        cp_async_commit();
    }

    // ---- q: rotated, times a power of two that puts its largest value in
    // [2^14, 2^15), as f16 hi + lo in 16 rows of shared memory ----
    uint16_t *qs = reinterpret_cast<uint16_t *>(smem + (S::SMEM - S::QF));
    for (int i = threadIdx.x; i < (HT * WPT < 32 ? 32 : HT * WPT); i += NW * 32) {  // whole warps: lanes exchange values
        const int h = i / WPT, u = i % WPT;
        uint4 raw[4] = {};
        if (h < nh) {
            const uint4 *p = reinterpret_cast<const uint4 *>(a.q + b * a.q_b + (int64_t)(h0 + h) * a.q_h + u * 32);
#pragma unroll
            for (int e = 0; e < 4; e++) raw[e] = __ldg(p + e);
        }
        float v[32];
        unpack_unit(raw, v);
        rotate_unit(v, a.hk, a.ck, lane);
        float amax = absmax_tree<32>(v);
#pragma unroll
        for (int m = 1; m < WPT; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
        if (h >= HT) continue;
        int e = amax > 0.0f ? (int)((__float_as_uint(amax) >> 23) & 0xFF) - 127 - 14 : 0;
        e = e < -126 ? -126 : e;  // 2^-e stays finite
        const float down = exp2i(-e);
        if (u == 0) q_exp[h] = exp2i(e);
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const float x0 = __fmul_rn(v[2 * j], down), x1 = __fmul_rn(v[2 * j + 1], down);
            const uint32_t hi = pack_f16(x0, x1);
            const __half2 hh = *reinterpret_cast<const __half2 *>(&hi);
            const uint32_t lo = pack_f16(__fsub_rn(x0, __low2float(hh)), __fsub_rn(x1, __high2float(hh)));
            reinterpret_cast<uint32_t *>(qs)[(h * D + u * 32) / 2 + j] = hi;
            reinterpret_cast<uint32_t *>(qs)[((HT + h) * D + u * 32) / 2 + j] = lo;
        }
    }
    __syncthreads();
    uint32_t qf[2 * WPT][4];  // A operand: rows g (hi) and g + 8 (lo)
#pragma unroll
    for (int s = 0; s < 2 * WPT; s++) {
        const int w = s >> 1;
        const int e = (D == 256 ? ((w >> 2) * 4 + c) * 32 + (w & 3) * 8 : c * (D / 4) + w * 8) + (s & 1) * 4;
        const uint2 hi = *reinterpret_cast<const uint2 *>(qs + g * D + e);
        const uint2 lo = *reinterpret_cast<const uint2 *>(qs + (HT + g) * D + e);
        qf[s][0] = hi.x;
        qf[s][1] = lo.x;
        qf[s][2] = hi.y;
        qf[s][3] = lo.y;
    }
    float xscale = __fmul_rn(a.scale, q_exp[g]);
    if (NV) xscale = __fmul_rn(xscale, *a.c.gk);
    if (!NV) xscale = __fmul_rn(xscale, 0.00390625f);  // e8m0_rel's 2^8

    float m_run = -INFINITY, l_run = 0.0f;
    uint32_t v_ref = 0;  // E8M0: the largest V scale byte so far
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; i++) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;

    int stage = 0;
    for (int64_t t0 = first; t0 < ce; t0 += NW * S::TS) {
        cp_async_wait<S::ST - 2>();
        __syncwarp();
        {
            const int64_t tn = t0 + (int64_t)(S::ST - 1) * NW * S::TS;
            const int sn = stage == 0 ? S::ST - 1 : stage - 1;  // the stage consumed last
            if (tn < ce) fetch(tn, sn);
            cp_async_commit();
        }
        const uint32_t kq = ring + (uint32_t)(stage * S::STAGE), vq = kq + S::TS * S::QB, ks = vq + S::TS * S::QB,
                       vs = ks + S::TS * S::SB;

        // tokens of this step that take part
        uint32_t live = 0xFFFFFFFFu;
        if (t0 + S::TS > ce) live &= (1u << (int)(ce - t0)) - 1u;
        if (t0 < r.begin) live &= 0xFFFFFFFFu << min((int)(r.begin - t0), 31);
        if (t0 + 31 < r.begin) live = 0;
        if ((holes >> (2 * stage)) & 1u) live &= 0xFFFF0000u;
        if ((holes >> (2 * stage)) & 2u) live &= 0x0000FFFFu;
        if (S::TS < 32) live |= 0xFFFFFFFFu << (S::TS % 32);
        const bool all = live == 0xFFFFFFFFu;

        // ---- scores ----
        float x[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const int tk = n * 8 + tau(g);
            uint32_t w[WPT], sc[(WPT + 1) / 2], ref = 0;
#pragma unroll
            for (int p = 0; p < (D == 256 ? 2 : 1); p++)
                lds(kq + k_piece<D>(tk, D == 64 ? c >> 1 : p * 4 + c) + (D == 64 ? (c & 1) * 8 : 0), w + 4 * p, D == 64 ? 2 : 4);
            if (FMT == FP4_MXFP4) {  // one scale per 4 words (dim 64: shared by two lanes)
                uint32_t e[D == 256 ? 2 : 1];
#pragma unroll
                for (int p = 0; p < (D == 256 ? 2 : 1); p++) e[p] = lds8(ks + tk * S::SB + (D == 64 ? c >> 1 : p * 4 + c));
                ref = D == 256 ? max(e[0], e[D / 256]) : e[0];
                ref = max(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, 1));
                ref = max(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, 2));
#pragma unroll
                for (int i = 0; i < WPT / 2; i++) sc[i] = e8m0_rel(e[i >> 1], ref);
            } else if (D == 64) {
                const uint32_t e = lds8(ks + tk * S::SB + c);
                if (NV) {
                    sc[0] = e4m3x2_to_f16x2(e * 0x101u);
                } else {
                    ref = e;
                    ref = max(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, 1));
                    ref = max(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, 2));
                    sc[0] = e8m0_rel(e, ref);
                }
            } else {
                uint32_t e[D == 256 ? 2 : 1];
#pragma unroll
                for (int p = 0; p < (D == 256 ? 2 : 1); p++) e[p] = lds16(ks + tk * S::SB + (p * 4 + c) * 2);
                if (NV) {
#pragma unroll
                    for (int p = 0; p < (D == 256 ? 2 : 1); p++) {
                        const uint32_t f = e4m3x2_to_f16x2(e[p]);
                        sc[2 * p] = __byte_perm(f, 0, 0x1010);
                        sc[2 * p + 1] = __byte_perm(f, 0, 0x3232);
                    }
                } else {
                    ref = max(e[0] & 0xFF, e[0] >> 8);
                    if (D == 256) ref = max(ref, max(e[D / 256] & 0xFF, e[D / 256] >> 8));
                    ref = max(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, 1));
                    ref = max(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, 2));
#pragma unroll
                    for (int i = 0; i < WPT / 2; i++) sc[i] = e8m0_rel((e[i >> 1] >> (8 * (i & 1))) & 0xFF, ref);
                }
            }
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < WPT; i++) {
                uint32_t h[4];
                e2m1x8_to_f16(w[i], h);
#pragma unroll
                for (int j = 0; j < 4; j++) h[j] = mul_f16x2(h[j], sc[i >> 1]);
                mma_f16(s, qf[2 * i][0], qf[2 * i][1], qf[2 * i][2], qf[2 * i][3], h[0], h[1]);
                mma_f16(s, qf[2 * i + 1][0], qf[2 * i + 1][1], qf[2 * i + 1][2], qf[2 * i + 1][3], h[2], h[3]);
            }
            // columns 2c and 2c + 1: hi and lo rows together
            x[n][0] = __fmul_rn(__fadd_rn(s[0], s[2]), xscale);
            x[n][1] = __fmul_rn(__fadd_rn(s[1], s[3]), xscale);
            if (!NV) {  // times the rows' reference scales, which the lanes of those tokens hold
                const uint32_t r0 = __shfl_sync(0xFFFFFFFFu, ref, 8 * c), r1 = __shfl_sync(0xFFFFFFFFu, ref, 8 * c + 4);
                x[n][0] = __fmul_rn(x[n][0], exp2i((int)r0 - 127));
                x[n][1] = __fmul_rn(x[n][1], exp2i((int)r1 - 127));
            }
            if (!all) {
                if (!((live >> (n * 8 + tau(2 * c))) & 1u)) x[n][0] = -INFINITY;
                if (!((live >> (n * 8 + tau(2 * c + 1))) & 1u)) x[n][1] = -INFINITY;
            }
        }

        // ---- running maximum ----
        float mx = fmaxf(x[0][0], x[0][1]);
#pragma unroll
        for (int n = 1; n < NT; n++) mx = fmaxf(mx, fmaxf(x[n][0], x[n][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float m_new = fmaxf(m_run, mx);
        uint32_t ref_new = v_ref;
        if (!NV) {  // largest V scale of the step's live tokens
            uint32_t e = 0;
#pragma unroll
            for (int i = 0; i < (S::TS * S::SB + 127) / 128; i++) {
                const int w = i * 32 + lane;
                if (w * 4 < S::TS * S::SB) {
                    uint32_t q;
                    lds(vs + w * 4, &q, 1);
                    if (!all) {
                        if (S::SB == 2) {
                            if (!((live >> (2 * w)) & 1u)) q &= 0xFFFF0000u;
                            if (!((live >> (2 * w + 1)) & 1u)) q &= 0x0000FFFFu;
                        } else if (!((live >> (w * 4 / S::SB)) & 1u)) {
                            q = 0;
                        }
                    }
                    e = max(e, max_byte(q));
                }
            }
            ref_new = max(v_ref, __reduce_max_sync(0xFFFFFFFFu, e));
        }
        if (__any_sync(0xFFFFFFFFu, m_new > m_run) || (!NV && ref_new != v_ref)) {
            const float alpha = m_new > m_run ? ex2(__fsub_rn(m_run, m_new)) : 1.0f;  // 0 from -inf
            l_run = __fmul_rn(l_run, alpha);
            const float f = NV ? 1.0f : exp2i(max((int)v_ref - (int)ref_new, -127));
            const float a0 = __fmul_rn(__shfl_sync(0xFFFFFFFFu, alpha, 8 * c), f);
            const float a1 = __fmul_rn(__shfl_sync(0xFFFFFFFFu, alpha, 8 * c + 4), f);
#pragma unroll
            for (int i = 0; i < MT; i++) {
                acc[i][0] = __fmul_rn(acc[i][0], a0);
                acc[i][1] = __fmul_rn(acc[i][1], a1);
                acc[i][2] = __fmul_rn(acc[i][2], a0);
                acc[i][3] = __fmul_rn(acc[i][3], a1);
            }
            m_run = m_new;
            v_ref = ref_new;
        }
        const float off = __fsub_rn(m_run == -INFINITY ? 0.0f : m_run, kPShift);
        uint32_t ph[NT], pl[NT];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const float p0 = ex2(__fsub_rn(x[n][0], off)), p1 = ex2(__fsub_rn(x[n][1], off));
            l_run = __fadd_rn(l_run, __fadd_rn(p0, p1));
            ph[n] = pack_f16(p0, p1);
            if (!BF16OUT) {
                const __half2 hh = *reinterpret_cast<const __half2 *>(&ph[n]);
                pl[n] = pack_f16(__fsub_rn(p0, __low2float(hh)), __fsub_rn(p1, __high2float(hh)));
            }
        }

        // ---- values ----
#pragma unroll
        for (int j = 0; j < NT / 2; j++) {
            int tk[4] = {16 * j + tau(2 * c), 16 * j + tau(2 * c + 1), 16 * j + 8 + tau(2 * c), 16 * j + 8 + tau(2 * c + 1)};
            uint32_t w[4][VW], s01[(VW + 1) / 2], s23[(VW + 1) / 2];
            uint32_t e[4][(VW + 1) / 2];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                lds(vq + v_piece<D>(tk[i], D == 64 ? g >> 2 : D == 128 ? g >> 1 : g) + (D == 64 ? (g & 3) * 4 : D == 128 ? (g & 1) * 8 : 0), w[i], VW);
                const bool on = all || ((live >> tk[i]) & 1u);
                if (FMT == FP4_MXFP4) {
                    e[i][0] = lds8(vs + tk[i] * S::SB + (D == 64 ? g >> 2 : D == 128 ? g >> 1 : g));
                } else if (D == 256) {
                    e[i][0] = lds16(vs + tk[i] * S::SB + 2 * g);
                } else {
                    e[i][0] = lds8(vs + tk[i] * S::SB + (D == 64 ? g >> 1 : g));
                }
                if (!on) e[i][0] = 0;
                if (FMT != FP4_MXFP4 && D == 256) {
                    e[i][VW / 4] = e[i][0] >> 8;
                    e[i][0] &= 0xFF;
                } else if (D == 256) {
                    e[i][VW / 4] = e[i][0];
                }
            }
#pragma unroll
            for (int k = 0; k < (VW + 1) / 2; k++) {
                if (NV) {
                    s01[k] = e4m3x2_to_f16x2(e[0][k] | (e[1][k] << 8));
                    s23[k] = e4m3x2_to_f16x2(e[2][k] | (e[3][k] << 8));
                } else {
                    // a dead token's byte 0 could still meet a reference of 0..22
                    s01[k] = e8m0_rel2(e[0][k], e[1][k], v_ref);
                    s23[k] = e8m0_rel2(e[2][k], e[3][k], v_ref);
                }
            }
#pragma unroll
            for (int i = 0; i < VW; i++) {
                const uint32_t M = 0x0F0F0F0Fu;
                uint32_t a0[4], a1[4], a2[4], a3[4];
                e2m1x8_to_f16((w[0][i] & M) | ((w[1][i] << 4) & ~M), a0);
                e2m1x8_to_f16(((w[0][i] >> 4) & M) | (w[1][i] & ~M), a1);
                e2m1x8_to_f16((w[2][i] & M) | ((w[3][i] << 4) & ~M), a2);
                e2m1x8_to_f16(((w[2][i] >> 4) & M) | (w[3][i] & ~M), a3);
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
        stage = stage == S::ST - 1 ? 0 : stage + 1;
    }

    // ---- join the warps ----
    l_run = __fadd_rn(l_run, __shfl_xor_sync(0xFFFFFFFFu, l_run, 1));
    l_run = __fadd_rn(l_run, __shfl_xor_sync(0xFFFFFFFFu, l_run, 2));
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with the ring
    float *so = reinterpret_cast<float *>(smem) + warp * HT * D;
    if (c == 0) {
        sm_m[warp][g] = m_run;
        sm_l[warp][g] = l_run;
    }
    const float vf = NV ? 1.0f : __fmul_rn(exp2i((int)v_ref - 127), 0.00390625f);
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int d = g * (D / 8) + 2 * i;
        so[(2 * c) * D + d] = __fmul_rn(acc[i][0], vf);
        so[(2 * c + 1) * D + d] = __fmul_rn(acc[i][1], vf);
        so[(2 * c) * D + d + 1] = __fmul_rn(acc[i][2], vf);
        so[(2 * c + 1) * D + d + 1] = __fmul_rn(acc[i][3], vf);
    }
    __syncthreads();
    const float gv = NV ? *a.c.gv : 1.0f;
    float *o = reinterpret_cast<float *>(smem);
    for (int i = threadIdx.x; i < nh * D; i += NW * 32) {
        const int h = i / D;
        float m = sm_m[0][h];
#pragma unroll
        for (int w = 1; w < NW; w++) m = fmaxf(m, sm_m[w][h]);
        float s = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float f = sm_m[w][h] == -INFINITY ? 0.0f : ex2(__fsub_rn(sm_m[w][h], m));
            s = __fmaf_rn(f, o[w * HT * D + i], s);
            l = __fmaf_rn(f, sm_l[w][h], l);
        }
        const int64_t row = (int64_t)b * a.q_heads + h0 + h;
        if (a.chunks > 1) {
            const int64_t p = row * a.chunks + chunk;
            a.part_o[p * D + i % D] = s;
            if (i % D == 0) a.part_ml[p] = make_float2(m, l);
        } else {
            o[i] = l == 0.0f ? 0.0f : __fmul_rn(__fdiv_rn(s, l), gv);  // this thread's own element of warp 0's part
            if (a.lse && i % D == 0)
                a.lse[row] = l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fsub_rn(m, kPShift), log2f(l)), 0.693147180559945f);
        }
    }
    if (a.chunks > 1) return;
    __syncthreads();
    write_rows<D, BF16OUT>(o, nh, (int64_t)b * a.q_heads + h0, a, NW * 32);
}

// Joins a row's chunks: o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c.
template <int FMT, int D, int BF16OUT>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args a)
{
    constexpr int LANES = D / 4, GROUPS = 128 / LANES;
    __shared__ float f[kMaxChunks];
    __shared__ float red[8];
    __shared__ __align__(16) float o[GROUPS][D];
    grid_dep_launch();
    grid_dep_wait();
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)b * a.q_heads + blockIdx.x;
    const Range r = live_range(a, b);
    const int n = r.end > r.base ? (int)((r.end - r.base + a.chunk - 1) / a.chunk) : 0;
    const float2 *ml = a.part_ml + row * a.chunks;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += 128) {
        f[i] = ml[i].x;
        m = fmaxf(m, f[i]);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float l = 0.0f;
    for (int i = threadIdx.x; i < n; i += 128) {
        f[i] = f[i] == -INFINITY ? 0.0f : ex2(__fsub_rn(f[i], m));
        l = __fmaf_rn(f[i], ml[i].y, l);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xFFFFFFFFu, l, s));
    if (lane == 0) red[4 + warp] = l;
    __syncthreads();
    l = __fadd_rn(__fadd_rn(red[4], red[5]), __fadd_rn(red[6], red[7]));
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
    const float gv = FMT == FP4_NVFP4 ? *a.c.gv : 1.0f;
    for (int d = threadIdx.x; d < D; d += 128) {
        float t = o[0][d];
#pragma unroll
        for (int k = 1; k < GROUPS; k++) t = __fadd_rn(t, o[k][d]);
        o[0][d] = l == 0.0f ? 0.0f : __fmul_rn(__fdiv_rn(t, l), gv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row] = l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fsub_rn(m, kPShift), log2f(l)), 0.693147180559945f);
    __syncthreads();
    write_rows<D, BF16OUT>(o[0], 1, row, a, 128);
}

// ---------------------------------------------------------------------------
// How a call is cut: tokens per chunk (a multiple of 32) and chunks per
// sequence, from its sizes alone (lengths live on the device).
struct Plan {
    int64_t chunk;
    int chunks;
};

static Plan plan(int64_t batch, int kv_heads, int head_tiles, int64_t tokens, int sms)
{
    const int64_t rows = batch * kv_heads * head_tiles;
    int64_t want = ((int64_t)sms * 4 + rows - 1) / rows;  // CTAs for every resident slot
    if (want < 1) want = 1;
    int64_t chunk = (tokens + want - 1) / want;
    if (chunk < 512) chunk = 512;
    if (chunk > 2048) chunk = 2048;
    int64_t chunks = (tokens + chunk - 1) / chunk;
    if (chunks > kMaxChunks) {
        chunk = (tokens + kMaxChunks - 1) / kMaxChunks;
    }
    chunk = (chunk + 31) / 32 * 32;
    chunks = (tokens + chunk - 1) / chunk;
    Plan p = {chunk, (int)(chunks < 1 ? 1 : chunks)};
    return p;
}

// Tokens that a sequence's chunks have to cover: its live range from the last
// multiple of 32 before it.
static int64_t span(int64_t max_len, int64_t window)
{
    return window > 0 && max_len > window ? window + 31 : max_len;
}

template <int FMT, int D, int BF16OUT>
static cudaError_t launch_t(const Args &a, int64_t batch, int kv_heads, cudaStream_t st)
{
    using S = Shape<FMT, D>;
    auto kern = paged_kernel<FMT, D, BF16OUT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_k(kern, dim3((unsigned)(a.chunks * a.head_tiles), (unsigned)kv_heads, (unsigned)batch), dim3(NW * 32), S::SMEM, st, true, a);
    if (e != cudaSuccess || a.chunks == 1) return e;
    return launch_k(join_kernel<FMT, D, BF16OUT>, dim3((unsigned)a.q_heads, (unsigned)batch), dim3(128), 0, st, true, a);
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
    const attn::Plan p = attn::plan(batch > 0 ? batch : 1, kv_heads, tiles, attn::span(max_len, window), sms);
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
    a.table_tokens = table_cols << c.page_shift;
    a.lens = lens;
    a.max_len = max_len;
    a.window = window;
    a.group = q_heads / c.heads;
    a.head_tiles = (a.group + attn::HT - 1) / attn::HT;
    a.q_heads = q_heads;
    a.scale = (float)((double)scale * 1.4426950408889634);
    a.ck = ck;
    a.hk = hk;
    const attn::Plan p = attn::plan(batch, c.heads, a.head_tiles, attn::span(max_len, window), sms);
    a.chunk = p.chunk;
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
