// w4a16.cu — the weight-only linear layer of a decode step
// (fp4_linear_w4a16): C = (H x) W^T for M <= 16 rows of bf16 activations that
// stay in 16 bits, W in FP4 with block scales as fp4_quantize wrote it.
//
// What bounds it: W is read once, N * K * (1/2 + 1/block) bytes; x and C are
// small.  Every element of W becomes an f16 operand in registers (one
// conversion and one multiply by its scale per pair), which at the measured
// HBM rate takes about half of the issue slots; the products run on mma.sync
// m16n8k16, W the 16-row operand, the activations the 8 columns.  tcgen05
// would need the converted tile in shared memory, four times the packed bytes.
//
// Operand order.  The inner index of a product may be permuted, so a lane
// holds 16 whole bytes (32 elements) of a W row: the 4 lanes of a row cover
// 128 elements, and a warp's 16-byte loads are 64-byte pieces of 8 rows.
// A lane's four rows are r, r + 32, r + 64, r + 96 of a 128-row scale tile:
// their scale words are 16 consecutive bytes, one load.
//
// Exactness.  q * s_b is exact in f16 for NVFP4.  For E8M0 scales it is taken
// relative to the row's largest scale among 128 elements, and each 128-element
// sum is added times that power of two in fp32 (blocks more than 2^22 below
// it count as zero).  x in f16 is a power of two (per row and K slice, the
// largest value in [2^14, 2^15)) times its bf16 value: exact down to 2^-28 of
// the largest.  After a rotation x has 24 bits: rounded to f16's 11 for bf16
// output (2^-11 per value, below the output's own 2^-8), split into hi + lo
// columns for fp32 output.
//
// Work split, two forms.  By tiles: a CTA is 8 warps, WR of them side by side
// along N (32 rows each), 8 / WR along K, each with its own ring of asynchronous
// copies; a cluster of up to 8 CTAs splits K further and joins its sums over
// distributed shared memory.  One launch, no workspace; x is turned to f16 by
// every CTA for its part of K.  Streamed, for more columns or larger weights:
// below.  Sums have a fixed order in both: results repeat bit for bit.
//
// Measured (NVFP4, a graph of calls; % of the time of W's bytes at the measured
// copy rate): 28672 x 8192, 1 row to fp32 30.8 us (66 %; its loads alone 25.2),
// 8 rows 33.5, 16 rows 44.1 (both streamed); 14336 x 4096, 1 row 11.6 (44 %),
// 16 rows 19.8; 4096 x 14336, 16 rows rotated by H_128 20.0, by tiles 22.2 (27.6
// while a cluster's CTAs stored every 8th value instead of 256 in a row).
#include <math.h>

#include <algorithm>

#include "frag.cuh"
#include "sm100.cuh"

namespace fp4 {
namespace w4 {

constexpr int kThreads = 256;
constexpr int kStep = 2560;                     // bytes of a warp's step: 32 rows x 64, and the scale words
// Steps of a warp's ring: with more than 8 columns one less, for x.
__host__ __device__ constexpr int stages_of(int nt) { return nt == 1 ? 4 : 3; }
__host__ __device__ constexpr int ring_of(int nt) { return 8 * stages_of(nt) * kStep; }
constexpr int kMaxSmem = 224 * 1024;            // what a launch may ask for
// CTAs per SM: with 32 columns one, whose sums then stay in registers (4096 x
// 4096, 16 rotated rows to fp32: 12.4 us, with two 20.2).
__host__ __device__ constexpr int resident(int nt) { return nt > 2 ? 1 : 2; }
constexpr int x_bytes(int cols) { return kMaxSmem / resident((cols + 7) / 8) - ring_of((cols + 7) / 8); }  // a stage of x

struct Args {
    const uint16_t *x;
    int64_t ldx;
    int M, hk, cols;      // cols: operand columns (M, or 2 M with the lo parts)
    float ck;
    const uint8_t *wq, *ws;
    const float *gw;
    int64_t N, K;
    int64_t nkb4;         // scale tiles along K
    void *out;
    int64_t ldc;
    int chunks;           // 128-element steps of K
    int slice;            // steps per CTA of a cluster
    int stage;            // steps of x held in shared memory at a time
    int cluster;          // CTAs that share a tile
    int w_early;          // W may be read before the grid-dependency wait
};

// E8M0: a step's sums are added times the row's largest scale and kDown; 2^kRest
// is what is left (e8m0_rel's 2^8 is in the sums).  A step's sum stays below
// 2^33, so scales up to 2^110 keep the fp32 sums finite; down to 2^-127 the
// factor is exact.
constexpr float kDown = 1.0f / (1 << 18);
constexpr int kRest = 18 - 8;

// What a row's sums are multiplied by: its power of two 2^e and that of the
// tensor scale as one pair of factors, the scale's significand (left in gw)
// last.  So no product on the way is larger than the result (2^e alone can be
// 2^113).
template <bool NV>
FP4_DEV float2 row_factors(int e, float &gw)
{
    return exp2_pair(e + (NV ? take_exponent(gw) : kRest));
}

// A lane's part of a step of W: 32 elements and a scale word of 4 rows.
struct Piece {
    uint32_t w[4][4], s[4];
};

FP4_DEV void take(uint32_t at, Piece &p)
{
#pragma unroll
    for (int j = 0; j < 4; j++) lds(at + j * 512, p.w[j], 4);
    lds(at + 2048, p.s, 4);
}

// One warp's step: 32 rows of W (a lane's part p) times 128 elements of the
// columns of x at `xb` (this lane's pieces, `pitch` bytes a column).
// Columns from `cols` on count as zeros (8 * NT: all are there).
template <int FMT, int NT, int BF16OUT>
FP4_DEV void multiply_step(const Piece &p, uint32_t xb, uint32_t pitch, int cols, int g, int c, float (&acc)[2][NT][4])
{
    constexpr bool NV = FMT == FP4_NVFP4;
    // The step's own sums, added with a rounding to nearest, which the product's
    // accumulation of many steps would not give.  Not needed for NVFP4 with
    // bf16 output: what it loses (1e-6 at K = 8192) is far below 2^-8.
    constexpr bool PART = !NV || !BF16OUT;
    uint32_t sc[4][2], ref[2];  // ref: the largest scale bytes, of two rows each
    if (!NV) {
#pragma unroll
        for (int t = 0; t < 2; t++) {
            ref[t] = max_bytes2(p.s[2 * t], p.s[2 * t + 1]);
            if (FMT != FP4_MXFP4) ref[t] = __vmaxu2(ref[t], __shfl_xor_sync(0xFFFFFFFFu, ref[t], 2));  // the step's other scale word
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t top = NV ? 0 : j & 1 ? ref[j / 2] >> 16 : ref[j / 2] & 0xFFFF;
        if (FMT == FP4_MXFP4) {
            sc[j][0] = sc[j][1] = e8m0_rel((p.s[j] >> (8 * c)) & 0xFF, top);
        } else {
            const uint32_t two = (p.s[j] >> (16 * (c & 1))) & 0xFFFF;
            if (NV) {
                const uint32_t f = e4m3x2_to_f16x2(two);
                sc[j][0] = __byte_perm(f, 0, 0x1010);
                sc[j][1] = __byte_perm(f, 0, 0x3232);
            } else {
                sc[j][0] = e8m0_rel(two & 0xFF, top);
                sc[j][1] = e8m0_rel(two >> 8, top);
            }
        }
    }
    float part[2][NT][4];
    if (PART) {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int n = 0; n < NT; n++) part[t][n][0] = part[t][n][1] = part[t][n][2] = part[t][n][3] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t h[4][4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            e2m1x8_to_f16(p.w[j][i], h[j]);
#pragma unroll
            for (int e = 0; e < 4; e++) h[j][e] = mul_f16x2(h[j][e], sc[j][i >> 1]);
        }
#pragma unroll
        for (int n = 0; n < NT; n++) {
            uint32_t bx[4] = {0, 0, 0, 0};
            if (8 * n + g < cols)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(bx[0]), "=r"(bx[1]), "=r"(bx[2]), "=r"(bx[3]) : "r"(xb + (8 * n + g) * pitch + i * 64));
#pragma unroll
            for (int t = 0; t < 2; t++) {
                float *d = PART ? part[t][n] : acc[t][n];
                mma_f16(d, h[2 * t][0], h[2 * t + 1][0], h[2 * t][1], h[2 * t + 1][1], bx[0], bx[1]);
                mma_f16(d, h[2 * t][2], h[2 * t + 1][2], h[2 * t][3], h[2 * t + 1][3], bx[2], bx[3]);
            }
        }
    }
    if (PART) {
#pragma unroll
        for (int t = 0; t < 2; t++) {
            // (a NaN among the scales is the largest byte: the row's sum becomes NaN)
            const float2 f = NV ? make_float2(1.0f, 1.0f) : e8m0x2_to_f32(ref[t]);
            const float f0 = NV ? 1.0f : __fmul_rn(f.x, kDown), f1 = NV ? 1.0f : __fmul_rn(f.y, kDown);
#pragma unroll
            for (int n = 0; n < NT; n++) {
                acc[t][n][0] = __fmaf_rn(part[t][n][0], f0, acc[t][n][0]);
                acc[t][n][1] = __fmaf_rn(part[t][n][1], f0, acc[t][n][1]);
                acc[t][n][2] = __fmaf_rn(part[t][n][2], f1, acc[t][n][2]);
                acc[t][n][3] = __fmaf_rn(part[t][n][3], f1, acc[t][n][3]);
            }
        }
    }
}

template <int FMT, int WR, int NT, int BF16OUT>
__global__ void __launch_bounds__(kThreads, resident(NT)) w4a16_kernel(const __grid_constant__ Args a)
{
    constexpr int WK = 8 / WR, ROWS = 32 * WR, kStages = stages_of(NT), kRing = ring_of(NT);
    constexpr bool NV = FMT == FP4_NVFP4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float x_up[16];
    __shared__ uint32_t x_top[16];
    __shared__ float2 x_out[16];  // factors of the sums
    __shared__ float w_out;
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int wr = warp % WR, wk = warp / WR;
    const uint32_t rank = cluster_ctarank();
    const int tile = blockIdx.x / a.cluster;           // ROWS rows of W
    const int64_t atom = tile / (4 / WR);              // its 128-row scale tile
    const int r0 = (tile % (4 / WR)) * (8 * WR) + wr * 8 + g;  // row in the tile: r0 + 32 j
    const int s0 = (int)rank * a.slice, s1 = min(s0 + a.slice, a.chunks);  // K steps

    // Nothing is predicated per row or lane: rows past N read row N - 1 (their
    // results are not stored), elements past K the row's first (x is 0 there).
    const uint32_t row_bytes = (uint32_t)(a.K / 2);
    const uint8_t *wp[4];
#pragma unroll
    for (int j = 0; j < 4; j++) wp[j] = a.wq + min(atom * 128 + r0 + 32 * j, a.N - 1) * row_bytes;
    const uint8_t *sp = a.ws + (atom * a.nkb4 * 512 + r0 * 16);
    // A lane's pieces of a step (4 rows' elements, their scale words) go through
    // its own slots of a ring of asynchronous copies: no other lane waits.
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages * kStep) + lane * 16;
    auto load = [&](int step, int i) {
        if (step < s1) {
            uint32_t k = (uint32_t)step * 64 + c * 16;
            k = k < row_bytes ? k : 0;
            const uint32_t t = FMT == FP4_MXFP4 ? (uint32_t)step : min(2 * (uint32_t)step + (c >> 1), (uint32_t)a.nkb4 - 1);
#pragma unroll
            for (int j = 0; j < 4; j++) cp_async16(ring + i * kStep + j * 512, wp[j] + k, true);
            cp_async16(ring + i * kStep + 2048, sp + (uint64_t)t * 512, true);
        }
        cp_async_commit();
    };
    if (threadIdx.x < 16) x_top[threadIdx.x] = 0;
    if (!a.w_early) grid_dep_wait();
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) load(s0 + wk + i * WK, i);
    if (a.w_early) grid_dep_wait();
    __syncthreads();

    // ---- the slice's largest |x| per row (after H_k where each thread holds
    // its one unit of x; else before it, |H x| <= sqrt(k) max |x|) ----
    const int units = (s1 - s0) * 4;  // 32-element units per row
    const bool kept = a.M * units <= kThreads && s1 - s0 <= a.stage;
    // plain loads: what earlier launches wrote is no constant data (no wait orders that)
    auto fetch_x = [&](int m, int64_t k, float *v) {
        uint4 raw[4] = {};
        if (m < a.M && k < a.K) {
            const uint4 *p = reinterpret_cast<const uint4 *>(a.x + m * a.ldx + k);
#pragma unroll
            for (int e = 0; e < 4; e++) raw[e] = p[e];
        }
        unpack_unit(raw, v);
    };
    // one unit (u of the stage) of row m to f16, in the order the lanes read it
    const uint32_t xs = smem_u32(smem) + kRing;
    const uint32_t pitch = (uint32_t)a.stage * 256 + 64;  // bytes per column: two columns' pieces fill all banks
    auto put_x = [&](int m, int u, const float *v) {
        const float up = x_up[m];
        const float down = __uint_as_float((254u << 23) - __float_as_uint(up));  // its reciprocal
        const uint32_t at = xs + m * pitch + (u >> 2) * 256 + (u & 3) * 16;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float x0 = __fmul_rn(v[8 * q + 2 * e], down), x1 = __fmul_rn(v[8 * q + 2 * e + 1], down);
                hi[e] = pack_f16(x0, x1);
                const __half2 hh = *reinterpret_cast<const __half2 *>(&hi[e]);
                if (!BF16OUT) lo[e] = pack_f16(__fsub_rn(x0, __low2float(hh)), __fsub_rn(x1, __high2float(hh)));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + q * 64), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
            if (!BF16OUT && a.cols > a.M)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + a.M * pitch + q * 64), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
        }
    };
    float gw = NV && threadIdx.x < a.M ? *a.gw : 1.0f;
    float v[32];
    const int mine_m = threadIdx.x / units, mine_u = threadIdx.x - mine_m * units;
    if (kept) {
        fetch_x(mine_m, (int64_t)s0 * 128 + mine_u * 32, v);
        rotate_unit(v, a.hk, a.ck, lane);  // units of a row's step are 4 neighbouring lanes
        if (mine_m < a.M) atomicMax(&x_top[mine_m], __float_as_uint(absmax_tree<32>(v)));
    } else {
        const int64_t k0 = (int64_t)s0 * 128, k1 = min((int64_t)s1 * 128, a.K);
        const int pieces = (int)((k1 - k0) / 8), wpr = a.M < 8 ? 8 / a.M : 1;  // warps per row
        for (int m = warp / wpr; m < a.M; m += 8) {
            const uint4 *p = reinterpret_cast<const uint4 *>(a.x + m * a.ldx + k0);
            uint32_t top = 0;
#pragma unroll 4
            for (int i = (warp % wpr) * 32 + lane; i < pieces; i += 32 * wpr) {
                const uint4 t = p[i];
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int j = 0; j < 4; j++) top = max(top, max((w[j] << 16) & 0x7FFF0000u, w[j] & 0x7FFF0000u));
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (lane == 0) atomicMax(&x_top[m], top);
        }
    }
    __syncthreads();
    if (threadIdx.x < a.M) {
        const uint32_t top = x_top[threadIdx.x];
        int e = top ? (int)(top >> 23) - 127 - (a.hk && !kept ? 10 : 14) : 0;  // below 2^15 in f16
        e = e < -126 ? -126 : e;
        x_up[threadIdx.x] = exp2i(e);
        x_out[threadIdx.x] = row_factors<NV>(e, gw);
        if (NV) w_out = gw;  // all of them the same
    }

    float acc[2][NT][4];
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int n = 0; n < NT; n++) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.0f;

    int slot = 0;
    for (int st = s0; st < s1; st += a.stage) {
        const int se = min(st + a.stage, s1);
        __syncthreads();  // scales are set; the last stage is consumed
        if (kept) {
            if (mine_m < a.M) put_x(mine_m, mine_u, v);
        } else {
            const int n = (se - st) * 4;
            for (int i = threadIdx.x; i < (a.M * n + 31) / 32 * 32; i += kThreads) {
                const int m = i / n, u = i - m * n;
                fetch_x(m, (int64_t)st * 128 + u * 32, v);
                rotate_unit(v, a.hk, a.ck, lane);
                if (m < a.M) put_x(m, u, v);
            }
        }
        __syncthreads();

        // steps s0 + wk, s0 + wk + WK, ... (a stage of x is a multiple of WK steps)
        for (int step = st + wk; step < se; step += WK) {
            cp_async_wait<kStages - 2>();
            Piece now;
            take(ring + slot * kStep, now);
            load(step + (kStages - 1) * WK, slot == 0 ? kStages - 1 : slot - 1);  // the slot taken last
            slot = slot == kStages - 1 ? 0 : slot + 1;
            multiply_step<FMT, NT, BF16OUT>(now, xs + (step - st) * 256 + c * 16, pitch, a.cols, g, c, acc);
        }
    }

    // ---- sums: warps along K, hi and lo columns, then the cluster ----
    cp_async_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);            // [WK][cols][ROWS]
    float *sum = red + WK * a.cols * ROWS;                   // [M][ROWS]
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int col = 8 * n + 2 * c + (e & 1);
                const int row = (2 * t + (e >> 1)) * (8 * WR) + wr * 8 + g;  // rows of one j side by side
                if (col < a.cols) red[(wk * a.cols + col) * ROWS + row] = acc[t][n][e];
            }
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * ROWS; i += kThreads) {
        const int m = i / ROWS;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < WK; k++) {
            s = __fadd_rn(s, red[k * a.cols * ROWS + i]);
            if (a.cols > a.M) s = __fadd_rn(s, red[k * a.cols * ROWS + a.M * ROWS + i]);
        }
        sum[i] = __fmul_rn(__fmul_rn(s, x_out[m].x), x_out[m].y);
    }
    const uint32_t cl = (uint32_t)a.cluster;
    if (cl > 1) cluster_sync();
    else __syncthreads();
    for (int i = rank * kThreads + threadIdx.x; i < a.M * ROWS; i += kThreads * cl) {
        const int m = i / ROWS, row = i % ROWS;
        const int64_t n = atom * 128 + (row / (8 * WR)) * 32 + (tile % (4 / WR)) * (8 * WR) + row % (8 * WR);
        float t = 0.0f;
        for (uint32_t r = 0; r < cl; r++) t = __fadd_rn(t, ld_shared_cluster_f32(mapa_shared(smem_u32(sum + i), r)));
        if (NV) t = __fmul_rn(t, w_out);
        if (n < a.N) {
            if (BF16OUT)
                static_cast<__nv_bfloat16 *>(a.out)[m * a.ldc + n] = __float2bfloat16_rn(t);
            else
                static_cast<float *>(a.out)[m * a.ldc + n] = t;
        }
    }
    if (cl > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// ---- the streamed form -------------------------------------------------------
// x is turned to f16 once (prepare_kernel, into the workspace, in the order the
// lanes read it) instead of by every CTA, while the first steps of W are loaded
// already; the steps of all tiles form one sequence that is cut evenly over
// exactly the CTAs that fit on the GPU.  A tile cut between CTAs is summed by the
// last of them to finish, in CTA order, 16 bytes a lane and 8 parts in flight
// (28672 x 8192, 16 rows: 44.1 us; value by value it was 50).

struct Stream {
    uint8_t *xh;         // [cols][pairs * 2 steps][256 bytes]
    float2 *x_out;       // [17]: factors of the rows' sums, then (the tensor scale's significand, -)
    unsigned *counters;  // [tiles]
    float *part;         // [2 * grid][M][128]
    int pairs;           // pairs of steps per tile
    int share, more;     // a CTA's pairs of the sequence: share, one more for the first `more` CTAs
    FastDiv share1_div, share_div, pairs_div;  // by share + 1, share, pairs
};

FP4_DEV uint32_t stream_begin(uint32_t cta, const Stream &s) { return cta * (uint32_t)s.share + min(cta, (uint32_t)s.more); }

// The CTA whose part holds pair q of the sequence.
FP4_DEV uint32_t stream_owner(uint32_t q, const Stream &s)
{
    const uint32_t split = (uint32_t)s.more * ((uint32_t)s.share + 1u);
    return q < split ? fastdiv(q, s.share1_div) : (uint32_t)s.more + fastdiv(q - split, s.share_div);
}

// Row blockIdx.x of x: H_k, the power of two, f16 hi (and lo); also zeroes the counters.
template <int FMT, int BF16OUT>
__global__ void __launch_bounds__(512) prepare_kernel(const __grid_constant__ Args a, const __grid_constant__ Stream s, int tiles)
{
    __shared__ uint32_t top_w[16];
    // In this order: stream_kernel starts when everything before this launch
    // has ended, and reads W while x is prepared.
    grid_dep_wait();
    grid_dep_launch();
    const int m = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = m * 512 + threadIdx.x; i < tiles; i += a.M * 512) s.counters[i] = 0;
    float gw = FMT == FP4_NVFP4 ? *a.gw : 1.0f;
    const int units = s.pairs * 8, real = (int)(a.K / 32);
    float v[32];
    auto fetch = [&](int u) {
        uint4 raw[4] = {};
        if (u < real) {
            const uint4 *p = reinterpret_cast<const uint4 *>(a.x + m * a.ldx + (int64_t)u * 32);
#pragma unroll
            for (int e = 0; e < 4; e++) raw[e] = p[e];
        }
        unpack_unit(raw, v);
        rotate_unit(v, a.hk, a.ck, lane);
    };
    uint32_t top = 0;
    for (int u = threadIdx.x; u < (units + 31) / 32 * 32; u += 512) {
        fetch(u);
        top = max(top, __float_as_uint(absmax_tree<32>(v)));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) top_w[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, lane < 16 ? top_w[lane] : 0u);
    int e = top ? (int)(top >> 23) - 127 - 14 : 0;  // the largest in [2^14, 2^15)
    e = e < -126 ? -126 : e;
    const float down = exp2i(-e);
    if (threadIdx.x == 0) {
        s.x_out[m] = row_factors<FMT == FP4_NVFP4>(e, gw);
        if (m == 0) s.x_out[16].x = gw;
    }
    for (int u = threadIdx.x; u < (units + 31) / 32 * 32; u += 512) {
        if (units > 512) fetch(u);  // else v still holds the thread's one unit
        if (u >= units) continue;
        uint8_t *hi_at = s.xh + ((int64_t)m * s.pairs * 2 + (u >> 2)) * 256 + (u & 3) * 16;
        uint8_t *lo_at = hi_at + (int64_t)a.M * s.pairs * 512;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float x0 = __fmul_rn(v[8 * q + 2 * j], down), x1 = __fmul_rn(v[8 * q + 2 * j + 1], down);
                hi[j] = pack_f16(x0, x1);
                const __half2 hh = *reinterpret_cast<const __half2 *>(&hi[j]);
                if (!BF16OUT) lo[j] = pack_f16(__fsub_rn(x0, __low2float(hh)), __fsub_rn(x1, __high2float(hh)));
            }
            *reinterpret_cast<uint4 *>(hi_at + q * 64) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (!BF16OUT && a.cols > a.M) *reinterpret_cast<uint4 *>(lo_at + q * 64) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// Shared memory of stream_kernel: every lane's own ring of W, two buffers of XG
// pairs of x for the CTA (so its warps meet once in XG pairs), the join.
template <int NT>
struct StreamShape {
    static constexpr int ST = NT == 1 ? 4 : 3;
    static constexpr int XG = 2;
    static constexpr uint32_t XP = 512 + 64;  // bytes of a column's pair of steps: two columns' pieces fill all banks
    static constexpr uint32_t XSLOT = 8 * NT * XP;
    static constexpr uint32_t SMEM = ST * 8 * kStep + 2 * XG * XSLOT + 8 * NT * 512;
};

template <int FMT, int NT, int BF16OUT>
__global__ void __launch_bounds__(kThreads, resident(NT)) stream_kernel(const __grid_constant__ Args a, const __grid_constant__ Stream s)
{
    using S = StreamShape<NT>;
    constexpr int ST = S::ST, XG = S::XG;
    constexpr bool NV = FMT == FP4_NVFP4;
    constexpr uint32_t XP = S::XP, WSLOT = 8 * kStep, XSLOT = S::XSLOT;
    constexpr int TILES_PER_STEP = FMT == FP4_MXFP4 ? 1 : 2;  // scale tiles along K
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned arrived;
    __shared__ float2 x_out[17];
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int wr = warp & 3, wk = warp >> 2, r0 = wr * 8 + g;
    const uint32_t ring = smem_u32(smem), mine = ring + warp * kStep + lane * 16, xat = ring + ST * WSLOT;
    float *red = reinterpret_cast<float *>(smem + ST * WSLOT + 2 * XG * XSLOT);  // [cols][128]
    const uint32_t begin = stream_begin(blockIdx.x, s), count = stream_begin(blockIdx.x + 1, s) - begin;

    // the stream of loads: this lane's pieces of the next pair's step
    uint32_t lt = fastdiv(begin, s.pairs_div), ln = 0;
    int lp = (int)(begin - lt * (uint32_t)s.pairs);
    const uint8_t *wp[4], *sp;
    auto aim = [&]() {
#pragma unroll
        for (int j = 0; j < 4; j++)
            wp[j] = a.wq + min((int64_t)lt * 128 + r0 + 32 * j, a.N - 1) * (a.K / 2) + (2 * lp + wk) * 64 + c * 16;
        sp = a.ws + ((int64_t)lt * a.nkb4 + (2 * lp + wk) * TILES_PER_STEP + (FMT == FP4_MXFP4 ? 0 : c >> 1)) * 512 + r0 * 16;
    };
    aim();
    auto load_w = [&](uint32_t slot) {
        const int step = 2 * lp + wk;
        // past K: zeros (the second step of a pair, the last step's upper lanes)
        const bool w_in = step * 128 + c * 32 < (int)a.K, s_in = step * TILES_PER_STEP + (FMT == FP4_MXFP4 ? 0 : c >> 1) < (int)a.nkb4;
#pragma unroll
        for (int j = 0; j < 4; j++) cp_async16(mine + slot * WSLOT + j * 512, wp[j], w_in);
        cp_async16(mine + slot * WSLOT + 2048, sp, s_in);
    };
    const uint8_t *xg = s.xh + (int64_t)(threadIdx.x >> 5) * s.pairs * 512 + (threadIdx.x & 31) * 16;
    const uint32_t xd = xat + (threadIdx.x >> 5) * XP + (threadIdx.x & 31) * 16;
    uint32_t xn = 0;  // pairs of x asked for
    int xpair = lp;
    auto load_x = [&]() {  // the next XG pairs
#pragma unroll
        for (int k = 0; k < XG; k++) {
            if (xn >= count) return;
            const uint32_t at = xd + (xn % (2 * XG)) * XSLOT;
#pragma unroll
            for (int i = 0; i < NT; i++)
                if (8 * i + (int)(threadIdx.x >> 5) < a.cols) cp_async16(at + i * 8 * XP, xg + ((int64_t)i * 8 * s.pairs + xpair) * 512, true);
            xn++;
            xpair = xpair + 1 == s.pairs ? 0 : xpair + 1;
        }
    };
    auto advance = [&]() {
        ln++;
        if (++lp == s.pairs) {
            lp = 0;
            lt++;
            if (ln < count) aim();
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) wp[j] += 128;
            sp += 2 * TILES_PER_STEP * 512;
        }
    };
    // columns that x does not have stay zero
    for (int i = threadIdx.x; i < 2 * XG * (8 * NT - a.cols) * 32; i += kThreads) {
        const int slot = i / ((8 * NT - a.cols) * 32), p = i - slot * (8 * NT - a.cols) * 32;
        *reinterpret_cast<uint4 *>(smem + ST * WSLOT + slot * XSLOT + (a.cols + (p >> 5)) * XP + (p & 31) * 16) = make_uint4(0, 0, 0, 0);
    }
    // W at once: prepare_kernel let this launch begin only after its own wait
#pragma unroll
    for (int i = 0; i < ST - 1; i++) {
        if (ln < count) {
            load_w(i);
            advance();
        }
        if (i < ST - 2) cp_async_commit();
    }
    grid_dep_wait();
    float2 factors = {};
    if (threadIdx.x <= a.M) factors = s.x_out[threadIdx.x < a.M ? threadIdx.x : 16];
    load_x();  // in the last group
    cp_async_commit();

    float acc[2][NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int n = 0; n < NT; n++) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.0f;
    };
    clear();
    uint32_t tile = fastdiv(begin, s.pairs_div);
    int pair = (int)(begin - tile * (uint32_t)s.pairs), from = pair;
    uint32_t slot = 0;
    Piece next;
    if (threadIdx.x <= a.M) x_out[threadIdx.x] = factors;  // (read after many barriers)
    cp_async_wait<0>();  // x came last
    take(mine, next);
    for (uint32_t n = 0; n < count; n++) {
        if (n % XG == 0) {
            __syncthreads();  // these pairs' x has arrived; every warp has left the buffer before
            load_x();
            cp_async_commit();
        }
        if (ln < count) {  // a lane's ring is its own
            load_w(slot == 0 ? ST - 1 : slot - 1);
            advance();
        }
        cp_async_commit();
        slot = slot == ST - 1 ? 0 : slot + 1;
        cp_async_wait<ST - 2>();  // the next pair's W, and x when that begins a buffer
        const Piece now = next;
        take(mine + slot * WSLOT, next);
        multiply_step<FMT, NT, BF16OUT>(now, xat + (n % (2 * XG)) * XSLOT + wk * 256 + c * 16, XP, 8 * NT, g, c, acc);
        const bool done = pair == s.pairs - 1;
        if (done || n == count - 1) {
            // ---- this CTA's part of the tile ----
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int i = 0; i < NT; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int col = 8 * i + 2 * c + (e & 1);
                        if (wk && col < a.cols) red[col * 128 + (2 * t + (e >> 1)) * 32 + r0] = acc[t][i][e];
                    }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int i = 0; i < NT; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int col = 8 * i + 2 * c + (e & 1);
                        float *d = red + col * 128 + (2 * t + (e >> 1)) * 32 + r0;
                        if (!wk && col < a.cols) *d = __fadd_rn(acc[t][i][e], *d);
                    }
            __syncthreads();
            const float gw = NV ? x_out[a.M].x : 1.0f;
            const bool whole = from == 0 && done;
            // a CTA has two places for parts: of a tile that its sequence begins in, of a later one
            float *place = s.part + (int64_t)(2 * blockIdx.x + (begin < tile * (uint32_t)s.pairs)) * a.M * 128;
            auto store = [&](int i, float v) {
                const int64_t row = (int64_t)tile * 128 + i % 128;
                if (row >= a.N) return;
                if (BF16OUT)
                    static_cast<__nv_bfloat16 *>(a.out)[(i / 128) * a.ldc + row] = __float2bfloat16_rn(v);
                else
                    static_cast<float *>(a.out)[(i / 128) * a.ldc + row] = v;
            };
            for (int i = threadIdx.x; i < a.M * 128; i += kThreads) {
                float t = red[i];
                if (a.cols > a.M) t = __fadd_rn(t, red[a.M * 128 + i]);
                const float2 f = x_out[i / 128];
                t = __fmul_rn(__fmul_rn(t, f.x), f.y);
                if (NV) t = __fmul_rn(t, gw);
                if (whole)
                    store(i, t);
                else
                    place[i] = t;
            }
            if (whole) {
                __syncthreads();  // the sums are read: the next pair may end a tile too
            } else {
                // the last CTA to get here adds all parts, in CTA order
                const uint32_t q = tile * (uint32_t)s.pairs;
                const uint32_t first_cta = stream_owner(q, s), last_cta = stream_owner(q + s.pairs - 1, s);
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) arrived = atomicAdd(s.counters + tile, 1u);
                __syncthreads();
                if (arrived == last_cta - first_cta) {
                    __threadfence();
                    const float *p0 = s.part + (int64_t)(2 * first_cta + (stream_begin(first_cta, s) < q)) * a.M * 128;
                    const float *p1 = s.part + (int64_t)(2 * first_cta + 2) * a.M * 128;  // the others begin in this tile
                    for (int i = threadIdx.x; i < a.M * 32; i += kThreads) {
                        float4 t = __ldcg(reinterpret_cast<const float4 *>(p0) + i);
#pragma unroll 8
                        for (uint32_t k = 0; k < last_cta - first_cta; k++) {
                            const float4 u = __ldcg(reinterpret_cast<const float4 *>(p1 + (int64_t)k * 2 * a.M * 128) + i);
                            t.x = __fadd_rn(t.x, u.x);
                            t.y = __fadd_rn(t.y, u.y);
                            t.z = __fadd_rn(t.z, u.z);
                            t.w = __fadd_rn(t.w, u.w);
                        }
                        store(4 * i, t.x);
                        store(4 * i + 1, t.y);
                        store(4 * i + 2, t.z);
                        store(4 * i + 3, t.w);
                    }
                }
            }
            clear();
            from = 0;
        }
        if (++pair == s.pairs) {
            pair = 0;
            tile++;
        }
    }
    cp_async_wait<0>();
}

// How a call runs: the cheaper of the two forms by a model of the time in
// microseconds, fitted to sweeps on the B200 (67 shapes, N 303 .. 28672, K 256 ..
// 28672, M 1 .. 16, all formats, every tile width and cluster size: what it picks
// is within 4 % of the best on average, 28 % off in the worst).  Measured, NVFP4:
// 14336 x 4096, M = 1: tiles of 64 rows 11.4 us, of 128 rows in clusters of 2
// 11.5, in clusters of 4 (1.5 rounds of CTAs) 15.6; 28672 x 8192, M = 16: by
// tiles 65 us, streamed 44.1; 4096 x 4096, M = 16: 10.0 and 13.3.
struct Plan {
    int wr, cluster, slice, stage;  // by tiles: 32 * wr rows, K cut over a cluster
    bool streamed;
    double cost;
};

// What a step costs with 16 columns, against 8 (32: one CTA per SM, alone at it).
static double step_factor(int cols) { return cols <= 8 || cols > 16 ? 1.0 : 2.2; }

static Plan plan_tiles(int64_t N, int64_t K, int cols, bool rotated, int sms)
{
    const int per_sm = resident((cols + 7) / 8);
    // resident CTAs, as far as clusters of that size fill a GPC
    static constexpr double kFill[9] = {0, 1.0, 1.0, 0.95, 0.95, 0.92, 0.89, 0.87, 0.87};
    const int64_t chunks = (K + 127) / 128, atoms = (N + 127) / 128;
    Plan best = {};
    for (int wr = 4; wr >= 1; wr /= 2) {
        const int wk = 8 / wr;
        for (int cl = 1; cl <= 8; cl++) {
            const int64_t slice = (chunks + cl - 1) / cl;
            if ((chunks + slice - 1) / slice != cl) continue;  // every CTA has work
            const double ctas = (double)(atoms * (4 / wr) * cl), slots = (double)per_sm * sms * kFill[cl];
            const double rounds = ctas / slots, whole = floor(rounds), part = rounds - whole;
            const double turns = rounds <= 1.0 ? 1.0 : whole + (part > 0.0 ? 0.81 + 0.19 * part : 0.0);
            const double t = (0.505 + 0.584 * std::min(1.0, ctas / ((double)per_sm * sms))) * step_factor(cols);
            int64_t stage = (x_bytes(cols) / cols - 64) / 256 / wk * wk;
            stage = std::min(std::max<int64_t>(stage, wk), (slice + wk - 1) / wk * wk);
            // start and end, x to f16, the join of CTAs, the steps, further stages of x
            const double cost = turns * ((cl == 1 ? 2.06 : 2.69 + 0.021 * cl) + 0.0158 * (rotated ? 1.6 : 1.0) * cols * (double)slice +
                                         0.0345 * cols * (cl - 1) + t * (double)((slice + wk - 1) / wk) +
                                         2.66 * (double)((slice + stage - 1) / stage - 1));
            if (best.wr == 0 || cost < best.cost) best = {wr, cl, (int)slice, (int)stage, false, cost};
        }
    }
    return best;
}

static int stream_grid(int64_t total, int cols, int sms) { return (int)std::min<int64_t>(total, (int64_t)sms * resident((cols + 7) / 8)); }

static Plan search(int64_t N, int64_t K, int cols, bool rotated, int sms)
{
    Plan p = plan_tiles(N, K, cols, rotated, sms);
    const int64_t tiles = (N + 127) / 128, pairs = (K + 255) / 256, total = tiles * pairs;
    if (total >= int64_t(1) << 31) return p;  // the stream's 32-bit sequence; such a weight fits no GPU
    const double grid = stream_grid(total, cols, sms);
    // two launches and the join, x, the steps (over 16 columns: one CTA per SM)
    const double cost = 10.3 + 0.065 * cols + 1.02 * (cols <= 8 ? 1.0 : cols <= 16 ? 1.43 : 1.29) * (double)total / grid;
    p.streamed = cost < p.cost;
    return p;
}

// The last search of this thread is kept (a call asks twice, a decode loop again).
static Plan plan(int64_t N, int64_t K, int cols, bool rotated, int sms)
{
    struct Last {
        int64_t key[5];
        Plan p;
    };
    static thread_local Last last = {{-1, -1, -1, -1, -1}, {}};
    const int64_t key[5] = {N, K, cols, rotated, sms};
    if (!std::equal(key, key + 5, last.key)) {
        last.p = search(N, K, cols, rotated, sms);
        std::copy(key, key + 5, last.key);
    }
    return last.p;
}

template <int FMT, int WR, int NT, int BF16OUT>
static cudaError_t launch_t(const Args &a, const Plan &p, cudaStream_t st)
{
    auto kern = w4a16_kernel<FMT, WR, NT, BF16OUT>;
    const size_t x = (size_t)a.cols * (a.stage * 256 + 64);
    const size_t red = (size_t)(8 / WR) * a.cols * 32 * WR * 4 + (size_t)a.M * 32 * WR * 4;
    const size_t smem = std::max(ring_of(NT) + x, red);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), kMaxSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + 127) / 128 * (4 / WR) * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int FMT, int BF16OUT>
static cudaError_t launch_f(const Args &a, const Plan &p, cudaStream_t st)
{
    const int nt = (a.cols + 7) / 8;
#define FP4_W4_CASE(WR)                                                  \
    if (p.wr == WR) {                                                    \
        if (nt == 1) return launch_t<FMT, WR, 1, BF16OUT>(a, p, st);     \
        if (nt == 2) return launch_t<FMT, WR, 2, BF16OUT>(a, p, st);     \
        if (!BF16OUT) return launch_t<FMT, WR, BF16OUT ? 2 : 4, BF16OUT>(a, p, st); \
    }
    FP4_W4_CASE(4)
    FP4_W4_CASE(2)
    FP4_W4_CASE(1)
#undef FP4_W4_CASE
    return cudaErrorInvalidValue;
}

// Workspace of the streamed form, and its sizes.
struct Layout {
    size_t x_out, counters, part, total;
    int64_t tiles;
    int pairs, grid;
};

static Layout layout(int64_t M, int64_t N, int64_t K, int cols, int sms)
{
    Layout l;
    l.tiles = (N + 127) / 128;
    l.pairs = (int)((K + 255) / 256);
    l.grid = stream_grid(l.tiles * l.pairs, cols, sms);
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    l.x_out = up((size_t)cols * l.pairs * 512);
    l.counters = l.x_out + 256;
    l.part = l.counters + up((size_t)l.tiles * 4);
    l.total = l.part + (size_t)2 * l.grid * M * 128 * 4;
    return l;
}

template <int FMT, int NT, int BF16OUT>
static cudaError_t stream_t(const Args &a, const Stream &s, int64_t tiles, int grid, cudaStream_t st)
{
    auto kern = stream_kernel<FMT, NT, BF16OUT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), kMaxSmem, done);
    if (e != cudaSuccess) return e;
    e = launch_k(prepare_kernel<FMT, BF16OUT>, dim3((unsigned)a.M), dim3(512), 0, st, true, a, s, (int)tiles);
    if (e != cudaSuccess) return e;
    constexpr size_t smem = StreamShape<NT>::SMEM;
    return launch_k(kern, dim3((unsigned)grid), dim3(kThreads), smem, st, true, a, s);
}

template <int FMT, int BF16OUT>
static cudaError_t stream_f(const Args &a, void *ws, int sms, cudaStream_t st)
{
    const Layout l = layout(a.M, a.N, a.K, a.cols, sms);
    uint8_t *base = static_cast<uint8_t *>(ws);
    const int share = (int)(l.tiles * l.pairs / l.grid), more = (int)(l.tiles * l.pairs % l.grid);
    const Stream s = {base, reinterpret_cast<float2 *>(base + l.x_out), reinterpret_cast<unsigned *>(base + l.counters),
                      reinterpret_cast<float *>(base + l.part), l.pairs, share, more, make_fastdiv((uint32_t)share + 1),
                      make_fastdiv((uint32_t)share), make_fastdiv((uint32_t)l.pairs)};
    if (a.cols <= 8) return stream_t<FMT, 1, BF16OUT>(a, s, l.tiles, l.grid, st);
    if (a.cols <= 16) return stream_t<FMT, 2, BF16OUT>(a, s, l.tiles, l.grid, st);
    return stream_t<FMT, BF16OUT ? 2 : 4, BF16OUT>(a, s, l.tiles, l.grid, st);
}

}  // namespace w4

size_t linear_w4a16_workspace_bytes(int64_t M, int64_t N, int64_t K, int cols, bool rotated, int sms)
{
    return M > 0 && N > 0 && K > 0 && w4::plan(N, K, cols, rotated, sms).streamed ? w4::layout(M, N, K, cols, sms).total : 0;
}

cudaError_t launch_linear_w4a16(const uint16_t *x, int64_t ldx, int64_t M, int64_t K, int fmt, int hk, float ck,
                                const uint8_t *Wq, const uint8_t *Ws, const float *gW, int64_t N, int bf16out, void *C,
                                int64_t ldc, int w_early, void *ws, int sms, cudaStream_t st)
{
    w4::Args a = {};
    a.x = x;
    a.ldx = ldx;
    a.M = (int)M;
    a.hk = hk;
    a.cols = (int)(hk && !bf16out ? 2 * M : M);
    a.ck = ck;
    a.wq = Wq;
    a.ws = Ws;
    a.gw = gW;
    a.N = N;
    a.K = K;
    a.nkb4 = (K / (fmt == FP4_MXFP4 ? 32 : 16) + 3) / 4;
    a.out = C;
    a.ldc = ldc;
    a.chunks = (int)((K + 127) / 128);
    a.w_early = w_early;
    const w4::Plan p = w4::plan(N, K, a.cols, hk != 0, sms);
    if (p.streamed) {
        if (fmt == FP4_MXFP4) return bf16out ? w4::stream_f<FP4_MXFP4, 1>(a, ws, sms, st) : w4::stream_f<FP4_MXFP4, 0>(a, ws, sms, st);
        if (fmt == FP4_NVFP4) return bf16out ? w4::stream_f<FP4_NVFP4, 1>(a, ws, sms, st) : w4::stream_f<FP4_NVFP4, 0>(a, ws, sms, st);
        return bf16out ? w4::stream_f<FP4_MXFP4_16, 1>(a, ws, sms, st) : w4::stream_f<FP4_MXFP4_16, 0>(a, ws, sms, st);
    }
    a.cluster = p.cluster;
    a.slice = p.slice;
    a.stage = p.stage;
    if (fmt == FP4_MXFP4) return bf16out ? w4::launch_f<FP4_MXFP4, 1>(a, p, st) : w4::launch_f<FP4_MXFP4, 0>(a, p, st);
    if (fmt == FP4_NVFP4) return bf16out ? w4::launch_f<FP4_NVFP4, 1>(a, p, st) : w4::launch_f<FP4_NVFP4, 0>(a, p, st);
    return bf16out ? w4::launch_f<FP4_MXFP4_16, 1>(a, p, st) : w4::launch_f<FP4_MXFP4_16, 0>(a, p, st);
}

}  // namespace fp4
