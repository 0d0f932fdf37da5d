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
// output (2^-12 per value, below the output's own 2^-9), split into hi + lo
// columns for fp32 output.
//
// Work split.  A CTA is 8 warps: WR of them side by side along N (32 rows
// each), 8 / WR along K; a cluster of up to 8 CTAs splits K further and joins
// its sums over distributed shared memory in a fixed order.  One launch, no
// workspace, results repeat bit for bit.
#include <algorithm>

#include "frag.cuh"
#include "sm100.cuh"

namespace fp4 {
namespace w4 {

constexpr int kThreads = 256;
constexpr int kStep = 2560;                     // bytes of a warp's step: 32 rows x 64, and the scale words
constexpr int kStages = 4;                      // steps of a warp's ring
constexpr int kRing = 8 * kStages * kStep;
constexpr int kMaxSmem = 224 * 1024;            // what a launch may ask for
constexpr int kXBytes = 112 * 1024 - kRing;     // a stage of x: two CTAs per SM

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

template <int FMT, int WR, int NT, int BF16OUT>
__global__ void __launch_bounds__(kThreads, 2) w4a16_kernel(const __grid_constant__ Args a)
{
    constexpr int WK = 8 / WR, ROWS = 32 * WR;
    constexpr bool NV = FMT == FP4_NVFP4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float x_up[16];
    __shared__ uint32_t x_top[16];
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
    const bool kept = a.M * units <= kThreads;
    auto fetch_x = [&](int m, int64_t k, float *v) {
        uint4 raw[4] = {};
        if (m < a.M && k < a.K) {
            const uint4 *p = reinterpret_cast<const uint4 *>(a.x + m * a.ldx + k);
#pragma unroll
            for (int e = 0; e < 4; e++) raw[e] = __ldg(p + e);
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
                const uint4 t = __ldg(p + i);
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
            const uint32_t at = ring + slot * kStep;
            load(step + (kStages - 1) * WK, slot == 0 ? kStages - 1 : slot - 1);  // the slot consumed last
            slot = slot == kStages - 1 ? 0 : slot + 1;
            uint32_t w[4][4], sw[4], sc[4][2], ref[4];
#pragma unroll
            for (int j = 0; j < 4; j++) lds(at + j * 512, w[j], 4);
            lds(at + 2048, sw, 4);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (FMT == FP4_MXFP4) {
                    ref[j] = max_byte(sw[j]);
                    sc[j][0] = sc[j][1] = e8m0_rel((sw[j] >> (8 * c)) & 0xFF, ref[j]);
                } else {
                    const uint32_t two = (sw[j] >> (16 * (c & 1))) & 0xFFFF;
                    if (NV) {
                        const uint32_t f = e4m3x2_to_f16x2(two);
                        sc[j][0] = __byte_perm(f, 0, 0x1010);
                        sc[j][1] = __byte_perm(f, 0, 0x3232);
                    } else {
                        ref[j] = max_byte(sw[j]);
                        ref[j] = max(ref[j], __shfl_xor_sync(0xFFFFFFFFu, ref[j], 2));  // the step's other scale word
                        sc[j][0] = e8m0_rel(two & 0xFF, ref[j]);
                        sc[j][1] = e8m0_rel(two >> 8, ref[j]);
                    }
                }
            }
            // the step's own sums: added below with a rounding to nearest, which
            // the product's accumulation of many steps would not give
            float part[2][NT][4];
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int n = 0; n < NT; n++) part[t][n][0] = part[t][n][1] = part[t][n][2] = part[t][n][3] = 0.0f;
            const uint32_t xb = xs + (step - st) * 256 + c * 16;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t h[4][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    e2m1x8_to_f16(w[j][i], h[j]);
#pragma unroll
                    for (int e = 0; e < 4; e++) h[j][e] = mul_f16x2(h[j][e], sc[j][i >> 1]);
                }
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    uint32_t bx[4] = {0, 0, 0, 0};
                    if (8 * n + g < a.cols)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(bx[0]), "=r"(bx[1]), "=r"(bx[2]), "=r"(bx[3]) : "r"(xb + (8 * n + g) * pitch + i * 64));
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        float *d = part[t][n];
                        mma_f16(d, h[2 * t][0], h[2 * t + 1][0], h[2 * t][1], h[2 * t + 1][1], bx[0], bx[1]);
                        mma_f16(d, h[2 * t][2], h[2 * t + 1][2], h[2 * t][3], h[2 * t + 1][3], bx[2], bx[3]);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const float f0 = NV ? 1.0f : exp2i((int)ref[2 * t] - 127), f1 = NV ? 1.0f : exp2i((int)ref[2 * t + 1] - 127);
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
        sum[i] = __fmul_rn(s, x_up[m]);
    }
    const uint32_t cl = (uint32_t)a.cluster;
    if (cl > 1) cluster_sync();
    else __syncthreads();
    const float gw = NV ? *a.gw : 0.00390625f;  // e8m0_rel's 2^8
    for (int i = threadIdx.x * cl + rank; i < a.M * ROWS; i += kThreads * cl) {
        const int m = i / ROWS, row = i % ROWS;
        const int64_t n = atom * 128 + (row / (8 * WR)) * 32 + (tile % (4 / WR)) * (8 * WR) + row % (8 * WR);
        float t = 0.0f;
        for (uint32_t r = 0; r < cl; r++) t = __fadd_rn(t, ld_shared_cluster_f32(mapa_shared(smem_u32(sum + i), r)));
        t = __fmul_rn(t, gw);
        if (n < a.N) {
            if (BF16OUT)
                static_cast<__nv_bfloat16 *>(a.out)[m * a.ldc + n] = __float2bfloat16_rn(t);
            else
                static_cast<float *>(a.out)[m * a.ldc + n] = t;
        }
    }
    if (cl > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

struct Plan {
    int wr, cluster, slice, stage;
};

// Cuts N into tiles of 32 * wr rows and K into cluster slices.
static Plan plan(int64_t N, int64_t K, int cols, int sms)
{
    const int64_t chunks = (K + 127) / 128, atoms = (N + 127) / 128;
    Plan best = {};
    double least = 0.0;
    for (int wr = 4; wr >= 1; wr /= 2) {
        const int wk = 8 / wr;
        for (int cl = 1; cl <= 8; cl++) {
            const int64_t slice = (chunks + cl - 1) / cl;
            if ((chunks + slice - 1) / slice != cl) continue;  // every CTA has work
            const int64_t steps = (slice + wk - 1) / wk;
            const int64_t ctas = atoms * (4 / wr) * cl;
            const int64_t rounds = (ctas + 2 * sms - 1) / (2 * sms);
            const double full = (double)std::min<int64_t>(ctas, 2 * (int64_t)sms) / (2.0 * sms);
            const double cost = rounds * (2.5 + 0.005 * cols * slice + (0.3 + 0.3 * full) * steps);
            if (best.wr == 0 || cost < least) {
                least = cost;
                int64_t stage = (kXBytes / cols - 64) / 256 / wk * wk;
                stage = std::max<int64_t>(stage, wk);
                best = {wr, cl, (int)slice, (int)std::min<int64_t>(stage, (slice + wk - 1) / wk * wk)};
            }
        }
    }
    return best;
}

template <int FMT, int WR, int NT, int BF16OUT>
static cudaError_t launch_t(const Args &a, const Plan &p, cudaStream_t st)
{
    auto kern = w4a16_kernel<FMT, WR, NT, BF16OUT>;
    const size_t x = (size_t)a.cols * (a.stage * 256 + 64);
    const size_t red = (size_t)(8 / WR) * a.cols * 32 * WR * 4 + (size_t)a.M * 32 * WR * 4;
    const size_t smem = std::max(kRing + x, red);
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

}  // namespace w4

cudaError_t launch_linear_w4a16(const uint16_t *x, int64_t ldx, int64_t M, int64_t K, int fmt, int hk, float ck,
                                const uint8_t *Wq, const uint8_t *Ws, const float *gW, int64_t N, int bf16out, void *C,
                                int64_t ldc, int w_early, int sms, cudaStream_t st)
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
    const w4::Plan p = w4::plan(N, K, a.cols, sms);
    a.cluster = p.cluster;
    a.slice = p.slice;
    a.stage = p.stage;
    if (fmt == FP4_MXFP4) return bf16out ? w4::launch_f<FP4_MXFP4, 1>(a, p, st) : w4::launch_f<FP4_MXFP4, 0>(a, p, st);
    if (fmt == FP4_NVFP4) return bf16out ? w4::launch_f<FP4_NVFP4, 1>(a, p, st) : w4::launch_f<FP4_NVFP4, 0>(a, p, st);
    return bf16out ? w4::launch_f<FP4_MXFP4_16, 1>(a, p, st) : w4::launch_f<FP4_MXFP4_16, 0>(a, p, st);
}

}  // namespace fp4
