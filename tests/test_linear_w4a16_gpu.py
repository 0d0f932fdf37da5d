"""GPU tests of the weight-only decode linear against a plain 64-bit product
of the dequantized weight and the (rotated) bf16 activations.

Bounds.  Unrotated x and the scaled weights are exact f16 operands, so fp32
output is off by the accumulation alone: K / 16 additions split over warps and
CTAs, held to the library's product tolerance 1e-5 * sum |x| |w|.  Rotated x:
hi + lo for fp32 output (2^-22) and the butterfly's fp32 (8 roundings, 2^-24),
within the same; for bf16 output each value's f16 rounding adds 2^-11 of its
term.  bf16 output: half a step, 2^-8 of the result.
"""
import pytest

import decode_ref as ref

pytestmark = pytest.mark.gpu

MX, NV, MX16 = 0, 1, 2


@pytest.fixture(scope="module")
def fp4():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_microscaling_quantization_b200 import build
    build.build()
    import fp4_microscaling_quantization_b200 as m
    return m


def inputs(M, N, K, seed, size=0.02):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=gen, device="cuda")
    x[:, ::61] *= 20
    w = torch.randn(N, K, generator=gen, device="cuda") * size
    return x.to(torch.bfloat16), w.to(torch.bfloat16)


def product64(x, W, fmt, hk, N, K):
    """(C, sum |x| |w|) in the rotated domain, which leaves the product alone."""
    q, s, g = W
    s = s[ref.atoms_index(N, K // ref.block_of(fmt), s.device)]
    w = ref.values64(q, s, fmt, g if fmt == NV else 1.0)
    xr = ref.rotate64(x.double(), hk)
    return xr @ w.T, xr.abs() @ w.abs().T


def check(fp4, x, W, fmt, hk, N, **kw):
    import torch
    want, bound = product64(x, W, fmt, hk, N, x.shape[1])
    got = fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, out_dtype=fp4.FP4_OUT_F32, **kw)
    half = fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, **kw)
    torch.cuda.synchronize()
    off = (got.double() - want).abs()
    assert (off <= 1e-5 * bound + 1e-30).all(), float((off / (bound + 1e-30)).max())
    off = (half.double() - want).abs()
    assert (off <= (1e-5 + (2.0**-11 if hk else 0)) * bound + 2.0**-8 * want.abs() + 1e-30).all()
    return got


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 8, 9, 15, 16])
def test_rows(fp4, fmt, M):
    x, w = inputs(M, 384, 1024, M)
    check(fp4, x, fp4.quantize(w, fmt), fmt, 0, 384)


# K tails of 32, one step, fewer steps than warps; N of one row, ragged tiles, many tiles
SIZES = [(1, 1, 32), (16, 1, 32), (3, 127, 96), (5, 129, 160), (4, 200, 4064), (2, 1000, 128), (1, 128 * 150 + 3, 256),
         (16, 300, 14336), (8, 64, 28704), (1, 4096, 4096)]


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(fp4, fmt, M, N, K):
    x, w = inputs(M, N, K, 7)
    check(fp4, x, fp4.quantize(w, fmt), fmt, 0, N)


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("hk", [16, 32, 64, 128])
@pytest.mark.parametrize("M,K", [(1, 128), (5, 1408), (16, 4096), (13, 14336)])
def test_rotated(fp4, fmt, hk, M, K):
    x, w = inputs(M, 320, K, hk + M)
    check(fp4, x, fp4.quantize(w, fmt, hadamard_k=hk), fmt, hk, 320)


def test_same_weight_as_the_quantizing_linear(fp4):
    """One weight serves both decode linears; with activations that E2M1 holds
    exactly they agree up to the sums' rounding."""
    import torch
    M, N, K = 4, 512, 2048
    gen = torch.Generator().manual_seed(1)
    x = torch.tensor(ref.GRID)[torch.randint(0, 8, (M, K), generator=gen)] * (1 - 2 * torch.randint(0, 2, (M, K), generator=gen))
    x[:, ::32] = 6.0
    x = x.to(torch.bfloat16).cuda()
    _, w = inputs(M, N, K, 2)
    W = fp4.quantize(w, MX)
    a = fp4.linear(x, W, MX, out_dtype=fp4.FP4_OUT_F32)
    _, bound = product64(x, W, MX, 0, N, K)
    b = fp4.linear_w4a16(x, W, MX, out_dtype=fp4.FP4_OUT_F32)
    assert ((a.double() - b.double()).abs() <= 2e-5 * bound).all()


def test_strides_and_outputs(fp4):
    """x as a view with a row stride, C inside a wider buffer; nothing else is written."""
    import torch
    M, N, K = 6, 260, 512
    x, w = inputs(M, N, K + 64, 3)
    W = fp4.quantize(w[:, :K].contiguous(), NV)
    xv = x[:, 64:]
    assert xv.stride(0) == K + 64
    buf = torch.full((M + 1, N + 20), 7.0, dtype=torch.bfloat16, device="cuda")
    got = fp4.linear_w4a16(xv, W, NV, out=buf)
    assert got is buf
    assert torch.equal(buf[:M, :N], fp4.linear_w4a16(xv.contiguous(), W, NV))
    assert (buf[M:] == 7).all() and (buf[:, N:] == 7).all()
    check(fp4, xv, W, NV, 0, N)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_ends_of_the_range(fp4, fmt):
    """Activations near bf16's largest and smallest, zero rows, rows far apart."""
    import torch
    x, w = inputs(5, 256, 512, 4)
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, :] = 0
    x[3, 77] = 2.0**100
    check(fp4, x, fp4.quantize(w, fmt), fmt, 0, 256)


def test_rows_of_far_apart_weights(fp4):
    """E8M0: rows up to 2^100 apart, and blocks 2^16 apart in a row."""
    import torch
    x, w = inputs(3, 256, 1024, 5)
    W = fp4.quantize(w, MX)
    gen = torch.Generator().manual_seed(6)
    s = (torch.randint(40, 140, (256, 1), generator=gen) + torch.randint(0, 17, (256, 32), generator=gen)).to(torch.uint8)
    W[1][ref.atoms_index(256, 32)] = s.cuda()
    check(fp4, x, W, MX, 0, 256)


def test_padding_rows_reach_no_result(fp4):
    """Scale rows past the weight's last may hold anything: NaN there."""
    import torch
    M, N, K = 2, 70, 128
    x, w = inputs(M, N, K, 8)
    for fmt in (NV, MX, MX16):
        W = fp4.quantize(w, fmt)
        want = fp4.linear_w4a16(x, W, fmt)
        used = torch.zeros_like(W[1], dtype=torch.bool)
        used[ref.atoms_index(N, K // ref.block_of(fmt)).cuda()] = True
        W[1][~used] = 0x7F if fmt == NV else 0xFF
        assert torch.equal(fp4.linear_w4a16(x, W, fmt), want)


def test_weights_static_and_graph(fp4):
    """Early weight loads give the same bits; captured and replayed with new x."""
    import torch
    x, w = inputs(4, 1024, 2048, 9)
    W = fp4.quantize(w, NV, hadamard_k=64)
    want = fp4.linear_w4a16(x, W, NV, hadamard_k=64)
    torch.cuda.synchronize()
    assert torch.equal(fp4.linear_w4a16(x, W, NV, hadamard_k=64, weights_static=True), want)
    xin, out = torch.zeros_like(x), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.linear_w4a16(xin, W, NV, hadamard_k=64, weights_static=True, out=out)
        again = fp4.linear_w4a16(xin, W, NV, hadamard_k=64)
    xin.copy_(x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(again, want)


# sizes that run as one stream over all CTAs (a workspace is asked for): odd
# numbers of steps, a ragged last tile, tiles cut between two and many CTAs,
# 8, 16 and 32 columns
@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("M,N,K,hk", [(8, 28003, 6176, 0), (16, 28003, 8224, 0), (9, 8192, 28672, 128), (12, 28672, 4096, 128)])
def test_streamed(fp4, fmt, M, N, K, hk):
    import torch
    x, w = inputs(M, N, K, M + hk)
    W = fp4.quantize(w, fmt, hadamard_k=hk)
    before = fp4.kernel_launches()
    fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, out_dtype=fp4.FP4_OUT_F32)
    assert fp4.kernel_launches() - before == 2  # x prepared, then the stream
    want = check(fp4, x, W, fmt, hk, N)
    # a workspace full of anything, used again, and early weight loads
    ws = torch.full((fp4.linear_w4a16_workspace_size(M, N, K, fmt),), 0xFF, dtype=torch.uint8, device="cuda")
    for static in (False, True, True):
        got = fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, out_dtype=fp4.FP4_OUT_F32, workspace=ws, weights_static=static)
        assert torch.equal(got, want)


# more tiles than CTAs: whole tiles that end a step after one another (K up to
# 256: at every step), and a cut one right behind a whole one
@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("M,N,K,hk", [(16, 128 * 2000 - 3, 256, 0), (14, 128 * 1000, 224, 32), (16, 128 * 800 + 1, 1024, 0),
                                      (8, 128 * 600, 2048, 0), (16, 128 * 333, 1536, 128)])
def test_streamed_whole_tiles(fp4, fmt, M, N, K, hk):
    import torch
    x, w = inputs(M, N, K, N + hk)
    W = fp4.quantize(w, fmt, hadamard_k=hk)
    before = fp4.kernel_launches()
    fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, out_dtype=fp4.FP4_OUT_F32)
    assert fp4.kernel_launches() - before == 2
    want = check(fp4, x, W, fmt, hk, N)
    for _ in range(8):
        assert torch.equal(fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, out_dtype=fp4.FP4_OUT_F32), want)


def test_streamed_graphs_share_a_workspace(fp4):
    """Two graphs of one stream with one workspace, replayed in turn; two
    streams at once with a workspace each."""
    import torch
    M, N, K = 16, 28003, 4128
    ws = torch.empty(fp4.linear_w4a16_workspace_size(M, N, K, NV), dtype=torch.uint8, device="cuda")
    sides = []
    for seed in (1, 2):
        x, w = inputs(M, N, K, seed)
        W = fp4.quantize(w, NV)
        want = fp4.linear_w4a16(x, W, NV)
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fp4.linear_w4a16(x, W, NV, out=out, workspace=ws)
        sides.append((g, x, W, out, want))
    for _ in range(3):
        for g, _, _, out, _ in sides:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, _, _, out, want in sides)
    streams, outs = [torch.cuda.Stream() for _ in sides], []
    for _ in range(4):
        for st, (_, x, W, _, want) in zip(streams, sides):
            with torch.cuda.stream(st):
                outs.append((fp4.linear_w4a16(x, W, NV), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


@pytest.mark.parametrize("M,N,K", [(8, 28003, 4096), (2, 4096, 2048)])
def test_weight_written_by_the_launch_before(fp4, M, N, K):
    """W quantized right before the product, into memory that the product before
    it read as another weight: in one stream, eager and as a graph."""
    import torch
    sides = []
    for seed in range(3):
        x, w = inputs(M, N, K, 20 + seed)
        W = fp4.quantize(w, NV)
        sides.append((x, w, fp4.linear_w4a16(x, W, NV)))
        torch.cuda.synchronize()
        del W

    def run():
        outs = []
        for _ in range(4):
            for x, w, want in sides:
                W = fp4.quantize(w, NV)
                outs.append((fp4.linear_w4a16(x, W, NV), want))
                del W
        return outs

    outs = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(2):
        for a, _ in outs:
            a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in outs)


@pytest.mark.parametrize("M,N,K", [(2, 256, 32768), (1, 128, 65536), (4, 130, 16384), (8, 64, 32768), (16, 40, 32768), (16, 200, 4096)])
def test_long_slices(fp4, M, N, K):
    """Slices of x longer than the part of it that is held at a time, hi and lo
    columns among them."""
    x, w = inputs(M, N, K, 11)
    check(fp4, x, fp4.quantize(w, NV, hadamard_k=64), NV, 64, N)
    check(fp4, x, fp4.quantize(w, MX), MX, 0, N)


def test_empty(fp4):
    import torch
    x, w = inputs(1, 128, 64, 10)
    W = fp4.quantize(w, NV)
    assert fp4.linear_w4a16(x[:0], W, NV).shape == (0, 128)


def check_one(fp4, x, W, fmt, hk, N, f32, launches):
    """One output type, and the form that it ran as: 1 launch by tiles, 2 streamed."""
    import torch
    want, bound = product64(x, W, fmt, hk, N, x.shape[1])
    before = fp4.kernel_launches()
    got = fp4.linear_w4a16(x, W, fmt, hadamard_k=hk, out_dtype=fp4.FP4_OUT_F32 if f32 else fp4.FP4_OUT_BF16)
    assert fp4.kernel_launches() - before == launches
    torch.cuda.synchronize()
    tol = 1e-5 * bound if f32 else (1e-5 + (2.0**-11 if hk else 0)) * bound + 2.0**-8 * want.abs()
    off = (got.double() - want).abs()
    assert (off <= tol + 1e-30).all(), float((off / (tol + 1e-30)).max())


# by tiles and streamed
BOTH_FORMS = [(4, 256, 512, 1), (3, 28672, 8192, 2)]


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("hk", [0, 64])
@pytest.mark.parametrize("M,N,K,launches", BOTH_FORMS)
def test_results_near_the_largest(fp4, fmt, hk, M, N, K, launches):
    """x up to 2^127, with finite results above 2^120."""
    x, w = inputs(M, N, K, 30)
    x[0] = 0
    x[0, 77] = 2.0**127
    x[1] = (x[1].double() * 2.0**116).to(x.dtype)
    W = fp4.quantize(w, fmt, hadamard_k=hk)
    want, _ = product64(x, W, fmt, hk, N, K)
    assert 2.0**120 < float(want.abs().max()) < 2.0**127
    for f32 in (True, False):
        check_one(fp4, x, W, fmt, hk, N, f32, launches)


@pytest.mark.parametrize("M,N,K,launches", BOTH_FORMS)
def test_far_tensor_scales(fp4, M, N, K, launches):
    """NVFP4 tensor scales from one end to the other, against x of the other."""
    x, w = inputs(M, N, K, 31)
    q, s, g = fp4.quantize(w, NV)
    for e in (-126, -100, -10, 60, 110):
        xs = (x.double() * 2.0 ** min(-e, 110)).to(x.dtype)
        for f32 in (True, False):
            check_one(fp4, xs, (q, s, g * 0 + 1.37 * 2.0**e), NV, 0, N, f32, launches)


@pytest.mark.parametrize("fmt", [MX, MX16])
@pytest.mark.parametrize("M,N,K,launches", BOTH_FORMS)
def test_far_block_scales(fp4, fmt, M, N, K, launches):
    """Rows with E8M0 scales from 2^-127 to 2^110 and x that keeps their results finite."""
    import torch
    x, w = inputs(M, N, K, 32)
    W = fp4.quantize(w, fmt)
    nkb = K // ref.block_of(fmt)
    gen = torch.Generator().manual_seed(33)
    s = torch.randint(0, 220, (N, 1), generator=gen) + torch.randint(0, 17, (N, nkb), generator=gen)
    s[:9] = torch.tensor([0, 1, 2, 17, 18, 19, 22, 23, 237])[:, None]
    W[1][ref.atoms_index(N, nkb).cuda()] = s.to(torch.uint8).cuda()
    for e in (-20, 5, 60):  # 2^60: only rows of small scales have finite results
        xs = (x.double() * 2.0**e).to(x.dtype)
        want, bound = product64(xs, W, fmt, 0, N, K)
        fine = (bound < 2.0**127).all(0)
        got = fp4.linear_w4a16(xs, W, fmt, out_dtype=fp4.FP4_OUT_F32)
        assert ((got.double() - want).abs() <= 1e-5 * bound + 1e-30)[:, fine].all()


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("M,N,K,launches", BOTH_FORMS)
@pytest.mark.parametrize("f32", [True, False])
def test_nan_scales_show(fp4, fmt, M, N, K, launches, f32):
    """A NaN scale in a row of W: NaN for every row of x, and nothing else changes."""
    import torch
    x, w = inputs(M, N, K, 34)
    x[0] = 0
    W = fp4.quantize(w, fmt)
    out = dict(out_dtype=fp4.FP4_OUT_F32 if f32 else fp4.FP4_OUT_BF16)
    clean = fp4.linear_w4a16(x, W, fmt, **out)
    nkb = K // ref.block_of(fmt)
    at = ref.atoms_index(N, nkb)
    rows = [0, 7, 31, 32, 100, 127, 128, N - 1]
    for i, n in enumerate(rows):
        W[1][at[n, [0, nkb - 1, 1, 5, nkb // 2][i % 5]]] = 0x7F if fmt == NV else 0xFF
    got = fp4.linear_w4a16(x, W, fmt, **out)
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[rows] = True
    assert torch.isnan(got[:, bad]).all()
    assert torch.equal(got[:, ~bad], clean[:, ~bad])


# by tiles, with x in several parts (the slice of a CTA is longer than what it
# holds of x at a time): 128, 64 and 32 rows to a tile, one CTA and clusters,
# last parts of one step, K tails of 32 and 64
@pytest.mark.parametrize("M,N,K,hk,f32", [
    (8, 10676, 6912, 64, False), (8, 10676, 6912, 0, True), (8, 20088, 1824, 0, False), (4, 23993, 2304, 128, True),
    (7, 4704, 11296, 0, True), (8, 2815, 14656, 0, False), (8, 9371, 5472, 0, True), (8, 65, 13344, 0, True),
    (7, 300, 17440, 0, False), (4, 67, 14400, 64, True),
])
@pytest.mark.parametrize("fmt", [MX, NV, MX16])
def test_tiles_with_x_in_parts(fp4, fmt, M, N, K, hk, f32):
    x, w = inputs(M, N, K, M + N)
    check_one(fp4, x, fp4.quantize(w, fmt, hadamard_k=hk), fmt, hk, N, f32, 1)


# streamed with fewer than 8 rows: columns of zeros beside the live ones
@pytest.mark.parametrize("M,N,K,hk", [(1, 57344, 8192, 0), (1, 57344, 8192, 128), (2, 28672, 8192, 0), (3, 28672, 8224, 0),
                                      (3, 28600, 8192, 64), (5, 14336, 14336, 0)])
@pytest.mark.parametrize("f32", [False, True])
def test_streamed_few_rows(fp4, M, N, K, hk, f32):
    for fmt in (NV, MX):
        x, w = inputs(M, N, K, M + hk)
        check_one(fp4, x, fp4.quantize(w, fmt, hadamard_k=hk), fmt, hk, N, f32, 2)
