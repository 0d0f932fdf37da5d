"""GPU tests of attention over the paged FP4 cache against a plain 64-bit
implementation of its formula (decode_ref.attention64, where the error bounds
are derived).  fp32 output: within the bound; bf16 output: the weights' f16
rounding (2^-11 of sum w |v|) and the output's own (2^-8) come on top.
"""
import math

import pytest

import decode_ref as ref

pytestmark = pytest.mark.gpu

MX, NV, MX16 = 0, 1, 2
GK, GV = 0.037, 0.011


@pytest.fixture(scope="module")
def fp4():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_microscaling_quantization_b200 import build
    build.build()
    import fp4_microscaling_quantization_b200 as m
    return m


def make(fp4, fmt, dim, heads, page, hk, lens, seed, spread=4.0):
    """A cache with every page written, shuffled pages in the table, and a page
    of other tokens' data behind each sequence's last token."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need) + 2
    cache = fp4.KVCache.empty(pages, heads, page, dim, fmt, GK, GV, hk)
    n = pages * page
    x = torch.randn(2, n, heads, dim, generator=gen) * spread
    x[:, :: 7] *= 0.01
    x[0, :, :, ::13] *= 6
    x = x.to(torch.bfloat16).cuda()
    fp4.kv_append(cache, x[0], x[1], torch.arange(n, device="cuda"))
    order = torch.randperm(pages, generator=gen).int()
    table = torch.full((len(lens), max(need) + 1), 0, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def query(batch, heads, dim, seed, size=1.0):
    import torch
    return (torch.randn(batch, heads, dim, generator=torch.Generator().manual_seed(seed)) * size).to(torch.bfloat16).cuda()


def check(fp4, cache, q, table, lens, window=0, scale=None, **kw):
    import torch
    scale_ = cache.head_dim ** -0.5 if scale is None else scale
    want, lse, err, mag = ref.attention64(q, cache.k[0], cache.k[1], cache.v[0], cache.v[1], cache.fmt, cache.k[2],
                                          cache.v[2], cache.hadamard_k, table, lens, cache.page_size, scale_, window,
                                          cache.num_pages)
    got, l = fp4.paged_attention(q, cache, table, lens, scale=scale, window=window, out_dtype=fp4.FP4_OUT_F32,
                                 return_lse=True, **kw)
    half = fp4.paged_attention(q, cache, table, lens, scale=scale, window=window, **kw)
    torch.cuda.synchronize()
    tiny = 1e-30
    off = (got.double() - want).abs()
    assert (off <= err + tiny).all(), float((off / (err + tiny)).max())
    off = (half.double() - want).abs()
    assert (off <= err + 2.0**-11 * mag + 2.0**-8 * want.abs() + tiny).all()
    # log-sum-exp: the scores' error (err / mag is above it), and the logarithm in fp32
    fine = torch.isfinite(lse)
    assert torch.equal(torch.isfinite(l), fine) and (l[~fine] == -math.inf).all()
    rel = (err / mag.clamp(min=tiny)).amax(-1)
    assert ((l.double() - lse).abs()[fine] <= (rel + 2.0**-21 * (1 + lse.abs()))[fine]).all()
    return got


FORMATS = [(f, d, k) for f in (MX, NV, MX16) for d in (64, 128, 256) for k in (0, d if d < 256 else 128)]


@pytest.mark.parametrize("fmt,dim,hk", FORMATS)
def test_formats_and_lengths(fp4, fmt, dim, hk):
    """Every format, head size and rotation; lengths of 0, 1, page and step
    borders, several steps of every warp."""
    lens = [1, 0, 15, 16, 17, 31, 33, 64, 127, 200, 511, 700]
    cache, table, n = make(fp4, fmt, dim, 2, 16, hk, lens, 1)
    got = check(fp4, cache, query(len(lens), 8, dim, 2), table, n)
    assert not got[1].any()


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16, 17])
@pytest.mark.parametrize("fmt,dim", [(NV, 128), (MX, 64)])
def test_groups(fp4, group, fmt, dim):
    """Any number of query heads to a key head, below and above one CTA's 8."""
    cache, table, n = make(fp4, fmt, dim, 3, 32, 16, [70, 3], 3)
    check(fp4, cache, query(2, 3 * group, dim, 4), table, n)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fmt,dim", [(NV, 128), (MX, 256), (MX16, 64)])
def test_pages(fp4, page, fmt, dim):
    cache, table, n = make(fp4, fmt, dim, 2, page, 0, [page - 1, page, page + 1, 3 * page + 5], 5)
    check(fp4, cache, query(4, 4, dim, 6), table, n)


@pytest.mark.parametrize("fmt,dim,hk", [(NV, 128, 0), (MX, 128, 32), (MX16, 64, 0), (NV, 256, 0), (MX, 64, 64)])
def test_long_sequences_are_cut_and_joined(fp4, fmt, dim, hk):
    """Many chunks, uneven lengths (some end in the first chunk, one is empty)."""
    lens = [9000, 1, 0, 513, 4096, 2047]
    cache, table, n = make(fp4, fmt, dim, 1, 64, hk, lens, 7, spread=2.0)
    assert fp4.paged_attention_workspace_size(len(lens), 4, 1, dim, 9000) > 0
    check(fp4, cache, query(len(lens), 4, dim, 8), table, n, max_seq_len=9000)


@pytest.mark.parametrize("window", [1, 16, 31, 100, 1000, 5000])
@pytest.mark.parametrize("fmt", [NV, MX])
def test_window(fp4, window, fmt):
    cache, table, n = make(fp4, fmt, 64, 2, 16, 0, [1, 0, 40, 999, 2500], 9)
    check(fp4, cache, query(5, 4, 64, 10), table, n, window=window)


@pytest.mark.parametrize("fmt,dim", [(NV, 128), (MX, 64), (MX16, 256)])
def test_missing_pages_take_no_part(fp4, fmt, dim):
    """Entries outside the cache: single pages, a whole sequence."""
    import torch
    cache, table, n = make(fp4, fmt, dim, 2, 16, 0, [200, 90, 50, 1000], 11)
    table[0, 1::3] = -1
    table[0, 2] = 1 << 30
    table[1, :] = cache.num_pages  # nothing left
    table[2, :3] = torch.iinfo(torch.int32).min
    got = check(fp4, cache, query(4, 6, dim, 12), table, n)
    assert not got[1].any()


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_what_lies_past_the_length_is_not_used(fp4, fmt, dim):
    """NaN scales in every slot that takes no part."""
    import torch
    lens = [1, 17, 40, 600]
    cache, table, n = make(fp4, fmt, dim, 1, 32, 0, lens, 13)
    q = query(4, 2, dim, 14)
    clean = fp4.paged_attention(q, cache, table, n, window=30)
    live = torch.zeros(cache.num_pages * 32, dtype=torch.bool)
    for b, m in enumerate(lens):
        t = torch.arange(max(0, m - 30), m)
        live[table[b].cpu().long()[t // 32] * 32 + t % 32] = True
    dead = (~live).reshape(cache.num_pages, 32).cuda()
    for s in (cache.k[1], cache.v[1]):
        s[:, 0][dead] = 0x7F if fmt == NV else 0xFF
    assert torch.equal(fp4.paged_attention(q, cache, table, n, window=30), clean)


def test_live_nan_shows(fp4):
    import torch
    cache, table, n = make(fp4, NV, 64, 1, 16, 0, [40, 40], 15)
    cache.v[1][int(table[0, 1]), 0, 3] = 0x7F
    out = fp4.paged_attention(query(2, 2, 64, 16), cache, table, n)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    cache, table, n = make(fp4, NV, 64, 1, 16, 0, [40, 40], 15)
    cache.k[1][int(table[0, 1]), 0, 3] = 0x7F
    out = fp4.paged_attention(query(2, 2, 64, 16), cache, table, n)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


def test_large_scores_and_tiny_queries(fp4):
    """Scores of several hundred (one token takes all), queries near bf16's ends."""
    for size in (300.0, 1e-30, 0.0):
        cache, table, n = make(fp4, NV, 128, 1, 16, 0, [300], 17)
        check(fp4, cache, query(1, 4, 128, 18, size), table, n)
    cache, table, n = make(fp4, MX, 64, 1, 16, 0, [300], 17)
    check(fp4, cache, query(1, 4, 64, 18, 3e37), table, n, scale=1e-37)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, -3.0])
@pytest.mark.parametrize("fmt", [NV, MX])
def test_any_scale(fp4, scale, fmt):
    """Equal weights, scores turned over, with missing pages and a cut window."""
    cache, table, n = make(fp4, fmt, 64, 2, 16, 0, [100, 1, 0, 1500], 60)
    table[3, 5:9] = -1
    check(fp4, cache, query(4, 6, 64, 61), table, n, scale=scale)
    check(fp4, cache, query(4, 6, 64, 61), table, n, scale=scale, window=90)


def test_empty_tables_and_batches(fp4):
    cache, table, n = make(fp4, NV, 128, 1, 16, 0, [30, 40], 62)
    q = query(2, 4, 128, 63)
    out, lse = fp4.paged_attention(q, cache, table[:, :0], n, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    out, lse = fp4.paged_attention(q, cache, table[:, :0], n, max_seq_len=100000, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert fp4.paged_attention(q[:0], cache, table[:0], n[:0]).shape == (0, 4, 128)
    check(fp4, cache, q, table, n, max_seq_len=1 << 20)  # a bound far above the lengths and the table


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("dim,hk,group", [(256, 16, 16), (256, 64, 3), (128, 16, 12), (64, 32, 24)])
def test_rotations_and_wide_groups(fp4, fmt, dim, hk, group):
    cache, table, n = make(fp4, fmt, dim, 2, 64, hk, [77, 650, 2000], 64)
    check(fp4, cache, query(3, 2 * group, dim, 65), table, n)


def test_far_apart_scales(fp4):
    """E8M0 scales over many binades: between tokens, and 2^20 within a row."""
    import torch
    cache, table, n = make(fp4, MX, 128, 1, 16, 0, [400], 19)
    gen = torch.Generator().manual_seed(20)
    cache.k[1].copy_(torch.randint(110, 128, cache.k[1].shape, generator=gen).to(torch.uint8))
    cache.v[1].copy_(torch.randint(40, 128, cache.v[1].shape[:3] + (1,), generator=gen).to(torch.uint8).expand(cache.v[1].shape))
    check(fp4, cache, query(1, 4, 128, 21, 0.3), table, n)


def test_lengths_above_the_bounds(fp4):
    """Above max_seq_len or the table's reach a length is cut; negative is empty."""
    import torch
    cache, table, n = make(fp4, NV, 64, 1, 16, 0, [64, 64, 64], 22)
    q = query(3, 2, 64, 23)
    want = fp4.paged_attention(q, cache, table[:, :3], torch.tensor([48, 48, 0], dtype=torch.int32, device="cuda"))
    huge = torch.tensor([1 << 30, 49, -5], dtype=torch.int32, device="cuda")
    assert torch.equal(fp4.paged_attention(q, cache, table[:, :3], huge), want)
    assert torch.equal(fp4.paged_attention(q, cache, table, huge, max_seq_len=48), want)


def test_strided_and_shared(fp4):
    """Queries inside a fused projection, one table row for all sequences."""
    import torch
    cache, table, n = make(fp4, MX16, 128, 2, 16, 0, [100, 60, 100], 24)
    qkv = query(3, 12, 128, 25)
    q = qkv[:, 2:10]
    row = table[:1].expand(3, -1)
    assert row.stride(0) == 0
    check(fp4, cache, q, row, n.clamp(max=100))
    check(fp4, cache, qkv[:, ::3], table[:, :8], n)


def test_repeats_bit_for_bit_on_streams(fp4):
    """Two calls at once on two streams, each with its own workspace."""
    import torch
    cache, table, n = make(fp4, NV, 128, 1, 16, 0, [3000, 2000], 26)
    q = query(2, 8, 128, 27)
    want = fp4.paged_attention(q, cache, table, n)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(fp4.paged_attention(q, cache, table, n))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_far_pages(fp4):
    """Byte offsets past 2^32: the last pages of a cache of over 4 GiB a side."""
    import torch
    pages, heads, page, dim = 40000, 8, 256, 128
    cache = fp4.KVCache.empty(pages, heads, page, dim, NV, GK, GV)
    gen = torch.Generator().manual_seed(40)
    table = torch.tensor([[pages - 1, 0, pages - 2], [39000, 38999, 7]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([700, 513], dtype=torch.int32, device="cuda")
    for row in table.tolist():
        for pg in row:
            x = torch.randn(2, page, heads, dim, generator=gen).to(torch.bfloat16).cuda()
            fp4.kv_append(cache, x[0], x[1], pg * page + torch.arange(page, device="cuda"))
    check(fp4, cache, query(2, 16, dim, 41), table, lens)


def test_workspace_contents_do_not_matter(fp4):
    import torch
    cache, table, n = make(fp4, NV, 128, 1, 16, 0, [3000, 5], 42)
    q = query(2, 4, 128, 43)
    want = fp4.paged_attention(q, cache, table, n)
    need = fp4.paged_attention_workspace_size(2, 4, 1, 128, table.shape[1] * 16)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(fp4.paged_attention(q, cache, table, n, workspace=ws), want)
    with pytest.raises(fp4.Fp4Error):
        fp4.paged_attention(q, cache, table, n, workspace=ws[:need - 1])


def test_decode_layer(fp4):
    """One attention layer of a decode step as a server runs it, captured once
    and replayed: the fused projection (weight-only), its keys and values into
    the cache, attention, the output projection.  Each part is checked against
    64 bits from the values that it was given."""
    import torch
    B, H, G, D, page, E = 5, 2, 4, 128, 32, 1024
    HQ, rows = H * G, (H * G + 2 * H) * D
    gen = torch.Generator().manual_seed(50)
    cache, _, _ = make(fp4, NV, D, H, page, 64, [400] * B, 51)
    table = torch.arange(B * 13, dtype=torch.int32, device="cuda").reshape(B, 13)
    lens = torch.tensor([1, 33, 64, 400, 0], dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    x = torch.zeros(B, E, dtype=torch.bfloat16, device="cuda")
    w_in, w_out = ((torch.randn(n, k, generator=gen) * k ** -0.5).to(torch.bfloat16).cuda() for n, k in ((rows, E), (E, HQ * D)))
    Win, Wout = fp4.quantize(w_in, MX, hadamard_k=32), fp4.quantize(w_out, NV)
    qkv = torch.empty(B, rows, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(B, E, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(B, HQ, D, dtype=torch.bfloat16, device="cuda")

    def layer():
        fp4.linear_w4a16(x, Win, MX, hadamard_k=32, out=qkv, weights_static=True)
        q, k, v = qkv.view(B, HQ + 2 * H, D).split((HQ, H, H), 1)
        fp4.kv_append(cache, k, v, slots)
        fp4.paged_attention(q, cache, table, lens, out=out)
        fp4.linear_w4a16(out.view(B, HQ * D), Wout, NV, out=y, weights_static=True)

    layer()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for step in range(4):
        x.copy_(torch.randn(B, E, generator=gen).to(torch.bfloat16))
        pos = lens.long()
        slots.copy_(table.long().gather(1, (pos // page)[:, None])[:, 0] * page + pos % page)
        slots[4] = -1  # a padded row of the batch: no token, no length
        lens[:4] += 1
        g.replay()
        torch.cuda.synchronize()
        for got, a, W, wf, fmt, hk in ((qkv, x, Win, w_in, MX, 32), (y, out.view(B, HQ * D), Wout, w_out, NV, 0)):
            n, kk = wf.shape
            s = W[1][ref.atoms_index(n, kk // ref.block_of(fmt), "cuda")]
            wv = ref.values64(W[0], s, fmt, W[2] if fmt == NV else 1.0)
            av = ref.rotate64(a.double(), hk)
            want, bound = av @ wv.T, av.abs() @ wv.abs().T
            assert ((got.double() - want).abs() <= (1e-5 + (2.0**-11 if hk else 0)) * bound + 2.0**-8 * want.abs()).all()
        q, k, v = qkv.view(B, HQ + 2 * H, D).split((HQ, H, H), 1)
        fresh = fp4.KVCache.empty(1, H, 16, D, NV, GK, GV, 64)
        fp4.kv_append(fresh, k.contiguous(), v.contiguous(), torch.arange(B, device="cuda"))
        for b in range(4):
            pg, at = int(slots[b]) // page, int(slots[b]) % page
            for side in (0, 1):
                assert torch.equal((cache.k, cache.v)[side][0][pg, :, at], (fresh.k, fresh.v)[side][0][0, :, b])
        want, _, err, mag = ref.attention64(q, cache.k[0], cache.k[1], cache.v[0], cache.v[1], NV, cache.k[2], cache.v[2], 64,
                                            table, lens, page, D ** -0.5, 0, cache.num_pages)
        assert ((out.double() - want).abs() <= err + 2.0**-11 * mag + 2.0**-8 * want.abs() + 1e-30).all()
        assert not out[4].any() and not y[4].any()


def test_decode_step_captured(fp4):
    """Append and attention in one graph, replayed while the sequences grow, as
    a decode loop uses them; two graphs share one workspace in one stream."""
    import torch
    B, H, G, D, page = 3, 2, 4, 64, 16
    start = [30, 5, 600]
    cache, _, _ = make(fp4, NV, D, H, page, 32, [700] * B, 28)
    per = 44
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").reshape(B, per)
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    k, v, q = (torch.zeros(B, n, D, dtype=torch.bfloat16, device="cuda") for n in (H, H, H * G))
    ws = torch.empty(max(16, fp4.paged_attention_workspace_size(B, H * G, H, D, per * page)), dtype=torch.uint8, device="cuda")
    out = [torch.empty(B, H * G, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(o):
        fp4.kv_append(cache, k, v, slots)
        fp4.paged_attention(q, cache, table, lens, out=o, workspace=ws)

    step(out[0])
    torch.cuda.synchronize()
    graphs = []
    for o in out:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append(g)
    gen = torch.Generator().manual_seed(29)
    for i in range(6):
        pos = lens.long()
        slots.copy_(table.long().gather(1, (pos // page)[:, None])[:, 0] * page + pos % page)
        lens += 1
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen).to(torch.bfloat16))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        want, _, err, mag = ref.attention64(q, cache.k[0], cache.k[1], cache.v[0], cache.v[1], NV, cache.k[2], cache.v[2],
                                            32, table, lens, page, D ** -0.5, 0, cache.num_pages)
        off = (out[i % 2].double() - want).abs()
        assert (off <= err + 2.0**-11 * mag + 2.0**-8 * want.abs() + 1e-30).all()


def reference(cache, q, table, lens, scale=None, window=0):
    scale = cache.head_dim ** -0.5 if scale is None else scale
    return ref.attention64(q, cache.k[0], cache.k[1], cache.v[0], cache.v[1], cache.fmt, cache.k[2], cache.v[2],
                           cache.hadamard_k, table, lens, cache.page_size, scale, window, cache.num_pages)


@pytest.mark.parametrize("fmt", [MX, NV, MX16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("side", ["k", "v"])
def test_nan_scales_of_live_tokens(fp4, fmt, dim, side):
    """One NaN scale byte of a live token.  Of a key: its score is NaN, and with
    it every head of that key head, whatever the score's sign (both occur among
    the heads) and wherever the token lies: alone in its sequence, alone in its
    step, the last of many.  Of a value: NaN in its block's channels and in no
    other.  The other sequences keep their bits."""
    import torch
    lens = [1, 17, 33, 65, 129, 129, 700, 64]
    nblk = dim // ref.block_of(fmt)
    cache, table, n = make(fp4, fmt, dim, 2, 16, 0, lens, 70, spread=1.0)
    q = query(len(lens), 16, dim, 71)
    q[:, 8:] = -q[:, :8]  # heads of key head 1; key head 0 gets both signs below
    q[:, 4:8] = -q[:, :4]
    clean = reference(cache, q, table, n)
    for b, t in enumerate([0, 16, 32, 64, 128, 5, 699]):  # the last sequence has none
        s = (cache.k if side == "k" else cache.v)[1]
        s[int(table[b, t // 16]), 0, t % 16, [0, nblk - 1, nblk // 2][b % 3]] = 0x7F if fmt == NV else 0xFF
    want, lse, err, mag = reference(cache, q, table, n)
    assert torch.isnan(want[:7, :8]).any(-1).all() and not torch.isnan(want[:, 8:]).any() and not torch.isnan(want[7]).any()
    got, l = fp4.paged_attention(q, cache, table, n, out_dtype=fp4.FP4_OUT_F32, return_lse=True)
    half = fp4.paged_attention(q, cache, table, n)
    for o in (got, half):
        assert torch.equal(torch.isnan(o), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert ((got.double() - want).abs() <= err + 1e-30)[fine].all()
    assert ((half.double() - want).abs() <= err + 2.0**-11 * mag + 2.0**-8 * want.abs() + 1e-30)[fine].all()
    assert torch.equal(torch.isnan(l), torch.isnan(lse))
    rel = (clean[2] / clean[3].clamp(min=1e-30)).amax(-1)  # as in check, of the sequences without NaN
    ok = ~torch.isnan(lse)
    assert ((l.double() - lse).abs()[ok] <= (rel + 2.0**-21 * (1 + lse.abs()))[ok]).all()


@pytest.mark.parametrize("fmt", [MX, MX16])
@pytest.mark.parametrize("hk", [0, 32])
@pytest.mark.parametrize("cut", [False, True])
def test_nan_scales_rotated_and_cut(fp4, fmt, hk, cut):
    """The same through the join of chunks and the rotation, several NaN in a sequence."""
    import torch
    lens = [3000, 2000]
    cache, table, n = make(fp4, fmt, 128, 1, 16, hk, lens, 72)
    cache.v[1].clamp_(max=120)
    for t in (3, 900, 901, 2999):
        cache.v[1][int(table[0, t // 16]), 0, t % 16, 1] = 0xFF
    q = query(2, 4, 128, 73)
    want, _, err, _ = reference(cache, q, table, n)
    got = fp4.paged_attention(q, cache, table, n, out_dtype=fp4.FP4_OUT_F32, max_seq_len=(1 << 20) if cut else 3000)
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert ((got.double() - want).abs() <= err + 1e-30)[fine].all()
    cache.k[1][int(table[0, 1500 // 16]), 0, 1500 % 16, 2] = 0xFF
    for o in (fp4.paged_attention(q, cache, table, n), fp4.paged_attention(q, cache, table, n, out_dtype=fp4.FP4_OUT_F32)):
        assert torch.isnan(o[0]).all() and torch.isfinite(o[1]).all()


@pytest.mark.parametrize("fmt,dim", [(NV, 128), (MX, 64), (MX16, 256)])
@pytest.mark.parametrize("top", [1e7, 3e7, 1e8, 1e9, 1e12, 1e20, 1e30])
def test_scores_of_any_size(fp4, fmt, dim, top):
    """Scores far past the point where fp32 has steps of more than 1.  All keys
    are alike but every third, which is zero: a head attends to the first kind
    in equal shares where their score is positive, else to the second."""
    import torch
    lens = [1, 40, 333, 3000]
    cache, table, n = make(fp4, fmt, dim, 1, 16, 0, lens, 77)
    for t in cache.k[:2]:
        t.copy_(t[0, 0, 0].expand(t.shape).clone())
    k64 = ref.values64(cache.k[0][0, 0, 0], cache.k[1][0, 0, 0], fmt, cache.k[2])
    for b, m in enumerate(lens):
        for t in range(2, m, 3):
            cache.k[0][int(table[b, t // 16]), 0, t % 16] = 0
    q = query(4, 6, dim, 78)
    x = q.double() @ k64
    assert (x > 0).any() and (x < 0).any()
    scale = float(torch.tensor(top / float(x.abs().max()), dtype=torch.float32))
    assert float(x.abs().min()) * scale > 200.0  # the other kind's weight is below 2^-288
    got, lse = fp4.paged_attention(q, cache, table, n, scale=scale, out_dtype=fp4.FP4_OUT_F32, return_lse=True)
    half = fp4.paged_attention(q, cache, table, n, scale=scale)
    for b, m in enumerate(lens):
        for h in range(6):
            xb = float(x[b, h]) * scale
            t = [i for i in range(m) if (i % 3 != 2) == (xb > 0 or m == 1)]
            top_x = xb if xb > 0 or m == 1 else 0.0
            t = torch.tensor(t, device="cuda")
            pg = table[b].long()[t // 16]
            v = ref.values64(cache.v[0][pg, 0, t % 16], cache.v[1][pg, 0, t % 16], fmt, cache.v[2])
            want, mag = v.mean(0), v.abs().mean(0)
            # the weights are alike: additions, the split of a weight and the division remain
            tol = (len(t) / 16 + 64) * 2.0**-22 * mag
            assert ((got[b, h].double() - want).abs() <= tol).all()
            assert ((half[b, h].double() - want).abs() <= tol + 2.0**-11 * mag + 2.0**-8 * want.abs()).all()
            # the score: q in 22 bits, dim / 16 additions, scale factors; its steps in fp32 (four roundings)
            lim = (dim / 16 + 8) * 2.0**-22 * float(q[b, h].double().abs() @ k64.abs()) * scale * (top_x != 0)
            assert abs(float(lse[b, h]) - top_x - math.log(len(t))) <= lim + 2.0**-22 * abs(top_x) + 2.0**-20


@pytest.mark.parametrize("fmt,dim", [(NV, 128), (MX, 64), (MX16, 256)])
@pytest.mark.parametrize("top", [3e7, 1e9, 1e20])
def test_far_scores_that_are_passed(fp4, fmt, dim, top):
    """Scores of -top until the last token, whose score is 0: it takes all (for
    the heads whose scores are +top, none)."""
    import torch
    lens = [130, 700, 5000]
    cache, table, n = make(fp4, fmt, dim, 1, 16, 0, lens, 80)
    for t in cache.k[:2]:
        t.copy_(t[0, 0, 0].expand(t.shape).clone())
    k64 = ref.values64(cache.k[0][0, 0, 0], cache.k[1][0, 0, 0], fmt, cache.k[2])
    for b, m in enumerate(lens):
        cache.k[0][int(table[b, (m - 1) // 16]), 0, (m - 1) % 16] = 0
    q = query(3, 4, dim, 81)
    q[:, 2:] = -q[:, :2]
    x = q.double() @ k64
    scale = float(torch.tensor(top / float(x.abs().max()), dtype=torch.float32))
    assert float(x.abs().min()) * scale > 200.0
    got = fp4.paged_attention(q, cache, table, n, scale=scale, out_dtype=fp4.FP4_OUT_F32)
    half = fp4.paged_attention(q, cache, table, n, scale=scale)
    for b, m in enumerate(lens):
        for h in range(4):
            t = torch.arange(m - 1, device="cuda") if x[b, h] > 0 else torch.tensor([m - 1], device="cuda")
            pg = table[b].long()[t // 16]
            v = ref.values64(cache.v[0][pg, 0, t % 16], cache.v[1][pg, 0, t % 16], fmt, cache.v[2])
            want, mag = v.mean(0), v.abs().mean(0)
            tol = (len(t) / 16 + 64) * 2.0**-22 * mag
            assert ((got[b, h].double() - want).abs() <= tol).all()
            assert ((half[b, h].double() - want).abs() <= tol + 2.0**-11 * mag + 2.0**-8 * want.abs()).all()


@pytest.mark.parametrize("fmt", [MX, MX16])
@pytest.mark.parametrize("length", [300, 5000])
def test_far_value_scales(fp4, fmt, length):
    """E8M0 scales of values from 2^-127 to 2^110, values of one sign: each
    result is a mean of them, so it is finite."""
    import torch
    for lo in (0, 5, 60, 221):
        cache, table, n = make(fp4, fmt, 64, 1, 16, 0, [length], 74)
        cache.v[0].bitwise_and_(0x77)
        gen = torch.Generator().manual_seed(75)
        cache.v[1].copy_(torch.randint(lo, lo + 17, cache.v[1].shape, generator=gen).to(torch.uint8))
        q = query(1, 4, 64, 76, 0.3)
        want, _, err, mag = reference(cache, q, table, n)
        got = fp4.paged_attention(q, cache, table, n, out_dtype=fp4.FP4_OUT_F32)
        half = fp4.paged_attention(q, cache, table, n)
        small = 2.0**-125  # results below the normal numbers
        assert ((got.double() - want).abs() <= err + small).all()
        assert ((half.double() - want).abs() <= err + 2.0**-11 * mag + 2.0**-8 * want.abs() + small).all()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("fmt,dim,hk", [(NV, 128, 0), (MX, 64, 64), (MX16, 256, 0)])
def test_queries_that_are_not_finite(fp4, fmt, dim, hk, value):
    """NaN for that head of that sequence, every other row keeps its bits."""
    import torch
    lens = [1, 40, 600, 3000]
    cache, table, n = make(fp4, fmt, dim, 2, 16, hk, lens, 90)
    q = query(4, 6, dim, 91)
    cache.k[0][:, 0, :, 0] &= 0x0F  # element 1 of every key is 0: 0 * inf is NaN
    ref_out, ref_lse = fp4.paged_attention(q, cache, table, n, out_dtype=fp4.FP4_OUT_F32, return_lse=True)
    bad = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    bad[:, 1] = True
    bad[2, 0] = True
    q[:, 1, 1] = value
    q[2, 0, 1] = value
    got, l = fp4.paged_attention(q, cache, table, n, out_dtype=fp4.FP4_OUT_F32, return_lse=True)
    half = fp4.paged_attention(q, cache, table, n)
    assert torch.isnan(got[bad]).all() and torch.isnan(half[bad]).all() and torch.isnan(l[bad]).all()
    assert torch.equal(got[~bad], ref_out[~bad]) and torch.equal(l[~bad], ref_lse[~bad]) and torch.isfinite(half[~bad]).all()
