"""GPU tests of the paged FP4 key-value cache: what fp4_kv_append writes is
bit for bit what the oracle's quantizer gives for each head row (elements and
scales), in the right slots and nowhere else; what fp4_kv_gather reads is bit
for bit the oracle's dequantization.
"""
import numpy as np
import pytest

from helpers import bf16_tensor_bits

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


def draw(shape, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * torch.exp2(torch.randint(-6, 7, shape[:-1] + (1,), generator=gen).float())
    x.view(-1)[:: 97] *= 30
    return x.to(torch.bfloat16)


def oracle_rows(orc, x, fmt, hk, tie, rule, g):
    """(q, s) of each head row of x (T, H, D), and the values read back."""
    T, H, D = x.shape
    q, s, _ = orc.quantize(bf16_tensor_bits(x.reshape(T * H, D)), fmt, hadamard_k=hk, tie=tie, mx_rule=rule,
                           gscale=g if fmt == NV else None)
    back = orc.dequantize(q, s, np.float32(g) if fmt == NV else 1.0, fmt, hadamard_k=hk)
    return q.reshape(T, H, -1), s.reshape(T, H, -1), back.reshape(T, H, D)


def new_cache(fp4, pages, heads, page, dim, fmt, hk):
    """A cache full of a byte that no test writes everywhere: untouched places show."""
    c = fp4.KVCache.empty(pages, heads, page, dim, fmt, GK, GV, hk)
    for t in (c.k[0], c.k[1], c.v[0], c.v[1]):
        t.fill_(0x5A)
    return c


CASES = [  # fmt, dim, heads, page, hk, tokens
    (MX, 64, 1, 16, 0, 1), (MX, 128, 8, 16, 0, 37), (MX, 256, 2, 32, 128, 9), (MX, 64, 5, 64, 64, 130),
    (NV, 64, 8, 16, 16, 61), (NV, 128, 3, 256, 0, 200), (NV, 128, 8, 16, 128, 17), (NV, 256, 1, 64, 32, 33),
    (MX16, 64, 2, 128, 0, 5), (MX16, 128, 4, 32, 64, 50), (MX16, 256, 7, 16, 0, 19),
]


@pytest.mark.parametrize("fmt,dim,heads,page,hk,tokens", CASES)
@pytest.mark.parametrize("tie,rule", [(0, 0), (1, 1)])
def test_append_and_gather(fp4, orc, fmt, dim, heads, page, hk, tokens, tie, rule):
    import torch
    k, v = draw((tokens, heads, dim), 1), draw((tokens, heads, dim), 2)
    k[0] = 0  # a row of zeros
    v[-1, 0, 0] = -0.0
    pages = -(-tokens // page) + 3
    cache = new_cache(fp4, pages, heads, page, dim, fmt, hk)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:tokens]
    fp4.kv_append(cache, k.cuda(), v.cuda(), slots.cuda(), round=tie, mx_scale_rule=rule)
    kb, vb = fp4.kv_gather(cache, slots.cuda(), out_dtype=fp4.FP4_OUT_F32)
    kh, vh = fp4.kv_gather(cache, slots.cuda(), out_dtype=fp4.FP4_OUT_BF16)
    held = np.zeros(pages * page, bool)
    held[slots.numpy()] = True
    for x, (q, s, _), g, back, half in ((k, cache.k, GK, kb, kh), (v, cache.v, GV, vb, vh)):
        oq, os_, ob = oracle_rows(orc, x, fmt, hk, tie, rule, g)
        q = q.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, heads, -1)
        s = s.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, heads, -1)
        assert np.array_equal(q[slots.numpy()], oq)
        assert np.array_equal(s[slots.numpy()], os_)
        assert (q[~held] == 0x5A).all() and (s[~held] == 0x5A).all()  # nothing else is touched
        assert np.array_equal(back.cpu().numpy().view(np.uint32), ob.view(np.uint32))
        assert torch.equal(half.cpu(), torch.from_numpy(ob).to(torch.bfloat16))


@pytest.mark.parametrize("fmt,dim", [(MX, 128), (NV, 64), (MX16, 256)])
def test_strided_inputs(fp4, orc, fmt, dim):
    """Keys and values as views of one fused projection, and one shared head."""
    import torch
    T, H = 23, 4
    qkv = draw((T, 3 * H, dim), 5).cuda()
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:2 * H + 1].expand(T, H, dim)
    assert k.stride(0) != H * dim and v.stride(1) == 0
    cache = fp4.KVCache.empty(2, H, 32, dim, fmt, GK, GV)
    slots = torch.arange(T, device="cuda")
    fp4.kv_append(cache, k, v, slots)
    for got, x, g in zip(fp4.kv_gather(cache, slots, out_dtype=fp4.FP4_OUT_F32), (k, v), (GK, GV)):
        assert np.array_equal(got.cpu().numpy(), oracle_rows(orc, x.cpu().contiguous(), fmt, 0, 0, 0, g)[2])


@pytest.mark.parametrize("offset,pad", [(8, 0), (0, 8), (16, 16)])
def test_alignment_of_rows(fp4, orc, offset, pad):
    """Rows at 16 and at 32 bytes: both widths of load."""
    import torch
    T, H, D = 11, 3, 64
    buf = draw((T * (H * D + pad) + offset,), 6).cuda()
    k = buf[offset:].as_strided((T, H, D), (H * D + pad, D, 1))
    assert k.data_ptr() % 32 == (16 if offset == 8 else 0)
    cache = fp4.KVCache.empty(1, H, 16, D, MX)
    slots = torch.arange(T, device="cuda")
    fp4.kv_append(cache, k, k, slots)
    got = fp4.kv_gather(cache, slots, out_dtype=fp4.FP4_OUT_F32)
    want = oracle_rows(orc, k.cpu().contiguous(), MX, 0, 0, 0, 1.0)[2]
    assert np.array_equal(got[0].cpu().numpy(), want) and np.array_equal(got[1].cpu().numpy(), want)


def test_many_tokens(fp4, orc):
    """Enough for K and V to share their threads (one grid row)."""
    import torch
    T, H, D = 5003, 4, 128
    k, v = draw((T, H, D), 14), draw((T, H, D), 15)
    cache = fp4.KVCache.empty(-(-T // 64), H, 64, D, NV, GK, GV, 64)
    slots = torch.randperm(cache.num_pages * 64, generator=torch.Generator().manual_seed(16))[:T].cuda()
    fp4.kv_append(cache, k.cuda(), v.cuda(), slots)
    for got, x, g in zip(fp4.kv_gather(cache, slots, out_dtype=fp4.FP4_OUT_F32), (k, v), (GK, GV)):
        assert np.array_equal(got.cpu().numpy(), oracle_rows(orc, x, NV, 64, 0, 0, g)[2])


def test_slots_outside_are_dropped_and_read_as_zeros(fp4):
    import torch
    cache = new_cache(fp4, 2, 2, 16, 64, NV, 16)
    before = [t.clone() for t in (*cache.k, *cache.v)]
    bad = torch.tensor([-1, 32, -(1 << 62), (1 << 62), 33], device="cuda")
    x = draw((5, 2, 64), 7).cuda()
    fp4.kv_append(cache, x, x, bad)
    assert all(torch.equal(a, b) for a, b in zip(before, (*cache.k, *cache.v)))
    out = tuple(torch.full((5, 2, 64), 9.0, device="cuda") for _ in range(2))
    k, v = fp4.kv_gather(cache, bad, out_dtype=fp4.FP4_OUT_F32, out=out)
    assert k is out[0] and not k.any() and not v.any()


def test_gather_repeats_and_empty(fp4):
    import torch
    cache = fp4.KVCache.empty(1, 1, 16, 64, MX)
    x = draw((2, 1, 64), 9).cuda()
    fp4.kv_append(cache, x, x, torch.tensor([3, 8], device="cuda"))
    k, _ = fp4.kv_gather(cache, torch.tensor([8, 3, 8], device="cuda"))
    assert torch.equal(k[0], k[2]) and not torch.equal(k[0], k[1])
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    fp4.kv_append(cache, x[:0], x[:0], none)
    assert fp4.kv_gather(cache, none)[0].shape == (0, 1, 64)


def test_far_slots(fp4, orc):
    """Element offsets past 2^32: the last pages of a cache of over 4 GiB."""
    import torch
    pages, heads, page, dim = 40000, 8, 256, 128
    cache = fp4.KVCache.empty(pages, heads, page, dim, MX)
    assert cache.k[0].numel() > 1 << 32
    x = draw((3, heads, dim), 11)
    slots = torch.tensor([0, pages * page - 1, (pages - 1) * page], device="cuda")
    fp4.kv_append(cache, x.cuda(), x.cuda(), slots)
    oq, os_, ob = oracle_rows(orc, x, MX, 0, 0, 0, 1.0)
    assert np.array_equal(cache.v[0][-1, :, -1].cpu().numpy(), oq[1])
    assert np.array_equal(cache.k[1][-1, :, 0].cpu().numpy(), os_[2])
    k, v = fp4.kv_gather(cache, slots, out_dtype=fp4.FP4_OUT_F32)
    assert np.array_equal(k.cpu().numpy(), ob) and np.array_equal(v.cpu().numpy(), ob)


def test_side_stream_and_graph(fp4):
    """On a stream of its own, and captured and replayed with new inputs in place."""
    import torch
    cache = fp4.KVCache.empty(4, 2, 16, 128, NV, GK, GV)
    x, y = draw((6, 2, 128), 12).cuda(), draw((6, 2, 128), 13).cuda()
    slots = torch.arange(6, device="cuda") * 9
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        fp4.kv_append(cache, x, y, slots)
        first = fp4.kv_gather(cache, slots)
    st.synchronize()
    kin, vin, out = x.clone(), y.clone(), tuple(torch.empty_like(x) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fp4.kv_append(cache, kin, vin, slots)
        fp4.kv_gather(cache, slots, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    kin.copy_(y)
    vin.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    want = fp4.KVCache.empty(4, 2, 16, 128, NV, GK, GV)
    fp4.kv_append(want, y, x, slots)
    again = fp4.kv_gather(want, slots)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
