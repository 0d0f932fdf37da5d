"""CPU checks of the decode-time operators' host side: sizes, and every invalid
call refused before anything reaches a GPU."""
import ctypes

import pytest

from fp4_microscaling_quantization_b200 import _lib, build

F = 0x10000  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def cache(**kw):
    a = dict(kq=F, ks=F, vq=F, vs=F, gk=F, gv=F, num_pages=4, page_size=16, kv_heads=2, head_dim=128, fmt=1, hadamard_k=0)
    a.update(kw)
    return _lib.Fp4KvCache(*(a[n] for n, _ in _lib.Fp4KvCache._fields_))


BAD_CACHES = [
    (dict(kq=None), 1), (dict(ks=None), 1), (dict(vq=None), 1), (dict(vs=None), 1), (dict(gk=None), 1), (dict(gv=None), 1),
    (dict(num_pages=-1), 1), (dict(kv_heads=0), 1), (dict(kv_heads=65536), 2), (dict(num_pages=1 << 31), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=0), 2), (dict(page_size=512), 2),
    (dict(head_dim=96), 2), (dict(head_dim=32), 2), (dict(head_dim=0), 2), (dict(fmt=3), 2), (dict(fmt=-1), 2),
    (dict(hadamard_k=8), 2), (dict(hadamard_k=128, head_dim=64), 2),
    (dict(kq=F + 8), 3), (dict(ks=F + 2), 3), (dict(vq=F + 4), 3), (dict(vs=F + 1), 3), (dict(gk=F + 2), 3),
]


def append(L, c, **kw):
    a = dict(k=F, kt=256, kh=128, v=F, vt=256, vh=128, slots=F, tokens=3, opts=None)
    a.update(kw)
    return L.fp4_kv_append(ctypes.byref(c) if c else None, a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["slots"],
                           a["tokens"], a["opts"], None)


def gather(L, c, **kw):
    a = dict(slots=F, tokens=3, out=1, k=F, v=F)
    a.update(kw)
    return L.fp4_kv_gather(ctypes.byref(c) if c else None, a["slots"], a["tokens"], a["out"], a["k"], a["v"], None)


def attend(L, c, **kw):
    a = dict(q=F, batch=2, heads=4, qb=512, qh=128, table=F, ts=8, cols=8, lens=F, max=128, scale=0.1, window=0, out=1, o=F,
             lse=None, ws=None, wb=0)
    a.update(kw)
    return L.fp4_paged_attention(ctypes.byref(c) if c else None, a["q"], a["batch"], a["heads"], a["qb"], a["qh"], a["table"],
                                 a["ts"], a["cols"], a["lens"], a["max"], a["scale"], a["window"], a["out"], a["o"], a["lse"],
                                 a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(L, kw, code):
    c = cache(**kw)
    assert append(L, c) == code and gather(L, c) == code
    assert attend(L, c) == code


def test_null_cache(L):
    assert append(L, None) == 1 and gather(L, None) == 1 and attend(L, None) == 1


def test_tensor_scales_only_for_nvfp4(L):
    c = cache(fmt=0, gk=None, gv=None)
    assert append(L, c, tokens=0) == 0 and gather(L, c, tokens=0) == 0 and attend(L, c, batch=0) == 0


def test_cache_sizes(L):
    q, s = ctypes.c_size_t(), ctypes.c_size_t()
    p = ctypes.byref(q), ctypes.byref(s)
    assert L.fp4_kv_cache_sizes(10, 16, 8, 128, 1, *p) == 0
    assert q.value == 10 * 16 * 8 * 64 and s.value == 10 * 16 * 8 * 8
    assert L.fp4_kv_cache_sizes(10, 64, 3, 64, 0, *p) == 0 and s.value == 10 * 64 * 3 * 2
    assert L.fp4_kv_cache_sizes(0, 64, 3, 64, 2, *p) == 0 and q.value == 0
    assert L.fp4_kv_cache_sizes(1 << 20, 256, 8, 256, 2, *p) == 0 and q.value == (1 << 20) * 256 * 8 * 128
    assert L.fp4_kv_cache_sizes(1 << 21, 256, 8, 256, 2, *p) == 2  # 2^32 rows
    assert L.fp4_kv_cache_sizes(10, 24, 8, 128, 1, *p) == 2
    assert L.fp4_kv_cache_sizes(10, 16, 8, 100, 1, *p) == 2
    assert L.fp4_kv_cache_sizes(10, 16, 8, 128, 1, None, ctypes.byref(s)) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(tokens=-1), 1), (dict(kt=-8), 1), (dict(vh=-8), 1),
    (dict(k=F + 8), 3), (dict(v=F + 2), 3), (dict(kt=260), 3), (dict(vh=4), 3), (dict(slots=F + 4), 3),
    (dict(tokens=1 << 40), 2), (dict(tokens=0), 0),
])
def test_append_refuses(L, kw, code):
    assert append(L, cache(), **kw) == code


def test_append_options(L):
    for o, code in ((_lib.Fp4Opts(2), 1), (_lib.Fp4Opts(0, 2), 1), (_lib.Fp4Opts(0, 0, 0, _lib.FP4_SCALE_MSE), 2)):
        assert append(L, cache(), opts=ctypes.byref(o)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(slots=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(tokens=-1), 1), (dict(out=2), 1), (dict(k=F + 16), 3),
    (dict(v=F + 8), 3), (dict(slots=F + 2), 3), (dict(tokens=1 << 40), 2), (dict(tokens=0), 0),
])
def test_gather_refuses(L, kw, code):
    assert gather(L, cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(batch=-1), 1),
    (dict(batch=65536), 2), (dict(heads=3), 1), (dict(heads=0), 1), (dict(heads=65536), 2), (dict(max=0), 1),
    (dict(max=(1 << 30) + 1), 2), (dict(window=-1), 1), (dict(out=7), 1), (dict(qb=-8), 1), (dict(qh=100), 3),
    (dict(qb=4), 3), (dict(q=F + 8), 3), (dict(o=F + 8), 3), (dict(lens=F + 2), 3), (dict(table=F + 1), 3),
    (dict(lse=F + 2), 3), (dict(ts=-1), 1), (dict(cols=-1), 1), (dict(cols=(1 << 30) + 1), 2),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(batch=0), 0),
    (dict(max=1 << 20), 1), (dict(max=1 << 20, ws=F, wb=64), 1), (dict(max=1 << 20, ws=F + 4, wb=1 << 40), 3),
])
def test_attention_refuses(L, kw, code):
    assert attend(L, cache(), **kw) == code


def test_attention_workspace(L):
    b = ctypes.c_size_t()
    size = L.fp4_paged_attention_workspace_size
    assert size(4, 32, 8, 128, 100, 0, ctypes.byref(b)) == 0 and b.value == 0
    assert size(1, 32, 8, 128, 1 << 17, 0, ctypes.byref(b)) == 0 and b.value > 0
    long = b.value
    assert size(1, 32, 8, 128, 1 << 17, 128, ctypes.byref(b)) == 0 and b.value < long  # a window bounds the work
    assert size(1, 32, 8, 128, 1 << 30, 0, ctypes.byref(b)) == 0  # the number of chunks is bounded
    assert b.value <= 32 * 1024 * 130 * 4
    assert size(0, 32, 8, 128, 1 << 17, 0, ctypes.byref(b)) == 0 and b.value == 0
    assert size(1, 30, 8, 128, 100, 0, ctypes.byref(b)) == 1
    assert size(1, 32, 8, 80, 100, 0, ctypes.byref(b)) == 2
    assert size(1, 32, 8, 128, 100, 0, None) == 1


def linear(L, **kw):
    a = dict(x=F, M=4, K=256, ldx=256, fmt=1, hk=0, opts=None, wq=F, ws=F, gw=F, N=64, out=1, c=F, ldc=64, wsp=None, wsb=0)
    a.update(kw)
    return L.fp4_linear_w4a16(a["x"], a["M"], a["K"], a["ldx"], a["fmt"], a["hk"], a["opts"], a["wq"], a["ws"], a["gw"],
                              a["N"], a["out"], a["c"], a["ldc"], a["wsp"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=17), 2), (dict(M=-1), 1), (dict(K=100), 2), (dict(K=0, ldx=0), 2), (dict(ldx=128), 1), (dict(ldc=8), 1),
    (dict(fmt=4), 2), (dict(hk=48), 2), (dict(hk=128, K=320, ldx=320), 2), (dict(out=3), 1), (dict(x=None), 1),
    (dict(wq=None), 1), (dict(ws=None), 1), (dict(c=None), 1), (dict(gw=None), 1), (dict(x=F + 8), 3), (dict(ldx=260), 3),
    (dict(wq=F + 8), 3), (dict(ws=F + 4), 3), (dict(c=F + 4), 3), (dict(gw=F + 2), 3),
    (dict(M=16, N=28672, K=8192, ldx=8192, ldc=28672), 1),
    (dict(M=16, N=28672, K=8192, ldx=8192, ldc=28672, wsp=F, wsb=64), 1),
    (dict(M=16, N=28672, K=8192, ldx=8192, ldc=28672, wsp=F + 16, wsb=1 << 40), 3),
    (dict(N=(1 << 30) + 1, ldc=1 << 31), 2), (dict(K=1 << 31, ldx=1 << 31), 2), (dict(M=0), 0), (dict(N=0, ldc=0), 0),
])
def test_linear_refuses(L, kw, code):
    assert linear(L, **kw) == code


def test_linear_workspace(L):
    b = ctypes.c_size_t()
    size = L.fp4_linear_w4a16_workspace_size
    assert size(16, 28672, 8192, 1, ctypes.byref(b)) == 0 and b.value >= 16 * 8192 * 2
    assert size(1, 1024, 4096, 1, ctypes.byref(b)) == 0 and b.value == 0
    assert size(0, 4096, 4096, 1, ctypes.byref(b)) == 0 and b.value == 0
    assert size(17, 4096, 4096, 1, ctypes.byref(b)) == 2
    assert size(1, 4096, 4096, 3, ctypes.byref(b)) == 2
    assert size(-1, 4096, 4096, 1, ctypes.byref(b)) == 1
    assert size(1, 4096, 4096, 1, None) == 1


def test_linear_options(L):
    assert linear(L, opts=ctypes.byref(_lib.Fp4Opts(0, 0, 0, 0, 2))) == 1


def test_binding_refuses_host_tensors_and_shapes():
    import torch
    import fp4_microscaling_quantization_b200 as fp4
    q = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((4, 2, 16, 8), dtype=torch.uint8)
    g = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fp4.KVCache((q, s, g), (q, s, g), fp4.FP4_NVFP4)
    with pytest.raises(ValueError, match="num_pages, kv_heads"):
        fp4.KVCache((q[0], s, g), (q, s, g), fp4.FP4_NVFP4)
    with pytest.raises(fp4.Fp4Error):
        fp4.KVCache((q[:, :, :9], s, g), (q, s, g), fp4.FP4_NVFP4)
    with pytest.raises(fp4.Fp4Error):
        fp4.KVCache.empty(4, 2, 16, 80, fp4.FP4_MXFP4, device="cpu")
    assert fp4.kv_cache_sizes(4, 16, 2, 128, "nvfp4") == (q.numel(), s.numel())
    with pytest.raises(ValueError):
        fp4.linear_w4a16(torch.zeros((2, 64), dtype=torch.bfloat16), (q, s, g), fp4.FP4_NVFP4)
    assert fp4.paged_attention_workspace_size(1, 8, 8, 64, 64) == 0


def test_streams_without_the_private_call():
    """A torch that lacks the raw stream call is asked by the public one; one
    that has it, without making a stream object."""
    from types import SimpleNamespace
    import torch
    import fp4_microscaling_quantization_b200 as fp4
    asked = []

    def public(device):
        asked.append(device)
        return SimpleNamespace(cuda_stream=77)

    without = SimpleNamespace(_C=SimpleNamespace(), cuda=SimpleNamespace(current_stream=public))
    assert fp4._stream_handle(without, torch.device("cuda", 3)) == 77 and fp4._stream_handle(without, 1) == 77
    assert asked == [3, 1]
    having = SimpleNamespace(_C=SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 100 + index), cuda=None)
    assert fp4._stream_handle(having, torch.device("cuda", 3)) == 103 and fp4._stream_handle(having, 2) == 102


def test_calls_ask_for_the_device_by_the_public_call(monkeypatch):
    """An entry point of a device that is current runs without changing it; of
    another device, with that one current."""
    from contextlib import contextmanager
    from types import SimpleNamespace
    import torch
    import fp4_microscaling_quantization_b200 as fp4
    made, inside = [], []

    @contextmanager
    def device(d):
        inside.append(d.index)
        yield

    fake = SimpleNamespace(fp4_kv_gather=lambda *a: made.append(a) or 0)
    monkeypatch.setattr(fp4._lib, "_lib", fake)
    monkeypatch.setattr(fp4._lib, "lib", lambda: fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1 / 0, raising=False)
    fp4._run("fp4_kv_gather", torch.device("cuda", 1), 5)
    assert made == [(5,)] and not inside
    fp4._run("fp4_kv_gather", torch.device("cuda", 0), 6)
    assert made == [(5,), (6,)] and inside == [0]
