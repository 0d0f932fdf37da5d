"""Decode-time operators of a served language model on FP4 data: what is measured.

The four operators, each with its plain form here:
  write_read  new keys and values quantised into a paged FP4 cache as they arrive, and read back
  read        tokens of the cache read back by their slots
  attend      attention of one new token per sequence over the paged FP4 cache
  linear      a weight-only linear layer: FP4 weights with block scales, bf16 activations that stay bf16

Formats (E2M1 elements, two to a byte, the even index in the low nibble): "mx" has one power-of-two byte per 32
elements, "mx16" one per 16, "nv" one E4M3 byte per 16 and one fp32 scale for the tensor.  A cache holds, for each of
K and V, elements (pages, kv_heads, page, head_dim / 2) and scales (pages, kv_heads, page, head_dim / block); a slot is
page * page_size + position.  Weights have their scales in 512-byte tiles of 128 rows x 4 scales.
"""
import math

import torch

own = False

FMT = {"mx": 0, "nv": 1, "mx16": 2}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 61 sequences: its new keys and values go in, and come back (latency)
        dict(name="write_read_step", op="write_read", tokens=61, heads=8, dim=128, page=16, fmt="nv", rot=0, out="bf16"),
        # a long prompt's keys and values, rotated before they are quantised, read back for the prompt's next chunk
        dict(name="write_read_prompt", op="write_read", tokens=32749, heads=8, dim=128, page=64, fmt="mx", rot=64, out="bf16"),
        # a short shared prefix read back
        dict(name="read_prefix", op="read", tokens=1000, heads=8, dim=64, page=16, fmt="mx", rot=0, out="f32"),
        # the caches of a batch read back (a move to another machine, a prompt that continues)
        dict(name="read_batch", op="read", tokens=100003, heads=8, dim=128, page=16, fmt="nv", rot=0, out="bf16"),
        # one sequence that has just begun: all of it is latency
        dict(name="attend_short", op="attend", batch=1, q_heads=32, heads=8, dim=128, page=16, fmt="nv", rot=0, length=129, ragged=False, out="bf16"),
        # a full decode batch of uneven lengths, eight query heads to a key head
        dict(name="attend_batch", op="attend", batch=64, q_heads=64, heads=8, dim=128, page=16, fmt="nv", rot=0, length=8192, ragged=True, out="bf16"),
        # one very long document
        dict(name="attend_long", op="attend", batch=1, q_heads=32, heads=8, dim=128, page=64, fmt="mx", rot=0, length=262143, ragged=False, out="bf16"),
        # short heads, rotated cache
        dict(name="attend_d64", op="attend", batch=32, q_heads=64, heads=8, dim=64, page=32, fmt="mx", rot=64, length=8191, ragged=False, out="bf16"),
        # the smallest product of a decode step
        dict(name="linear_kv_proj", op="linear", m=1, n=1024, k=4096, fmt="nv", rot=0, out="bf16"),
        # the two projections of a feed-forward layer in a small batch
        dict(name="linear_up", op="linear", m=4, n=14336, k=4096, fmt="mx", rot=0, out="bf16"),
        dict(name="linear_down", op="linear", m=16, n=4096, k=14336, fmt="nv", rot=128, out="bf16"),
        # a large layer for one token
        dict(name="linear_large", op="linear", m=1, n=28672, k=8192, fmt="nv", rot=0, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write_read", "read", "attend", "attend", "linear", "linear"])
    fmt = rng.choice(["mx", "nv", "mx16"])
    if op == "linear":
        while True:
            n, k = _log(rng, 256, 28672), 32 * _log(rng, 8, 448)
            if n * k <= 28672 * 8192:
                break
        rot = rng.choice([0, 0] + [r for r in (16, 32, 64, 128) if k % r == 0])
        return dict(op=op, m=rng.randint(1, 16), n=n, k=k, fmt=fmt, rot=rot, out=rng.choice(["bf16", "f32"]))
    dim, page, heads = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    rot = rng.choice([0, 0] + [r for r in (16, 32, 64, 128) if dim % r == 0])
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        batch = _log(rng, 1, 64)
        length = _log(rng, 1, min(262143, 2097152 // (batch * heads * dim // 128 + 1)))
        return dict(op=op, batch=batch, q_heads=group * heads, heads=heads, dim=dim, page=page, fmt=fmt, rot=rot, length=length,
                    ragged=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    tokens = _log(rng, 1, 32749 * 1024 // (heads * dim))
    return dict(op=op, tokens=tokens, heads=heads, dim=dim, page=page, fmt=fmt, rot=rot, out="bf16" if rot else rng.choice(["bf16", "f32"]))


def _block(fmt):
    return 32 if fmt == "mx" else 16


def _lengths(case):
    """The batch's lengths: all alike, or spread evenly over 1 .. length in a mixed order."""
    b, n = case["batch"], case["length"]
    return [1 + int((n - 1) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(b)] if case["ragged"] else [n] * b


def work(case):
    size = 4 if case["out"] == "f32" else 2
    per = 0.5 + 1 / _block(case["fmt"])  # bytes of a quantised element
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * per + m * k * 2 + m * n * size, "flops": 2 * m * n * k}
    row = case["heads"] * case["dim"]
    if case["op"] == "attend":
        total, q = sum(_lengths(case)), case["batch"] * case["q_heads"] * case["dim"]
        return {"bytes": 2 * total * row * per + q * (2 + size), "flops": 4 * total * case["q_heads"] * case["dim"]}
    n = 2 * case["tokens"] * row
    turn = 2 * max(1, int(math.log2(case["rot"]))) if case["rot"] else 0
    if case["op"] == "read":
        return {"bytes": n * (per + size) + 8 * case["tokens"], "flops": n * (1 + turn / 2)}
    return {"bytes": n * (2 + per + size) + 8 * case["tokens"], "flops": n * (4 + turn)}


# ---- the formats, in 32 bits ---------------------------------------------------------------------------------------
def _rotate(x, k):
    """The normalised Sylvester transform of every k consecutive values: stages 1, 2, .. k/2, then times 1/sqrt(k)."""
    shape, h = x.shape, 1
    while h < k:
        x = x.reshape(-1, 2, h)
        x = torch.stack((x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]), 1)
        h *= 2
    x = x.reshape(shape)
    return x * torch.tensor(1.0 / math.sqrt(k), dtype=torch.float32, device=x.device) if k else x


def _codes(v):
    """Nearest E2M1 codes, midpoints to the even code; -0 and negatives that round to 0 keep their sign."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    for mid, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += a >= mid if up else a > mid
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _quantise(x, fmt, g):
    """(elements, scales) of x (..., n) in 32 bits, blocks along the last axis; no element of a power-of-two block clips."""
    b = x.reshape(*x.shape[:-1], -1, _block(fmt))
    amax = b.abs().amax(-1)
    if fmt == "nv":
        s = (amax / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = g * s.to(torch.float32)
        r = torch.where(d == 0, torch.zeros_like(d), (1.0 / d).clamp(max=torch.finfo(torch.float32).max))
        scales = s.view(torch.uint8)
    else:
        m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1): 6 * 2^(e - 3) is 0.75 * 2^e
        e = torch.where(amax == 0, torch.full_like(e, -127), (e - 3 + (m > 0.75)).clamp(-127, 127))
        r = torch.ldexp(torch.ones_like(amax), -e)
        scales = (e + 127).to(torch.uint8)
    c = _codes(b * r[..., None]).reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), scales


def _values(q, scales, fmt, g):
    """What elements and scales stand for: RN(RN(s_g * s_b) * q)."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float32, device=q.device)
    v = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), -1)
    if fmt == "nv":
        s = g * scales.view(torch.float8_e4m3fn).to(torch.float32)
    else:
        s = torch.ldexp(torch.ones(scales.shape, dtype=torch.float32, device=q.device), scales.int() - 127)
    return (v.reshape(*scales.shape, _block(fmt)) * s[..., None]).reshape(*q.shape[:-1], -1)


def _tiles(rows, cols, device):
    """Where scale (r, c) of a rows x cols weight lies: 512-byte tiles of 128 rows x 4 scales."""
    r = torch.arange(rows, device=device)[:, None]
    c = torch.arange(cols, device=device)[None, :]
    return ((r // 128) * ((cols + 3) // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


# ---- inputs --------------------------------------------------------------------------------------------------------
def _activations(gen, *shape):
    """Normal values in which one channel of 64 is eight times the others."""
    x = torch.randn(*shape, generator=gen, device=DEV)
    loud = torch.rand(shape[-1], generator=gen, device=DEV) < 1 / 64
    return (x * torch.where(loud, 8.0, 1.0)).to(torch.bfloat16)


def _new_cache(case, pages, gen, filled):
    """kq, ks, vq, vs of a cache, written as a prompt would have left it, or empty."""
    shape, b = (pages, case["heads"], case["page"]), _block(case["fmt"])
    c = {"kg": torch.full((1,), 0.037, device=DEV), "vg": torch.full((1,), 0.011, device=DEV)}
    for n in "kv":
        if filled:
            c[n + "q"], c[n + "s"] = _quantise(_rotate(_activations(gen, *shape, case["dim"]).float(), case["rot"]), case["fmt"], c[n + "g"])
        else:
            c[n + "q"] = torch.zeros(*shape, case["dim"] // 2, dtype=torch.uint8, device=DEV)
            c[n + "s"] = torch.zeros(*shape, case["dim"] // b, dtype=torch.uint8, device=DEV)
    return c


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "linear":
        n, k, fmt = case["n"], case["k"], case["fmt"]
        w = _rotate((torch.randn(n, k, generator=gen, device=DEV) * 0.02).to(torch.bfloat16).float(), case["rot"])
        s["g"] = (w.abs().amax() / 2688.0).reshape(1) if fmt == "nv" else torch.ones(1, device=DEV)
        s["q"], scales = _quantise(w, fmt, s["g"])
        cols = k // _block(fmt)
        s["s"] = torch.zeros((n + 127) // 128 * 128 * ((cols + 3) // 4 * 4), dtype=torch.uint8, device=DEV)
        s["s"][_tiles(n, cols, DEV)] = scales
        s["x"] = _activations(gen, case["m"], k)
        return s
    p, heads, dim = case["page"], case["heads"], case["dim"]
    if case["op"] == "attend":
        need = [-(-n // p) for n in _lengths(case)]
        pages = sum(need) + 1
        s["cache"] = _new_cache(case, pages, gen, True)
        order = torch.randperm(pages, generator=gen, device=DEV).int()
        first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)[:, None]
        cols = torch.arange(max(need), device=DEV)[None, :]
        held = cols < torch.tensor(need, device=DEV)[:, None]
        s["table"] = torch.where(held, order[torch.where(held, first + cols, 0)], 0).int().contiguous()
        s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
        s["query"] = (torch.randn(case["batch"], case["q_heads"], dim, generator=gen, device=DEV) * 0.5).to(torch.bfloat16)
        return s
    n = case["tokens"]
    pages = -(-n // p) + 2
    s["cache"] = _new_cache(case, pages, gen, case["op"] == "read")
    order = torch.randperm(pages, generator=gen, device=DEV)
    at = torch.arange(n, device=DEV)
    # a prompt's tokens fill pages one after another; a decode step's go to a page of their own each while there are enough
    s["slots"] = order[at // p] * p + at % p if n > 256 else torch.randperm(pages * p, generator=gen, device=DEV)[:n]
    if case["op"] == "write_read":
        s["k"], s["v"] = _activations(gen, n, heads, dim), _activations(gen, n, heads, dim)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _dtype(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def _run_plain(s):
    case, fmt = s["case"], s["case"]["fmt"]
    op, rot = case["op"], case["rot"]
    if op == "linear":
        scales = s["s"][_tiles(case["n"], case["k"] // _block(fmt), DEV)]
        return (_rotate(s["x"].float(), rot) @ _values(s["q"], scales, fmt, s["g"]).T).to(_dtype(case))
    c, p = s["cache"], case["page"]
    if op == "attend":
        t, groups = s["table"].shape[1] * p, case["q_heads"] // case["heads"]
        k, v = (_values(c[n + "q"][s["table"].long()], c[n + "s"][s["table"].long()], fmt, c[n + "g"]).transpose(1, 2)
                .reshape(case["batch"], case["heads"], t, case["dim"]) for n in "kv")
        q = _rotate(s["query"].float(), rot).reshape(case["batch"], case["heads"], groups, case["dim"])
        x = (q @ k.transpose(-1, -2)) / math.sqrt(case["dim"])
        x = x.masked_fill(torch.arange(t, device=DEV) >= s["lens"][:, None, None, None], -math.inf)
        w = (x - x.amax(-1, keepdim=True)).exp()
        o = _rotate((w @ v) / w.sum(-1, keepdim=True), rot)
        return o.reshape(case["batch"], case["q_heads"], case["dim"]).to(_dtype(case))
    page, pos = s["slots"] // p, s["slots"] % p
    if op == "write_read":
        for n in "kv":
            c[n + "q"][page, :, pos], c[n + "s"][page, :, pos] = _quantise(_rotate(s[n].float(), rot), fmt, c[n + "g"])
    k, v = (_rotate(_values(c[n + "q"][page, :, pos], c[n + "s"][page, :, pos], fmt, c[n + "g"]), rot).to(_dtype(case)) for n in "kv")
    return {"k": k, "v": v}


def _run_own(s):
    import fp4_microscaling_quantization_b200 as fp4

    case = s["case"]
    out = fp4.FP4_OUT_F32 if case["out"] == "f32" else fp4.FP4_OUT_BF16
    fmt = FMT[case["fmt"]]
    if case["op"] == "linear":
        return fp4.linear_w4a16(s["x"], (s["q"], s["s"], s["g"]), fmt, hadamard_k=case["rot"], out_dtype=out)
    if "handle" not in s:
        c = s["cache"]
        s["handle"] = fp4.KVCache((c["kq"], c["ks"], c["kg"]), (c["vq"], c["vs"], c["vg"]), fmt, hadamard_k=case["rot"])
    cache = s["handle"]
    if case["op"] == "attend":
        return fp4.paged_attention(s["query"], cache, s["table"], s["lens"], max_seq_len=case["length"], out_dtype=out)
    if case["op"] == "write_read":
        fp4.kv_append(cache, s["k"], s["v"], s["slots"])
    k, v = fp4.kv_gather(cache, s["slots"], out_dtype=out)
    return {"k": k, "v": v}


# ---- from the definitions, in 64 bits ------------------------------------------------------------------------------
def _hadamard64(k):
    """H_k with entries (-1)^popcount(i & j) / sqrt(k)."""
    i = torch.arange(k)
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> j) & 1 for j in range(8)) % 2
    return ((1 - 2 * odd).double() / math.sqrt(k)).to(DEV)


def _turn64(x, k):
    return (x.reshape(-1, k) @ _hadamard64(k)).reshape(x.shape) if k else x


def _nearest64(a):
    """Nearest of the E2M1 magnitudes to a >= 0, halfway cases to the even code."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=a.device)
    hi = torch.bucketize(a.clamp(max=6.0), grid).clamp(1, 7)
    up, down = grid[hi] - a, a - grid[hi - 1]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take_hi, grid[hi], grid[hi - 1])


def _rounded64(x, fmt, g):
    """x after quantisation and back.  A block's scale is rounded in 32 bits before its 8, as the format's definition has it."""
    b = x.reshape(*x.shape[:-1], -1, _block(fmt))
    amax = b.abs().amax(-1)
    if fmt == "nv":
        six = (6.0 * g.double()).float().double()
        s = ((amax.float().double() / six).float().clamp(max=448.0)).to(torch.float8_e4m3fn).double() * g.double()
    else:
        s = torch.exp2(torch.where(amax == 0, torch.full_like(amax, -127.0), torch.ceil(torch.log2(amax / 6.0))).clamp(-127, 127))
    y = torch.where(s[..., None] == 0, torch.zeros_like(b), _nearest64((b / torch.where(s == 0, 1.0, s)[..., None]).abs()) * s[..., None])
    return torch.copysign(y, b).reshape(x.shape)


def _read64(q, scales, fmt, g):
    both = torch.stack((q % 16, q // 16), -1).reshape(*q.shape[:-1], -1)
    grid = torch.tensor(GRID, dtype=torch.float64, device=q.device)
    v = grid[(both % 8).long()] * (1.0 - 2.0 * (both // 8).double())
    s = scales.view(torch.float8_e4m3fn).double() * g.double() if fmt == "nv" else torch.exp2(scales.double() - 127.0)
    return v * s.repeat_interleave(_block(fmt), -1)


def exact(case, seed):
    s, fmt, rot = prepare(case, seed), case["fmt"], case["rot"]
    if case["op"] == "linear":
        cols, step, parts = case["k"] // _block(fmt), 4096, []
        x, at = _turn64(s["x"].double(), rot), _tiles(case["n"], cols, DEV)
        for i in range(0, case["n"], step):
            parts.append(x @ _read64(s["q"][i:i + step], s["s"][at[i:i + step]], fmt, s["g"]).T)
        return torch.cat(parts, 1)
    c, p = s["cache"], case["page"]
    if case["op"] == "attend":
        rows, groups = [], case["q_heads"] // case["heads"]
        for b, n in enumerate(_lengths(case)):
            pages = s["table"][b, : -(-n // p)].long()
            q = _turn64(s["query"][b].double(), rot).reshape(case["heads"], groups, -1)
            heads = []
            for h in range(case["heads"]):
                k, v = (_read64(c[i + "q"][pages, h], c[i + "s"][pages, h], fmt, c[i + "g"]).reshape(-1, case["dim"])[:n] for i in "kv")
                heads.append(torch.softmax(q[h] @ k.T / math.sqrt(case["dim"]), -1) @ v)
            rows.append(_turn64(torch.cat(heads), rot))
        return torch.stack(rows)
    page, pos = s["slots"] // p, s["slots"] % p
    if case["op"] == "write_read":
        return {n: _turn64(_rounded64(_turn64(s[n].double(), rot), fmt, c[n + "g"]), rot) for n in "kv"}
    return {n: _turn64(_read64(c[n + "q"][page, :, pos], c[n + "s"][page, :, pos], fmt, c[n + "g"]), rot) for n in "kv"}
