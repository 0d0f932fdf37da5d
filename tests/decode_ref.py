"""Plain 64-bit references of the decode-time operators, and the bounds their
tests hold results to.  Written from the formulas; nothing of the library is
used.

Roundings counted below (half a step each): bf16 2^-8, f16 2^-11, fp32 2^-24.
A tensor-core sum of n products of 16-bit operands adds n / 16 times into an
fp32 accumulator, each time with an error of at most 2^-22 of the sum of the
terms' magnitudes (the products are exact; the additions of one instruction
may drop the bits below the accumulator's last).
"""
import math

import torch

MX, NV, MX16 = 0, 1, 2
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def block_of(fmt):
    return 32 if fmt == MX else 16


def values64(q, s, fmt, g=1.0):
    """What packed nibbles (..., n / 2) and row-wise scales (..., n / block) stand for."""
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=q.device)
    v = torch.stack((grid[(q & 15).long()], grid[(q >> 4).long()]), -1).reshape(*q.shape[:-1], -1)
    if fmt == NV:
        d = s.view(torch.float8_e4m3fn).double() * float(g)
    else:
        d = torch.exp2(s.double() - 127.0)
        d = torch.where(s == 255, torch.full_like(d, math.nan), d)
    return v * d.repeat_interleave(block_of(fmt), -1)


def hadamard64(k, device="cpu"):
    i = torch.arange(k)
    b = i[:, None] & i[None, :]
    odd = sum((b >> j) & 1 for j in range(8)) % 2
    return ((1 - 2 * odd).double() / math.sqrt(k)).to(device)


def rotate64(x, k):
    return (x.reshape(*x.shape[:-1], -1, k) @ hadamard64(k, x.device)).reshape(x.shape) if k else x


def spread64(x, k):
    """sum_j |H_ij| x_j of non-negative x: how far a bound on rotated values reaches."""
    if not k:
        return x
    t = x.reshape(*x.shape[:-1], -1, k).sum(-1, keepdim=True) / math.sqrt(k)
    return t.expand(*t.shape[:-1], k).reshape(x.shape)


def atoms_index(rows, nkb, device="cpu"):
    """Place of scale (r, kb) in the tile layout."""
    r = torch.arange(rows, device=device)[:, None]
    c = torch.arange(nkb, device=device)[None, :]
    return ((r // 128) * ((nkb + 3) // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


def attention64(q, kq, ks, vq, vs, fmt, gk, gv, hk, table, lens, page, scale, window, num_pages):
    """(out, lse, bound on |out|'s fp32 error, sum of w |v|) of attention over a
    paged cache, sequence by sequence, head by head."""
    B, HQ, D = q.shape
    H = kq.shape[1]
    out = torch.zeros(B, HQ, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, HQ), -math.inf, dtype=torch.float64, device=q.device)
    err, mag = torch.zeros_like(out), torch.zeros_like(out)
    qr = rotate64(q.double(), hk)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        t = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        if not len(t):
            continue
        pages = table[b].long()[t // page]
        ok = (pages >= 0) & (pages < num_pages)
        t, pages = t[ok], pages[ok]
        if not len(t):
            continue
        for h in range(H):
            k = values64(kq[pages, h, t % page], ks[pages, h, t % page], fmt, gk)
            v = values64(vq[pages, h, t % page], vs[pages, h, t % page], fmt, gv)
            rows = slice(h * (HQ // H), (h + 1) * (HQ // H))
            x = qr[b, rows] @ k.T * scale
            w = torch.softmax(x, -1)
            lse[b, rows] = torch.logsumexp(x, -1)
            o, a = w @ v, w @ v.abs()
            # scores: q in 22 bits, D / 16 additions, scale factors and their own rounding (|x| 2^-22)
            d = (D / 16 + 4) * 2.0**-22 * ((qr[b, rows].abs() @ k.abs().T * abs(scale)).amax(-1, keepdim=True))
            # weights: twice the scores' error (numerator and sum), ex2 and split (2^-21), len / 16 additions, joins
            e = a * (2 * d + (len(t) / 16 + 64) * 2.0**-22)
            # f16 weights, the largest at 2^15 or below it: under 2^-14 f16 has
            # steps of 2^-24, so a weight of any size is off by at most half
            # one, 2^-25, that is 2^-40 of the largest weight (the same for
            # the lo term of a split weight)
            e = e + 2.0**-40 * w.amax(-1, keepdim=True) * v.abs().sum(0)
            out[b, rows] = rotate64(o, hk)
            mag[b, rows] = spread64(a, hk)
            err[b, rows] = spread64(e, hk) + (8 * 2.0**-24) * spread64(a, hk)
    return out, lse, err, mag
