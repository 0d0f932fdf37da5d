// frag.cuh — FP4 operands of 16-bit tensor-core products: E2M1 bytes and
// block scales to f16 pairs, and the warp-level product itself.  Shared by
// the attention over the FP4 cache and the weight-only linear layer.
//
// E2M1 (2 significant bits) times an E4M3 scale (4) is exact in f16: 6 bits,
// 2^-10 .. 2688.  E8M0 scales reach far past f16, so they are taken relative
// to the largest of a row's part and the result is multiplied by that.
#pragma once

#include "encode.cuh"

namespace fp4 {

// Bytes of two E2M1 codes each -> f16 pairs (low nibble first).  The byte
// registers come from one unpacking move: a shift and mask per byte halves
// the rate (measured 21 against 42 conversions per clock and SM).
FP4_DEV void e2m1x8_to_f16(uint32_t w, uint32_t *h)
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

FP4_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

FP4_DEV uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

FP4_DEV uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

FP4_DEV void mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(e - ref + 8) in f16, twice in a register, for E8M0 bytes e <= ref.
// Scales more than 2^22 below the reference give zero.
FP4_DEV uint32_t e8m0_rel(uint32_t e, uint32_t ref)
{
    const int t = (int)e - (int)ref + 23;
    return (uint32_t)(t > 0 ? t : 0) * 0x04000400u;
}

// The largest byte of a in the lower half, of b in the upper.
FP4_DEV uint32_t max_bytes2(uint32_t a, uint32_t b)
{
    const uint32_t x = __vmaxu2(a & 0x00FF00FFu, (a >> 8) & 0x00FF00FFu), y = __vmaxu2(b & 0x00FF00FFu, (b >> 8) & 0x00FF00FFu);
    return __vmaxu2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
}

// E8M0 bytes in the halves of a word -> what they stand for, NaN for 0xFF.
FP4_DEV float2 e8m0x2_to_f32(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((unsigned short)__byte_perm(two, 0, 0x0020)));
    return make_float2(bf16lo(r), bf16hi(r));
}

// 2^e as a product of two factors, for any exponent that a product of two
// numbers can have: times one and then the other is exact, unless the result
// itself is subnormal or past the largest number.
FP4_DEV float2 exp2_pair(int e)
{
    const int e0 = max(-126, min(e, 127));
    return make_float2(exp2i(e0), exp2i(max(-126, min(e - e0, 127))));
}

// g = m 2^e with |m| in [1, 2): leaves m, returns e.  Zero, subnormal numbers,
// infinities and NaN stay whole (e = 0).
FP4_DEV int take_exponent(float &g)
{
    const uint32_t u = __float_as_uint(g), e = (u >> 23) & 0xFFu;
    if (e == 0 || e == 255) return 0;
    g = __uint_as_float((u & 0x807FFFFFu) | 0x3F800000u);
    return (int)e - 127;
}

// H_k of a unit of 32 values whose neighbours in the row are in neighbouring lanes.
FP4_DEV void rotate_unit(float *v, int hk, float ck, int lane)
{
    switch (hk) {
    case 16: fwht_unit<16>(v, ck, lane); break;
    case 32: fwht_unit<32>(v, ck, lane); break;
    case 64: fwht_unit<64>(v, ck, lane); break;
    case 128: fwht_unit<128>(v, ck, lane); break;
    default: break;
    }
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

}  // namespace fp4
