// kv.cuh — the paged FP4 key-value cache as the kernels see it, and what the
// cache kernels and the attention over the cache share.
//
// K and V each are two arrays: elements (pages, heads, page_size, dim / 2)
// bytes and scales (pages, heads, page_size, dim / block) bytes, so that the
// tokens of one head in one page are contiguous: what attention reads.  A
// slot is page * page_size + position.
#pragma once

#include "encode.cuh"

namespace fp4 {

struct KvView {
    uint8_t *kq, *ks, *vq, *vs;
    const float *gk, *gv;  // NVFP4 tensor scales (null for the E8M0 formats)
    int64_t num_pages;
    int page_shift;        // log2 page_size
    int heads;             // key-value heads
};

// Row (page, head, position) of a slot in the element and scale arrays.
FP4_DEV int64_t kv_row(int64_t slot, int head, const KvView &c)
{
    const int64_t page = slot >> c.page_shift;
    return ((page * c.heads + head) << c.page_shift) + (slot & (((int64_t)1 << c.page_shift) - 1));
}

// Decode factors of the two 16-element halves of a unit from its scale bytes
// (MXFP4: one byte for both), as fp4_dequantize takes them.
template <int FMT>
FP4_DEV void unit_decode_factors(uint32_t sb, float sg, float &d0, float &d1)
{
    if (FMT == FP4_MXFP4) {
        d0 = d1 = e8m0_to_f32(sb & 0xFF);
    } else if (FMT == FP4_MXFP4_16) {
        d0 = e8m0_to_f32(sb & 0xFF);
        d1 = e8m0_to_f32(sb >> 8);
    } else {
        d0 = __fmul_rn(sg, e4m3_to_f32(sb & 0xFF));
        d1 = __fmul_rn(sg, e4m3_to_f32(sb >> 8));
    }
}

}  // namespace fp4
