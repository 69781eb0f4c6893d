// Paged 8-bit key/value cache: what its kernels share (sm_103a).
#pragma once

#include <math.h>

#include "common.cuh"

namespace kv8 {

constexpr int kMinScaleExp = -100;  // scales are 2^e, e >= this

// Exponent e of the least power of two with amax / 2^e <= 448 = 1.75 * 2^8
// (amax >= 0 finite; zero and subnormals give the floor).
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = int(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kMinScaleExp ? kMinScaleExp : e;
}
// 2^e for a normal exponent.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The exponent of a power of two (of another positive number, its largest power of two's; -127 for zero).
__device__ __forceinline__ float exponent_of(float x) {
    return __uint_as_float(0x4b000000u | (__float_as_uint(x) >> 23)) - 8388735.f;  // 2^23 + 127
}

// Two fp32 -> two e4m3 codes (nearest even, +-448 beyond), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes -> two fp16 values (exact).
__device__ __forceinline__ uint32_t f16x2_of(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}
__device__ __forceinline__ float2 f32x2_of(uint16_t codes) {
    const uint32_t h = f16x2_of(codes);
    float2 f;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

}  // namespace kv8

namespace gdn_host {
inline int kv8_check(const kv8_cache *c) {
    if (!c) return GDN_ERR_NULL;
    if (!(c->d == 64 || c->d == 128 || c->d == 256)) return GDN_ERR_SHAPE;
    if (!(c->page_tokens == 16 || c->page_tokens == 32 || c->page_tokens == 64 || c->page_tokens == 128))
        return GDN_ERR_SHAPE;
    if (c->h_kv <= 0 || c->h_q <= 0 || c->h_q % c->h_kv != 0 || c->h_q / c->h_kv > 64 || c->h_kv > 1024)
        return GDN_ERR_SHAPE;
    if (c->window < 0 || c->num_pages <= 0 || c->num_layers <= 0 || !isfinite(c->sm_scale)) return GDN_ERR_ARG;
    if (!c->kv || !c->scale) return GDN_ERR_NULL;
    const int64_t page = int64_t(2) * c->h_kv * c->page_tokens * c->d;
    if (c->page_stride < page || c->layer_stride < page || c->page_stride % 16 || c->layer_stride % 16)
        return GDN_ERR_ARG;
    if (c->scale_page_stride < 2 * c->h_kv || c->scale_layer_stride < 2 * c->h_kv || c->scale_page_stride % 2 ||
        c->scale_layer_stride % 2)
        return GDN_ERR_ARG;
    if (!aligned16(c->kv) || (reinterpret_cast<uintptr_t>(c->scale) & 7u)) return GDN_ERR_ARG;
    return GDN_OK;
}
// Rows of `heads` heads of d bf16 values, `stride` elements apart.
inline bool kv8_rows_ok(const void *p, int64_t stride, int64_t heads, int d) {
    return aligned16(p) && stride >= heads * d && stride % 8 == 0;
}
constexpr int32_t kKv8MaxLen = 1 << 30;
}  // namespace gdn_host
