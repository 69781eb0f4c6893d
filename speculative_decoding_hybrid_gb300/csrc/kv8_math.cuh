// Arithmetic of the attention over the 8-bit cache: pairs of fp32 and fp16
// values, and rows split into e4m3 parts (sm_103a).
#pragma once

#include "kv8.cuh"
#include "tc.cuh"

namespace kv8 {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Barrier of a group's four softmax warps with an OR over a predicate.
__device__ __forceinline__ bool group_or(int group, bool p) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, "
        "q;\n}\n"
        : "=r"(r)
        : "r"(uint32_t(p)), "r"(group + 1)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(gdn::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Pairs of fp32 values: one instruction an operation.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 pair(uint32_t a, uint32_t b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 both(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// c - 32 h of two fp32 values c and two fp16 values h.
__device__ __forceinline__ float2 minus32(float2 c, uint32_t h) {
    float2 r;
    asm("{\n .reg .b16 a, b, k;\n mov.b32 {a, b}, %2;\n mov.b16 k, 0xd000;\n fma.rn.f32.f16 %0, a, k, %3;\n"
        " fma.rn.f32.f16 %1, b, k, %4;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ uint32_t join16(uint16_t lo, uint16_t hi) {
    uint32_t r;
    asm("mov.b32 %0, {%1, %2};" : "=r"(r) : "h"(lo), "h"(hi));
    return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// An fp16 value's upper byte is an e5m2 code, the value cut to 3 bits.  What that
// leaves of two values, times 8: exact.
__device__ __forceinline__ uint32_t rest8(uint32_t h) {
    uint32_t d, r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(h & 0xff00ff00u));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(d), "r"(0x48004800u));  // 8, 8
    return r;
}
// The upper bytes of four fp16 values.
__device__ __forceinline__ uint32_t upper4(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }

template <int D>
__device__ __forceinline__ void load_row(const uint16_t *p, int sub, bool have, uint4 (&w)[D / 64]) {
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
        w[e] = have ? *reinterpret_cast<const uint4 *>(p + sub * (D / 8) + e * 8) : make_uint4(0, 0, 0, 0);
}
// The largest magnitude of a row, as bf16's bits: magnitudes order like them, with
// infinities and NaN on top.
template <int D>
__device__ __forceinline__ uint32_t row_top(const uint4 (&w)[D / 64]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
        m = __vmaxu2(m, __vmaxu2(w[e].x & 0x7fff7fffu, w[e].y & 0x7fff7fffu));
        m = __vmaxu2(m, __vmaxu2(w[e].z & 0x7fff7fffu, w[e].w & 0x7fff7fffu));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m >> 16, m & 0xffffu);
}
// The power of two that brings such a magnitude to 2^7 .. 2^8; rows are scaled by at
// most 2^kMaxUp (32 times that, and 2^14 times, are still finite), and by 2^-120 at least;
// past 2^kMinFit scores are not left to the parts.
constexpr int kMaxUp = 110, kMinFit = -60;
__device__ __forceinline__ int fit_of(uint32_t top) { return 7 - (int(top >> 7) - 127); }

// A warp splits four rows of bf16, eight threads (sub) a row: x = (hi + lo/32) 2^-k
// into rows rh and rl of an operand tile of `rows` rows.  -> 2^-k, or NaN for a row
// that is not finite (whatever its parts then are: a row's products are its own).
// The low part ends at 2^-14: an element from 2^-7 on, 2^-14 of the largest at most,
// keeps all its 8 bits; a smaller one is off by up to 2^-15, 2^-22 of the largest.
// `maybe`: this thread has an element that small, zeros among them, or the row is past
// 2^67: row_loss has to say what that means.
template <int D>
__device__ __forceinline__ float split_row(const uint4 (&w)[D / 64], int sub, uint8_t *tile, int rows, int rh, int rl,
                                           bool &maybe) {
    constexpr int E = D / 8, kRow = D < 128 ? D : 128;
    const uint32_t top = row_top<D>(w);
    const int fit = fit_of(top), k = min(kMaxUp, fit);
    const f2 up = pair(pow2i(k), pow2i(k)), up32 = pair(32.f * pow2i(k), 32.f * pow2i(k));
    uint32_t h[E / 4], l[E / 4], large = ~0u;  // every byte's top bit: hi's code is 5 (5 * 2^-9) or more
#pragma unroll
    for (int e = 0; e < E / 8; ++e) {
        const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
        uint16_t hh[4], ll[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 x = pair(u[i] << 16, u[i] & 0xffff0000u);
            const float2 a = both(mul2(x, up));
            hh[i] = uint16_t(e4m3x2(a.x, a.y));
            const float2 r = minus32(both(mul2(x, up32)), f16x2_of(hh[i]));
            ll[i] = uint16_t(e4m3x2(r.x, r.y));
        }
        h[2 * e] = join16(hh[0], hh[1]);
        h[2 * e + 1] = join16(hh[2], hh[3]);
        l[2 * e] = join16(ll[0], ll[1]);
        l[2 * e + 1] = join16(ll[2], ll[3]);
        large &= ((h[2 * e] & 0x7f7f7f7fu) + 0x7b7b7b7bu) & ((h[2 * e + 1] & 0x7f7f7f7fu) + 0x7b7b7b7bu);
    }
    maybe = top > 0 && top < 0x7f80u && ((~large & 0x80808080u) || fit < kMinFit);
    if constexpr (E == 8) {
        uint8_t *t = tile + ((sub * 8) & 8);
        *reinterpret_cast<uint2 *>(t + tc::swz8_off<kRow>(rh, sub >> 1)) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint2 *>(t + tc::swz8_off<kRow>(rl, sub >> 1)) = make_uint2(l[0], l[1]);
    } else {
#pragma unroll
        for (int b = 0; b < E / 16; ++b) {
            const int e0 = sub * E + b * 16, in = e0 % kRow;
            uint8_t *t = tile + e0 / kRow * rows * kRow;
            *reinterpret_cast<uint4 *>(t + tc::swz8_off<kRow>(rh, in >> 4)) =
                make_uint4(h[4 * b], h[4 * b + 1], h[4 * b + 2], h[4 * b + 3]);
            *reinterpret_cast<uint4 *>(t + tc::swz8_off<kRow>(rl, in >> 4)) =
                make_uint4(l[4 * b], l[4 * b + 1], l[4 * b + 2], l[4 * b + 3]);
        }
    }
    return top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2i(-k);
}

// What a row's parts leave of it: the sum of its elements' losses, which times the other
// side's largest magnitude bounds what a product loses; -1 for a row past 2^67, whose
// factors might leave fp32 whatever its parts hold.
template <int D>
__device__ __forceinline__ float row_loss(const uint4 (&w)[D / 64]) {
    const uint32_t top = row_top<D>(w);
    const int fit = fit_of(top), k = min(kMaxUp, fit);
    // in units of 2^-14, the low part's last bit; an element from 2^-7 on is a whole number of them, and all
    // are below 2^22, where adding 1.5 * 2^23 rounds
    const f2 unit = pair(pow2i(k + 14), pow2i(k + 14)), whole = pair(12582912.f, 12582912.f),
             back = pair(-12582912.f, -12582912.f), minus = pair(-1.f, -1.f);
    float loss = 0.f;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
        const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 y = mul2(pair(u[i] << 16, u[i] & 0xffff0000u), unit);
            const float2 d = both(fma2(add2(add2(y, whole), back), minus, y));
            loss += fabsf(d.x) + fabsf(d.y);
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    if (top == 0 || top >= 0x7f80u) return 0.f;
    return fit < kMinFit ? -1.f : loss * pow2i(-k) * 0x1p-14f;
}

// Sums of products in fp32: of a key as the cache holds it and a query times up, of a
// new key times down and a query times up.
__device__ __forceinline__ void add4(float (&acc)[4], float2 a, float2 b, uint32_t y0, uint32_t y1, float up) {
    acc[0] = fmaf(a.x, __uint_as_float(y0 << 16) * up, acc[0]);
    acc[1] = fmaf(a.y, __uint_as_float(y0 & 0xffff0000u) * up, acc[1]);
    acc[2] = fmaf(b.x, __uint_as_float(y1 << 16) * up, acc[2]);
    acc[3] = fmaf(b.y, __uint_as_float(y1 & 0xffff0000u) * up, acc[3]);
}
template <int D>
__device__ __forceinline__ float dot_codes(const uint8_t *k, const uint16_t *q, float up) {
    float acc[4] = {};
#pragma unroll 2
    for (int e = 0; e < D; e += 8) {
        const uint2 x = *reinterpret_cast<const uint2 *>(k + e);
        const uint4 y = *reinterpret_cast<const uint4 *>(q + e);
        add4(acc, f32x2_of(uint16_t(x.x)), f32x2_of(uint16_t(x.x >> 16)), y.x, y.y, up);
        add4(acc, f32x2_of(uint16_t(x.y)), f32x2_of(uint16_t(x.y >> 16)), y.z, y.w, up);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}
template <int D>
__device__ __forceinline__ float dot_rows(const uint16_t *k, float down, const uint16_t *q, float up) {
    float acc[4] = {};
#pragma unroll 1
    for (int e = 0; e < D; e += 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(k + e), y = *reinterpret_cast<const uint4 *>(q + e);
        const auto two = [down](uint32_t w) {
            return make_float2(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
        };
        add4(acc, two(x.x), two(x.y), y.x, y.y, up);
        add4(acc, two(x.z), two(x.w), y.z, y.w, up);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Sums of N values over a warp's lanes: value k's sum lands in v[0] of the
// lanes whose top log2(N) bits are k.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
    constexpr int kSteps = N == 16 ? 4 : 3;
    static_assert(N == 16 || N == 8, "columns a thread");
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int off = 16 >> s, half = N >> (s + 1);
        const bool up = lane & off;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float give = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
#pragma unroll
    for (int off = 16 >> kSteps; off; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
}

}  // namespace kv8
