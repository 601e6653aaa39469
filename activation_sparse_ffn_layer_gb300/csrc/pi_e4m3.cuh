// pi_e4m3.cuh -- codes of the 8-bit cache: conversions, exponents, addresses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/pi.h"
#include "pi_common.cuh"

namespace pi {
namespace e4m3 {

constexpr int kBlock = 16;             // positions that share an exponent
constexpr int kMinExp = -32, kMaxExp = 32;

// Two codes (the low 16 bits) as two fp16 values, exactly: e4m3 has 4 bits of
// significand and lies within fp16's range.  A NaN stays one.
PI_DEV uint32_t widen2(uint32_t codes) {
    uint32_t h;
    const unsigned short c = (unsigned short)codes;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}
PI_DEV float2 values2(uint32_t codes) {
    const uint32_t h = widen2(codes);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Codes of two fp32 values, rounded to nearest even, magnitudes past 448 held
// as that (lo in bits 0-7).  A NaN becomes the code of NaN.
PI_DEV uint32_t encode2(float lo, float hi) {
    unsigned short c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}
// 2^e for -126 <= e <= 127
PI_DEV float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
PI_DEV int bounded(int e) { return min(max(e, kMinExp), kMaxExp); }

// The smallest e in range with m <= 448 2^e = 1.75 2^(8 + e), from the bits of m >= 0.
PI_DEV int exponent_of(uint32_t bits) {
    return bounded((int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0));
}

}  // namespace e4m3

// Strides (bytes) and sizes of an 8-bit cache in the kernels' arguments.
struct Cache8 {
    const uint8_t *k, *v;
    const int8_t *ke, *ve;
    long long page_stride, head_stride, token_stride;
    int kv_heads, page_shift, num_pages;
};

bool page8_desc_ok(const pi_page8_desc& c);

}  // namespace pi
