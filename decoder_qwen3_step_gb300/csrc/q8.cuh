// q8.cuh - the codes and scales of a KV cache held in 8 bits (device helpers).
//
// A page (the K or the V of 16 slots of one KV head of one block) has one scale
// 2^e, e in -40 .. 40; a value is code * 2^e.  Codes are whole numbers -127 ..
// 127 (Q = 127) or e4m3 numbers up to 448 (Q = 448); need(a) is the smallest e
// with a <= Q 2^e.
//
// Why a power of two and not a / Q: dividing by it is exact, so a code depends
// on the value alone and not on how the quotient rounds; a value is exact in
// bf16; and a page whose e rises token by token rounds its codes to steps that
// double, half of the last one + half of the one before it + .. < one step in
// all, where up to 15 rises of a free scale cost half a step each.  e4m3 loses
// nothing by it, i8 half a bit on average.  The range of e keeps ratios of two
// scales (2^80 at most) and their products with softmax weights inside fp32.
#pragma once

#include <cuda_fp8.h>

#include "tree_common.cuh"

namespace dec {

constexpr int kExpMin = -40, kExpMax = 40;

template <int kKind>  // kTreeE4m3 or kTreeI8
struct Q8 {
  static constexpr bool kInt = kKind == kTreeI8;
  static constexpr float kTop = kInt ? 127.f : 448.f;
};

__device__ __forceinline__ float q8_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// e of a stored scale; the least one for memory that holds none.
__device__ __forceinline__ int q8_exp(float scale) {
  const int e = (int)(__float_as_uint(scale) >> 23) - 127;
  return e < kExpMin || e > kExpMax ? kExpMin : e;
}
// need(amax), amax finite: 127 = (2 - 2^-6) 2^6, 448 = 1.75 2^8.
template <int kKind>
__device__ __forceinline__ int q8_need(float amax) {
  const uint32_t b = __float_as_uint(amax), m = b & 0x7FFFFFu;
  const int e = (int)(b >> 23) - 127 + (Q8<kKind>::kInt ? (m > 0x7E0000u) - 6 : (m > 0x600000u) - 8);
  return min(max(e, kExpMin), kExpMax);
}

// Codes of four values divided by their scale: nearest, ties to even, cut at Q.  No NaN.
template <int kKind>
__device__ __forceinline__ uint32_t q8_pack(float4 y) {
  constexpr float q = Q8<kKind>::kTop;
  const float v[4] = {fminf(fmaxf(y.x, -q), q), fminf(fmaxf(y.y, -q), q), fminf(fmaxf(y.z, -q), q), fminf(fmaxf(y.w, -q), q)};
  if constexpr (Q8<kKind>::kInt) {
    const uint32_t a = __byte_perm(__float2int_rn(v[0]), __float2int_rn(v[1]), 0x0040);
    const uint32_t b = __byte_perm(__float2int_rn(v[2]), __float2int_rn(v[3]), 0x0040);
    return __byte_perm(a, b, 0x5410);
  } else {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
  }
}
// The numbers of four codes.
template <int kKind>
__device__ __forceinline__ float4 q8_unpack(uint32_t w) {
  if constexpr (Q8<kKind>::kInt) {  // 2^23 + (code + 128), exact in fp32
    const uint32_t u = w ^ 0x80808080u;
    auto f = [&](uint32_t sel) { return __uint_as_float(__byte_perm(u, 0x4B000000u, sel)) - 8388736.f; };
    return make_float4(f(0x7440), f(0x7441), f(0x7442), f(0x7443));
  } else {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(a), y = __half22float2(b);
    return make_float4(x.x, x.y, y.x, y.y);
  }
}

// Two pairs of codes of a word as f16: bytes (0, 1), (2, 3), or the even and the odd ones.
template <int kKind, bool kEvenOdd>
__device__ __forceinline__ void q8_halves(uint32_t w, uint32_t& x, uint32_t& y) {
  if constexpr (Q8<kKind>::kInt) {
    const uint32_t u = w ^ 0x80808080u, bias = 0x64806480u;  // 1152
    const uint32_t p = __byte_perm(u, 0x64u, kEvenOdd ? 0x4240 : 0x4140), q = __byte_perm(u, 0x64u, kEvenOdd ? 0x4341 : 0x4342);
    const __half2 b = *reinterpret_cast<const __half2*>(&bias);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&p), b), g = __hsub2(*reinterpret_cast<const __half2*>(&q), b);
    x = *reinterpret_cast<const uint32_t*>(&h);
    y = *reinterpret_cast<const uint32_t*>(&g);
  } else {
    const uint32_t u = kEvenOdd ? __byte_perm(w, 0u, 0x3120) : w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(x), "=r"(y)
        : "r"(u));
  }
}

// Bytes (0, 1) and (2, 3) as f16 times a power of two (in both halves of `two`), rounded once where that is subnormal.
template <int kKind>
__device__ __forceinline__ void q8_halves_times(uint32_t w, uint32_t two, uint32_t& x, uint32_t& y) {
  const __half2 f = *reinterpret_cast<const __half2*>(&two);
  __half2 h, g;
  if constexpr (Q8<kKind>::kInt) {  // (1024 + 128 + c) f - 1152 f
    const uint32_t u = w ^ 0x80808080u, bias = 0xE480E480u;  // -1152
    const uint32_t p = __byte_perm(u, 0x64u, 0x4140), q = __byte_perm(u, 0x64u, 0x4342);
    const __half2 b = __hmul2(*reinterpret_cast<const __half2*>(&bias), f);
    h = __hfma2(*reinterpret_cast<const __half2*>(&p), f, b);
    g = __hfma2(*reinterpret_cast<const __half2*>(&q), f, b);
  } else {
    q8_halves<kKind, false>(w, x, y);
    h = __hmul2(*reinterpret_cast<const __half2*>(&x), f);
    g = __hmul2(*reinterpret_cast<const __half2*>(&y), f);
  }
  x = *reinterpret_cast<const uint32_t*>(&h);
  y = *reinterpret_cast<const uint32_t*>(&g);
}

// Codes that are no numbers (memory that no call has written) as 0.
__device__ __forceinline__ uint32_t e4m3_numbers(uint32_t w) {
  const uint32_t nan = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return w & ~((nan >> 7) * 0xFFu);
}

// Index of a page's scale: [layers][blocks][KV heads][K, V].
__device__ __forceinline__ int64_t q8_scale_at(const TreePoolDims& d, int layer, int block, int head, int is_v) {
  return (((int64_t)layer * d.n_blocks + block) * d.Hkv + head) * 2 + is_v;
}

}  // namespace dec
