// The 4-bit KV cache: what a row holds, and the conversions.
//
// A head's row of 128 values is 64 bytes of codes and 8 bytes of scales, in two
// arrays: value i = t * scale[i / 16] * code[i], code a 4-bit float (sign, two
// exponent bits, one mantissa bit: 0 0.5 1 1.5 2 3 4 6, the even i of a pair
// in a byte's low half), scale an e4m3, t the cache's own factor, a power of
// two.  4.5 bits a value.  A code has 2 significant bits and a scale 4, so that
// scale * code, 2^-10 to 2688 or 0, is exact in bf16 and in fp16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace qasc {

constexpr int kKv4Group = 16;                    // values of a scale
constexpr int kKv4Groups = kD / kKv4Group;       // scales of a row, bytes
constexpr int kKv4Codes = kD / 2;                // bytes of a row's codes

// Tokens of a sequence of `len` that its newest ql attend to, sink and window, and
// how many in between none of them does.
__device__ __forceinline__ int kv4_tokens_seen(int64_t len, int64_t ql, int sink, int local, int* between) {
  const int64_t lo = max(len - ql - local + 1, int64_t(0));   // the first row's window
  *between = static_cast<int>(max(lo - sink, int64_t(0)));
  return static_cast<int>(len) - *between;
}

// Two e4m3 of a word's low 16 bits -> fp16 pair (exact).
__device__ __forceinline__ __half2 kv4_scales(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<__half2*>(&h);
}

// The four bytes of w, two codes each -> fp16 pairs (low code, high code).
__device__ __forceinline__ void kv4_codes(uint32_t w, __half2 (&h)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<__half2*>(&r[i]);
}

// x rounded to 16 significant bits.  A quotient of 8 bits (bf16) by 4 (e4m3) or by 6
// meets a border between two values of the format exactly or stays 2^-8 of
// itself away from it, so that a quotient made with a rounded reciprocal (2^-22 off
// at most) has every comparison with a border, ties among them, as exact
// division has it once its last bits are rounded away.
__device__ __forceinline__ float kv4_quotient(float x) { return __uint_as_float((__float_as_uint(x) + 0x80u) & 0xffffff00u); }

// Scale byte of a group whose largest magnitude is `a` (NaN where it holds one):
// a / 6 rounded to e4m3, at most 448.
__device__ __forceinline__ uint32_t kv4_scale_of(float a) {
  uint16_t e;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(0.0f), "f"(a == a ? kv4_quotient(a * (1.0f / 6.0f)) : a));
  return e;
}

// 1 / scale, to an ulp; 0 for a scale of 0 or NaN.
__device__ __forceinline__ float kv4_divisor(uint32_t byte) {
  uint32_t h;
  float r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return s > 0.0f ? r : 0.0f;
}

// Eight quotients -> eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t kv4_pack(const float (&q)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 bytes copied to shared memory without passing through registers, and the thread's groups of copies.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace qasc
