// Device helpers shared by the kernels: bf16 packing, error reporting.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to_f32(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
};

// Eight consecutive elements loaded as fp32 (16-byte bf16 or 32-byte fp32 load).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  float4 a = __ldg(reinterpret_cast<const float4*>(p));
  float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Round two fp32 to bf16 (nearest even) and pack them, low half first.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

// SiLU(g) * u of the bf16 tensor-core forward epilogues.  __expf and the
// approximate divide keep it at two special-function operations and a few
// FMAs, where the IEEE quotient g / (1 + e^-g) costs a call per element that
// serialised the gate/up epilogue (10 us per 128 x 128 tile against 3 us this
// way).  It stays within a few fp32 ulp of the IEEE form, far inside the bf16
// rounding of H; for g -> -inf the denominator passes 2^126, where __fdividef
// returns 0, the limit of the function.  (The dH epilogue of the bf16 training
// pair keeps the IEEE sigmoid: there the fast form made the kernel 7% slower at
// Grok size.  That of the 8-bit checkpoints, which decodes as well, takes the fast
// one: 65 us a tile with the IEEE quotient, about 15 with it.)
__device__ __forceinline__ float silu_mul_fast(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// Programmatic dependent launch (kernels started with launch_pdl): the kernel
// is launched while the previous kernel of its stream finishes, and
// pdl_wait() blocks until that kernel has completed with its writes visible,
// so every kernel of the forward path calls it before its first access to
// global memory.  No kernel triggers its dependents early
// (griddepcontrol.launch_dependents): with the trigger at the start of each
// kernel, the next kernel's CTAs waited on the SMs through the whole GEMM and
// the Grok-size step took 12% longer; without it the launch overlaps only the
// previous kernel's exit, 3% off the mid-size step and neutral at Grok size.
// A no-op for a kernel launched without the attribute.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 8-bit code of a block of 32 values (activation checkpoints): s = bf16(amax /
// 127) and c = rint(v * (1 / s)) with 1 / s in fp32, which moves a quotient by up
// to 2^-17: next to a tie c may be the other neighbour, and an element is off by
// at most s / 2 (1 + 2^-16) (a divide instead would cost a call per element).
// s / 2 is about amax / 254 (an e4m3 code of the same 8 bits would be off by up to
// 1/16 of the element: for normally distributed rows a root mean square error of
// 2.6% against 0.5%).  A scale below 2^-126 counts as 0 (all codes 0); a block
// that holds a NaN or an infinity gets the scale NaN and decodes to NaN.  amax is
// found on the bit patterns (as unsigned integers NaN and inf are the largest).
// Rounding s to bf16 moves it down by less than 2^-8 of itself, so |v / s| stays
// under 127 (1 + 2^-8) < 127.5 and no clamp is needed; adding 1.5 * 2^23 rounds to
// an integer (ties to even) whose low byte is the code.
__device__ __forceinline__ uint16_t code32(const uint32_t (&v)[32], uint32_t (&codes)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, v[i] & 0x7fffffffu);
  const __nv_bfloat16 sb = __float2bfloat16_rn(__uint_as_float(m) / 127.0f);
  uint16_t bits = __bfloat16_as_ushort(sb);
  float inv = 0.f;
  if (m >= 0x7f800000u)
    bits = 0x7fc0;
  else if (bits < 0x0080)
    bits = 0;
  else
    inv = 1.0f / __bfloat162float(sb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      q[k] = __float_as_uint(inv > 0.f ? fmaf(__uint_as_float(v[4 * i + k]), inv, 12582912.0f) : 12582912.0f);
    codes[i] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  }
  return bits;
}

// Two fp32 values in a register pair, for the instructions that work on both.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(f32x2 v) {
  float a, b;
  unpack2(v, a, b);
  return pack_bf16x2(a, b);
}

// 32 bytes that are read once, a whole sector in one load: as two 16-byte
// streaming loads the second half missed L1 as well, which held the backward of
// 8-bit checkpoints at 153 against 122 us (T 2048, d 1536, f 8192).
__device__ __forceinline__ void load32_once(const void* p, uint4 (&v)[2]) {
  asm volatile("ld.global.L1::no_allocate.L2::128B.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                 "=r"(v[1].w)
               : "l"(p));
}

// Codes 2i and 2i + 1 of a word as fp32 integers: the biased byte b under the
// exponent of 2^23 reads 2^23 + b.
__device__ __forceinline__ f32x2 codes2(uint32_t w, int i) {
  w ^= 0x80808080u;
  return add2(pack2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + 2 * i)),
                    __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441 + 2 * i))),
              pack2(-8388736.0f, -8388736.0f));
}

__device__ __forceinline__ void flag_error(int* err, int bits) {
  if (err) atomicOr(err, bits);
}

}  // namespace moe
