// Rows of channels in eight-channel vectors, and the 8-bit checkpoint code: shared by the
// norm, residual and checkpoint kernels and the backward's row statistics.
//
// Checkpoint code.  A group is 128 channels of a row (the last group of a row may be
// shorter) and has one power-of-two scale 2^(E - 127), E in [1, 254] in one byte:
// the smallest one for which the group's largest magnitude still has a code
// (int8: |x| * 2^(127 - E) < 127.5; e4m3: <= 448).  Scaling by a power of two is exact,
// so a code is the nearest one to x with ties to even and nothing else is rounded, and a
// code times its scale (7 or 4 significant bits) is exact in bf16: what the tensor cores
// multiply is what the checkpoint holds.  (E never goes below 1.  The steps of e4m3 are then
// 2^-135, or 2^-134 with E = 2, below bf16's smallest number 2^-133; the codes of a bf16
// tensor do not use them, since its numbers are multiples of 2^-133.)  A finer scale would
// halve int8's step at most and put a rounding behind every read.  A group with an infinity,
// a NaN or a magnitude whose nearest value would be 2^128 gets E = 255 and reads as NaN
// throughout, so an overflow is not silently clipped.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ssta_f32x2.cuh"
#include "ssta_internal.h"

namespace ssta {
namespace rows {

using f32x2::f2_add;
using f32x2::f2_fma;
using f32x2::f2_mul;
using f32x2::f2_pack;
using f32x2::f2_unpack;

constexpr int kVec = 8;            // channels of one thread's vector
constexpr int kGroup = 128;        // channels of a checkpoint group
constexpr int kGroupLanes = kGroup / kVec;

__host__ __device__ inline int groups_per_row(int C) { return (C + kGroup - 1) / kGroup; }

// Eight channels as stored: 16 bytes of bf16, 32 of fp32, 8 of codes.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { uint4 a; };
template <> struct Raw<float> { float4 a, b; };

__device__ __forceinline__ Raw<__nv_bfloat16> load_raw(const __nv_bfloat16* p) {
  return {*reinterpret_cast<const uint4*>(p)};
}
// fp32: 32 bytes at once where the tensor allows it (it is 16-byte aligned at least, and
// rows are whole multiples of 32 bytes), since two 16-byte accesses of a warp touch every
// 32-byte sector twice.
__device__ __forceinline__ Raw<float> load_raw(const float* p) {
  Raw<float> r;
  if ((reinterpret_cast<uintptr_t>(p) & 16) == 0)
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r.a.x), "=f"(r.a.y), "=f"(r.a.z), "=f"(r.a.w), "=f"(r.b.x), "=f"(r.b.y), "=f"(r.b.z), "=f"(r.b.w)
                 : "l"(p)
                 : "memory");
  else
    r = {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
  return r;
}
template <typename T> __device__ __forceinline__ Raw<T> zero_raw() { return Raw<T>{}; }
__device__ __forceinline__ void store_raw(__nv_bfloat16* p, const Raw<__nv_bfloat16>& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
}
__device__ __forceinline__ void store_raw(float* p, const Raw<float>& r) {
  if ((reinterpret_cast<uintptr_t>(p) & 16) == 0) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(r.a.x), "f"(r.a.y), "f"(r.a.z),
                 "f"(r.a.w), "f"(r.b.x), "f"(r.b.y), "f"(r.b.z), "f"(r.b.w)
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = r.a;
    reinterpret_cast<float4*>(p)[1] = r.b;
  }
}

// Eight channels in fp32, as four pairs: the kernels' arithmetic runs on pairs
// (f32x2), which halves the instructions of what would otherwise be bound by issue
// (the scalar form of the residual kernels took 25 to 54 instructions per channel).
struct V8 {
  uint64_t p[4];
};
__device__ __forceinline__ uint64_t splat(float a) { return f2_pack(a, a); }
__device__ __forceinline__ V8 fill(float a) { return {splat(a), splat(a), splat(a), splat(a)}; }

__device__ __forceinline__ V8 unpack(const Raw<__nv_bfloat16>& r) {   // bf16 is the upper half of an fp32
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return v;
}
__device__ __forceinline__ V8 unpack(const Raw<float>& r) {
  return {f2_pack(r.a.x, r.a.y), f2_pack(r.a.z, r.a.w), f2_pack(r.b.x, r.b.y), f2_pack(r.b.z, r.b.w)};
}
__device__ __forceinline__ uint32_t pack2(uint64_t p) {
  float lo, hi;
  f2_unpack(p, lo, hi);
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ Raw<__nv_bfloat16> pack(const V8& v, __nv_bfloat16) {
  return {make_uint4(pack2(v.p[0]), pack2(v.p[1]), pack2(v.p[2]), pack2(v.p[3]))};
}
__device__ __forceinline__ Raw<float> pack(const V8& v, float) {
  Raw<float> r;
  f2_unpack(v.p[0], r.a.x, r.a.y);
  f2_unpack(v.p[1], r.a.z, r.a.w);
  f2_unpack(v.p[2], r.b.x, r.b.y);
  f2_unpack(v.p[3], r.b.z, r.b.w);
  return r;
}
template <typename T> __device__ __forceinline__ V8 load8(const T* p) { return unpack(load_raw(p)); }
template <typename T> __device__ __forceinline__ void store8(T* p, const V8& v) { store_raw(p, pack(v, T())); }

__device__ __forceinline__ V8 mul(const V8& a, const V8& b) {
  return {f2_mul(a.p[0], b.p[0]), f2_mul(a.p[1], b.p[1]), f2_mul(a.p[2], b.p[2]), f2_mul(a.p[3], b.p[3])};
}
__device__ __forceinline__ V8 mul(const V8& a, float s) { return mul(a, fill(s)); }
__device__ __forceinline__ V8 add(const V8& a, const V8& b) {
  return {f2_add(a.p[0], b.p[0]), f2_add(a.p[1], b.p[1]), f2_add(a.p[2], b.p[2]), f2_add(a.p[3], b.p[3])};
}
__device__ __forceinline__ V8 fma(const V8& a, const V8& b, const V8& c) {
  return {f2_fma(a.p[0], b.p[0], c.p[0]), f2_fma(a.p[1], b.p[1], c.p[1]), f2_fma(a.p[2], b.p[2], c.p[2]),
          f2_fma(a.p[3], b.p[3], c.p[3])};
}
__device__ __forceinline__ V8 fma(const V8& a, float b, float c) { return fma(a, fill(b), fill(c)); }
__device__ __forceinline__ V8 fma(float a, const V8& b, const V8& c) { return fma(fill(a), b, c); }
__device__ __forceinline__ float sum(uint64_t p) {
  float lo, hi;
  f2_unpack(p, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float sum(const V8& v) {
  return sum(f2_add(f2_add(v.p[0], v.p[1]), f2_add(v.p[2], v.p[3])));
}
// Sum of the products' pairs, for one more addition at the end.
__device__ __forceinline__ float dot(const V8& a, const V8& b) {
  return sum(f2_add(f2_fma(a.p[1], b.p[1], f2_mul(a.p[0], b.p[0])), f2_fma(a.p[3], b.p[3], f2_mul(a.p[2], b.p[2]))));
}

// Exponent byte of a group from the bits of its largest magnitude.  With the magnitude
// (1 + m) 2^f, int8 takes E = f - 6, or one more where (1 + m) 2^6 reaches 127.5 (m from
// 0x7f0000 on), e4m3 E = f - 8, or one more where (1 + m) 2^8 passes 448 (m above
// 0x600000): the addition carries into the exponent exactly there.
__device__ __forceinline__ int group_exponent(uint32_t amax, int format) {
  const bool int8 = format == SSTA_INT8;
  const int E = max(1, (int)((amax + (int8 ? 0x10000u : 0x1fffffu)) >> 23) - (int8 ? 6 : 8));
  // from 63.75 * 2^122 (int8) or 248 * 2^120 (e4m3) on, the nearest value is 2^128
  return amax >= (int8 ? 0x7f7f0000u : 0x7f780000u) ? 255 : E;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Bits of the largest magnitude of the group this thread's vector belongs to: 16
// consecutive lanes hold a group.  Infinities and NaN carry through.
__device__ __forceinline__ uint32_t group_amax(const V8& v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(v.p[i], lo, hi);
    m = max_nan(m, max_nan(fabsf(lo), fabsf(hi)));
  }
#pragma unroll
  for (int off = kGroupLanes / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  return __float_as_uint(m) & 0x7fffffffu;
}

// Eight codes of v under exponent byte E (zeros under 255).
__device__ __forceinline__ uint2 encode8(const V8& v, int E, int format) {
  const float up = __uint_as_float((uint32_t)(254 - E) << 23);   // 2^(127 - E)
  uint2 c;
  if (format == SSTA_INT8) {
    // adding 1.5 * 2^23 leaves the nearest integer (ties to even) in the low byte
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f2_unpack(f2_fma(v.p[i], splat(up), splat(12582912.0f)), lo, hi);
      b[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
    }
    c = make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      f2_unpack(f2_mul(v.p[i], splat(up)), f.x, f.y);
      h[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    c = make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
  }
  return E == 255 ? make_uint2(0u, 0u) : c;
}

// Scale of exponent byte E; NaN for 255.
__device__ __forceinline__ float code_scale(int E) { return __uint_as_float(E == 255 ? 0x7fc00000u : (uint32_t)E << 23); }

// Eight codes as numbers, before their scale.
__device__ __forceinline__ V8 decode8(uint2 c, int format) {
  const uint32_t w[2] = {c.x, c.y};
  V8 v;
  if (format == SSTA_INT8) {
    const uint32_t u[2] = {w[0] ^ 0x80808080u, w[1] ^ 0x80808080u};   // byte + 128
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // in the low mantissa bits of 2^23, less 2^23 + 128
      const uint32_t lo = __byte_perm(u[i >> 1], 0x4b000000u, 0x7440 | (2 * i & 3));
      const uint32_t hi = __byte_perm(u[i >> 1], 0x4b000000u, 0x7440 | (2 * i + 1 & 3));
      v.p[i] = f2_add(f2_pack(__uint_as_float(lo), __uint_as_float(hi)), splat(-8388736.0f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v.p[i] = f2_pack(f.x, f.y);
    }
  }
  return v;
}

}  // namespace rows
}  // namespace ssta
