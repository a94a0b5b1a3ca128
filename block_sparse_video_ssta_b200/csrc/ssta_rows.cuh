// Rows of channels in eight-channel vectors, and the 8-bit checkpoint code: shared by the
// norm, residual and checkpoint kernels and the backward's row statistics.
//
// Checkpoint code.  A group is 128 channels of a row (the last group of a row may be
// shorter) and has one power-of-two scale 2^(E - 127), E in [1, 254] in one byte:
// the smallest one for which the group's largest magnitude still has a code
// (int8: |x| * 2^(127 - E) < 127.5; e4m3: <= 448).  Scaling by a power of two is exact,
// so a code is the nearest one to x with ties to even and nothing else is rounded, and a
// code times its scale (7 or 4 significant bits) is exact in bf16: what the tensor cores
// multiply is what the checkpoint holds.  A finer scale would halve int8's step at most
// and put a rounding behind every read.  A group with an infinity, a NaN or a magnitude
// whose nearest value would be 2^128 gets E = 255 and reads as NaN throughout, so an
// overflow stays visible in the gradients.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ssta_internal.h"

namespace ssta {
namespace rows {

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
__device__ __forceinline__ Raw<float> load_raw(const float* p) {
  return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
}
template <typename T> __device__ __forceinline__ Raw<T> zero_raw() { return Raw<T>{}; }

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float (&v)[kVec]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {      // bf16 is the upper half of an fp32
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&v)[kVec]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ Raw<__nv_bfloat16> pack(const float (&v)[kVec], __nv_bfloat16) {
  return {make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]))};
}
__device__ __forceinline__ Raw<float> pack(const float (&v)[kVec], float) {
  return {make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
}
__device__ __forceinline__ void store_raw(__nv_bfloat16* p, const Raw<__nv_bfloat16>& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
}
__device__ __forceinline__ void store_raw(float* p, const Raw<float>& r) {
  reinterpret_cast<float4*>(p)[0] = r.a;
  reinterpret_cast<float4*>(p)[1] = r.b;
}
template <typename T> __device__ __forceinline__ void load8(const T* p, float (&v)[kVec]) { unpack(load_raw(p), v); }
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&v)[kVec]) { store_raw(p, pack(v, T())); }

// Eight elements of a parameter vector of either type (is_f32 is the same for a whole launch).
__device__ __forceinline__ void load_param8(const void* p, int64_t i, bool is_f32, float (&v)[kVec]) {
  if (is_f32)
    load8(static_cast<const float*>(p) + i, v);
  else
    load8(static_cast<const __nv_bfloat16*>(p) + i, v);
}

// Exponent byte of a group from the bits of its largest magnitude.
__device__ __forceinline__ int group_exponent(uint32_t amax, int format) {
  // from 63.75 * 2^122 (int8) or 248 * 2^120 (e4m3) on, the nearest value is 2^128
  if (amax >= (format == SSTA_INT8 ? 0x7f7f0000u : 0x7f780000u)) return 255;
  const int f = (int)(amax >> 23);
  const uint32_t m = amax & 0x7fffffu;
  // 127.5 = 1.9921875 * 2^6 (not reached), 448 = 1.75 * 2^8 (reached)
  const int E = format == SSTA_INT8 ? f - 6 + (m >= 0x7f0000u) : f - 8 + (m > 0x600000u);
  return E < 1 ? 1 : E;
}

// Bits of the largest magnitude of the group this thread's vector belongs to: 16
// consecutive lanes hold a group.  As integers infinities and NaN rank above all numbers.
__device__ __forceinline__ uint32_t group_amax(const float (&v)[kVec]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = kGroupLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// Eight codes of v under exponent byte E.
__device__ __forceinline__ uint2 encode8(const float (&v)[kVec], int E, int format) {
  if (E == 255) return make_uint2(0u, 0u);
  const float up = __uint_as_float((uint32_t)(254 - E) << 23);   // 2^(127 - E)
  if (format == SSTA_INT8) {
    // adding 1.5 * 2^23 leaves the nearest integer (ties to even) in the low byte
    uint32_t b[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) b[i] = __float_as_uint(fmaf(v[i], up, 12582912.0f));
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
  }
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * up, v[2 * i + 1] * up), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Values of eight codes.
__device__ __forceinline__ void decode8(uint2 c, int E, int format, float (&v)[kVec]) {
  const float scale = E == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)E << 23);
  const uint32_t w[2] = {c.x, c.y};
  if (format == SSTA_INT8) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      // byte + 128 in the low mantissa bits of 2^23
      const uint32_t u = __byte_perm(w[i >> 2] ^ 0x80808080u, 0x4b000000u, 0x7440 | (i & 3));
      v[i] = (__uint_as_float(u) - 8388736.0f) * scale;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
}

}  // namespace rows
}  // namespace ssta
