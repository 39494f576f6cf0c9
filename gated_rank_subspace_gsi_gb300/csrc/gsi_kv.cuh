// gsi_kv.cuh -- device-side pieces shared by the cache's kernels: where rows
// and pages lie, and the codes of both formats.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gsi_device.cuh"
#include "gsi_kv.h"

namespace gsi {

constexpr int kInt8 = GSI_KV_INT8, kE4m3 = GSI_KV_E4M3;

// Rows [first, first + count) of sequence b, and the tokens held before them;
// what the caller's arrays give outside their ranges is cut off.
struct SeqRows {
  int first, count, len;
};
__device__ __forceinline__ SeqRows seq_rows(const KvRows& r, const KvView& c, int b) {
  SeqRows s;
  const int lo = r.row_start[b], hi = r.row_start[b + 1], len = r.len[b];
  s.first = min(max(lo, 0), r.rows);
  s.count = min(max(hi, s.first), r.rows) - s.first;
  s.len = min(max(len, 0), c.max_pages * kPage);
  if (s.first != lo || s.first + s.count != hi || s.len != len || s.count > r.max_rows)
    atomicOr(c.status, kStatusBadPage);
  return s;
}

// Page of block `blk` of sequence b, or -1 (status set).
__device__ __forceinline__ int page_of(const KvView& c, int b, int blk) {
  int p = -1;
  if (blk >= 0 && blk < c.max_pages) p = c.page_table[size_t(b) * c.max_pages + blk];
  if (p < 0 || p >= c.pages) {
    atomicOr(c.status, kStatusBadPage);
    return -1;
  }
  return p;
}

// 16 bytes that are read once, without a place in L1.  Not by the read-only path
// (ld.global.nc): the kernels that fill the pages may still run when this one starts.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Exponent of the least power of two, at least 2^kScaleMin, with
// top <= Q 2^e.  With top = m 2^x (0.5 <= m < 1): Q = 127 = (127 / 128) 2^7,
// Q = 448 = 0.875 2^9.
template <int FMT>
__device__ __forceinline__ int scale_exp(float top) {
  const int x = int((__float_as_uint(top) >> 23) & 0xFF) - 126;  // 0 and subnormals: the minimum below
  const uint32_t frac = __float_as_uint(top) & 0x7FFFFFu;        // m = 0.5 + frac / 2^24
  const int e = FMT == kInt8 ? x - 7 + (frac > 0x7E0000u) : x - 9 + (frac > 0x600000u);
  return max(e, kScaleMin);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Codes of two values already divided by the scale, in the low and high byte.
template <int FMT>
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  if (FMT == kInt8)
    return (uint32_t(__float2int_rn(a)) & 0xFFu) | ((uint32_t(__float2int_rn(b)) & 0xFFu) << 8);
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Two codes (low 16 bits) as floats.
template <int FMT>
__device__ __forceinline__ float2 decode2(uint32_t w) {
  if (FMT == kInt8) return make_float2(float(int8_t(w & 0xFF)), float(int8_t((w >> 8) & 0xFF)));
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xFFFF), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float finite_or_zero(float x, bool& bad) {
  const bool ok = (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
  bad |= !ok;
  return ok ? x : 0.f;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 8 values from element `i` of a row of fp32 or bf16, rounded to bf16 and
// packed; non-finite ones are zero.
__device__ __forceinline__ uint4 load8_bf16(const void* p, int64_t i, int bf16, bool& bad) {
  float f[8];
  if (bf16) {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), f);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  uint4 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // a finite fp32 value may round to an infinite bf16
    f[j] = finite_or_zero(__bfloat162float(__float2bfloat16_rn(f[j])), bad);
  }
  o.x = pack_bf16(f[0], f[1]);
  o.y = pack_bf16(f[2], f[3]);
  o.z = pack_bf16(f[4], f[5]);
  o.w = pack_bf16(f[6], f[7]);
  return o;
}

__device__ __forceinline__ float max8(const uint4& v, float m) {
  float f[8];
  bf16x8_to_f32(v, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  return m;
}

// 8 bf16 values times inv (a power of two), as codes.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const uint4& v, float inv) {
  float f[8];
  bf16x8_to_f32(v, f);
  uint2 o;
  o.x = encode2<FMT>(f[0] * inv, f[1] * inv) | (encode2<FMT>(f[2] * inv, f[3] * inv) << 16);
  o.y = encode2<FMT>(f[4] * inv, f[5] * inv) | (encode2<FMT>(f[6] * inv, f[7] * inv) << 16);
  return o;
}

}  // namespace gsi
