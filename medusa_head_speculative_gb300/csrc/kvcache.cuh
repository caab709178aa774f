// Device helpers of the KV-cache kernels: which sequence an item belongs to, where a slot of
// a cache lies, groups of 16 elements, and the 4-bit format (described in include/medusa.h).
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "cache.h"
#include "common.cuh"
#include "f32x2.cuh"

namespace medusa {

constexpr int KV4_SLOTS = 16;                           // slots of a block
__host__ __device__ constexpr int kv4_block(int dh) { return 9 * dh; }   // its bytes

// Sequence (< 0: none) and place within it of item i.  Places are 0 .. rows - 1: an offset outside counts as
// the nearer end, here and in item_count(), so that a sequence has as many items as are found for it.
__device__ __forceinline__ int2 item_of(const ItemMap& m, int B, int i) {
  if (!m.start) {
    const int b = i / m.per_seq, j = i - b * m.per_seq;
    return make_int2(!m.count || j < m.count[b] ? b : -1, j);
  }
  int lo = 0, hi = B;                                   // the last b with start[b] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (m.start[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int s0 = max(m.start[lo], 0);                   // (i < rows)
  return make_int2(i >= s0 && i < m.start[lo + 1] ? lo : -1, i - s0);
}
// Items of sequence b; an offset or a count out of range sets MEDUSA_FLAG_ROW_RANGE.
__device__ __forceinline__ int item_count(const ItemMap& m, int b, uint32_t* status) {
  int n = m.per_seq;
  bool ok = true;
  if (m.start) {
    const int s0 = m.start[b], s1 = m.start[b + 1];
    ok = 0 <= s0 && s0 <= s1 && s1 <= m.rows;
    n = max(min(max(s1, 0), m.rows) - min(max(s0, 0), m.rows), 0);
  } else if (m.count) {
    const int x = m.count[b];
    n = min(max(x, 0), m.per_seq);
    ok = n == x;
  }
  if (!ok) set_flag(status, MEDUSA_FLAG_ROW_RANGE);
  return n;
}

// A length as the calls take it: outside 0..capacity the nearer end.
__device__ __forceinline__ int clamp_len(const CacheView& c, int len) { return min(max(len, 0), c.capacity); }

// Unit (page, or the sequence's whole stretch of a contiguous cache) and slot within it of
// slot t of sequence b; false when the page is outside the pool.
__device__ __forceinline__ bool unit_of(const CacheView& c, int b, int t, long& unit, int& in) {
  if (!c.page_table) {
    unit = b;
    in = t;
    return true;
  }
  const int p = t / c.page_size;
  const int page = c.page_table[(long)b * c.pages_per_seq + p];
  unit = page;
  in = t - p * c.page_size;
  return page >= 0 && page < c.num_pages;
}
// First element of head h in a plain cache, first byte of its block in a 4-bit one.
__device__ __forceinline__ long plain_offset(const CacheView& c, long unit, int in, int h) {
  const int per = c.page_table ? c.page_size : c.capacity;
  return ((unit * per + in) * c.Hkv + h) * c.dh;
}
__device__ __forceinline__ long kv4_offset(const CacheView& c, long unit, int in, int h) {
  const int per = (c.page_table ? c.page_size : c.capacity) / KV4_SLOTS;
  return ((unit * c.Hkv + h) * per + in / KV4_SLOTS) * kv4_block(c.dh);
}

// N consecutive elements (whole 16-byte units), vec: 16-byte aligned.
template <int N> __device__ __forceinline__ void load_n(const bf16* p, bool vec, float (&f)[N]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      float t[8];
      unpack16(reinterpret_cast<const uint4*>(p)[i], t);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[8 * i + e] = t[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = to_f32(p[e]);
  }
}
template <int N> __device__ __forceinline__ void load_n(const float* p, bool vec, float (&f)[N]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p)[i];
      f[4 * i] = t.x; f[4 * i + 1] = t.y; f[4 * i + 2] = t.z; f[4 * i + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = p[e];
  }
}
template <int N> __device__ __forceinline__ void store_n(bf16* p, bool vec, const float (&f)[N]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(pack2(f[8 * i], f[8 * i + 1]), pack2(f[8 * i + 2], f[8 * i + 3]),
                                                  pack2(f[8 * i + 4], f[8 * i + 5]), pack2(f[8 * i + 6], f[8 * i + 7]));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = from_f32<bf16>(f[e]);
  }
}
template <int N> __device__ __forceinline__ void store_n(float* p, bool vec, const float (&f)[N]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = f[e];
  }
}

// Eight floats to a word of e2m1 codes (nearest, ties to even, 6 at most).
__device__ __forceinline__ uint32_t e2m1x8(const float* y) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}
// Magnitude bits of the largest of 16; a NaN stays one, which fmaxf would drop.
__device__ __forceinline__ uint32_t largest_bits(const float (&f)[16]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int e = 1; e < 15; e += 2)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(f[e])), "f"(fabsf(f[e + 1])));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(f[15])));
  return __float_as_uint(m);
}
// What one number's 16-element groups are divided by: for each e4m3 scale byte, s = e4m3 * g and
// its correctly rounded reciprocal (0 for 0), in shared memory; 6 g with its reciprocal; and the bits of
// 448 * 6 g, from which on a group has the largest scale (below infinity's: g is at most 1e20).
struct Kv4Divisors {
  const float2* by_scale;                   // [128] (s, 1/s)
  float six, inv_six;
  uint32_t beyond;
};
__device__ __forceinline__ float2 kv4_divisor(uint32_t byte, float g) {
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3))) * g;
  return make_float2(s, s > 0.f ? __frcp_rn(s) : 0.f);
}
// 16 elements -> 8 bytes of e2m1 pairs and one e4m3 scale.  The scale is the nearest e4m3 to
// max|x| / (6 g), each code the nearest to x / (g s): the correctly rounded quotients, because a
// bf16 element divided by a 4-bit scale is often exactly half way between two codes, and a
// quotient off by one unit in the last place would send it the wrong way.  16 divisions took
// longer than the group's memory traffic, so the quotients come from a correctly rounded
// reciprocal r and Markstein's correction (IBM J. Res. Dev. 34, 1990): q = x r, then
// q + r (x - q s) with the residual exact in one fused multiply-add is the rounded quotient.
// (g lies in 1e-20..1e20, so no residual vanishes where it matters.)  A group whose largest element
// reaches 448 * 6 g has the largest scale whatever its quotient, which may pass a float's range and
// leave the correction infinity minus infinity; its elements are first cut to 8 s, which rounds to the
// largest code.  In any other group s is 0 or |x| < 10 s.
__device__ __forceinline__ bool kv4_encode(const float (&x)[16], const Kv4Divisors& d, uint2& codes, uint8_t& scale) {
  const uint32_t bits = largest_bits(x);
  const float top = __uint_as_float(bits), q = top * d.inv_six;
  scale = __nv_cvt_float_to_fp8(fmaf(fmaf(-q, d.six, top), d.inv_six, q), __NV_SATFINITE, __NV_E4M3);
  float y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = x[e];
  if (bits >= d.beyond) {
    if (bits >= 0x7f800000u) {              // the whole group reads back as NaN
      codes = make_uint2(0x22222222u, 0x22222222u);
      scale = 0x7f;
      return false;
    }
    scale = 0x7e;
    const float most = 8.f * d.by_scale[scale].x;
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = fminf(fmaxf(y[e], -most), most);
  }
  const float2 sr = d.by_scale[scale];
  const F2 s = f2(-sr.x, -sr.x), r = f2(sr.y, sr.y);
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const F2 v = f2(y[e], y[e + 1]), w = mul2(v, r);
    unf2(fma2(fma2(w, s, v), r, w), y[e], y[e + 1]);
  }
  codes = make_uint2(e2m1x8(y), e2m1x8(y + 8));
  return true;
}

// The four bytes of a word, two e2m1 codes each, as halves (exactly).
__device__ __forceinline__ void kv4_pairs(uint32_t w, __half2 (&y)[4]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(y);
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two e4m3 scales as halves.
__device__ __forceinline__ __half2 kv4_scales(uint16_t s) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)s, __NV_E4M3));
}
// An e4m3 scale as a half, exactly (NaN for a group that held none of the numbers).
__device__ __forceinline__ __half kv4_scale(uint8_t s) { return __half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)); }

// What N elements of a group stand for: codes are exact halves, the group's factor is one float.
template <int N> __device__ __forceinline__ void kv4_decode(uint32_t codes, uint8_t scale, float g, float (&f)[N]) {
  const float s = __half2float(kv4_scale(scale)) * g;
  __half2 y[4];
  kv4_pairs(codes, y);
  const F2 s2 = f2(s, s);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float2 v = __half22float2(y[e / 2]);
    unf2(mul2(f2(v.x, v.y), s2), f[e], f[e + 1]);
  }
}

}  // namespace medusa
