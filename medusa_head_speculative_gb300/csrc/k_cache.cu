// Appending rows to a KV cache, with the keys' rotation and the 4-bit rounding on the way,
// and reading slots back ("MEDUSA 精读" section 3: only the accepted path stays in the cache;
// section 6: the cache is paged).  Formats and rules: include/medusa.h.
#include "cache.h"
#include "common.cuh"
#include "kvcache.cuh"
#include "launch.cuh"

namespace medusa {

// 16 elements of a row from element d0 on, turned by the angles cs ([rot/2] cosines, then
// [rot/2] sines) where they lie below rot; the operations are those of k_rope.cu.
template <typename T>
__device__ __forceinline__ void load_turned(const T* row, int d0, bool vec, const RopeTable& t, const float* cs,
                                            float (&f)[16]) {
  load16(row + d0, vec, f);
  if (!cs || d0 >= t.rot) return;
  const int h = t.rot / 2;
  if (t.layout == MEDUSA_ROPE_HALF) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = d0 + e;
      if (d >= t.rot) continue;
      const bool first = d < h;
      const float o = to_f32(row[first ? d + h : d - h]);
      const float c = cs[first ? d : d - h], s = cs[first ? h + d : d];
      f[e] = first ? __fsub_rn(__fmul_rn(f[e], c), __fmul_rn(o, s)) : __fadd_rn(__fmul_rn(f[e], c), __fmul_rn(o, s));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const int d = d0 + e;
      if (d >= t.rot) continue;
      const float c = cs[d / 2], s = cs[h + d / 2], x1 = f[e], x2 = f[e + 1];
      f[e] = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
      f[e + 1] = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    }
  }
}

// One thread per (item, keys or values, head, 16 elements).
template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  const CacheView& c = a.c;
  const int groups = c.dh / 16;
  const long tid = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c.len_out != c.len)
    for (long b = tid; b < c.B; b += (long)gridDim.x * blockDim.x)
      c.len_out[b] = min(clamp_len(c, c.len[b]) + item_count(a.m, (int)b), c.capacity);
  const long n = (long)a.m.rows * 2 * c.Hkv * groups;
  for (long e = tid; e < n; e += (long)gridDim.x * blockDim.x) {
    const int grp = (int)(e % groups);
    long r = e / groups;
    const int h = (int)(r % c.Hkv);
    r /= c.Hkv;
    const int part = (int)(r & 1);
    const int i = (int)(r >> 1);
    const int2 it = item_of(a.m, c.B, i);
    if (it.x < 0) continue;
    const int len = c.len[it.x], t = clamp_len(c, len) + it.y;
    const bool lead = part == 0 && h == 0 && grp == 0;
    if (lead && len != clamp_len(c, len)) set_flag(c.status, MEDUSA_FLAG_KV_CAPACITY);
    if (t >= c.capacity) {
      if (lead) set_flag(c.status, MEDUSA_FLAG_KV_CAPACITY);
      continue;
    }
    long row = i;
    if (a.index) {
      const int x = a.index[i];
      if (x < 0 || x >= a.index_rows) {
        if (lead) set_flag(c.status, MEDUSA_FLAG_ROW_RANGE);
        continue;
      }
      row = (long)it.x * a.index_rows + x;
    }
    long unit;
    int in;
    if (!unit_of(c, it.x, t, unit, in)) {
      if (lead) set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
      continue;
    }
    float f[16];
    if (part == 0) {
      const float* cs = nullptr;
      if (a.turn) {
        const int pos = a.pos ? a.pos[i] : t;
        if (pos >= 0 && pos < a.t.max_pos) cs = a.t.cs + (long)pos * a.t.rot;
        else if (lead) set_flag(c.status, MEDUSA_FLAG_POS_RANGE);
      }
      load_turned(static_cast<const T*>(a.k) + row * a.k_row + h * a.k_head, grp * 16, a.vec, a.t, cs, f);
    } else {
      load16(static_cast<const T*>(a.v) + row * a.v_row + h * a.v_head + grp * 16, a.vec, f);
    }
    if (FMT == MEDUSA_KV4) {
      uint8_t* block = static_cast<uint8_t*>(part ? c.v : c.k) + kv4_offset(c, unit, in, h);
      const int slot = in % KV4_SLOTS;
      uint2 codes;
      uint8_t scale;
      if (!kv4_encode(f, part ? c.gv : c.gk, codes, scale)) set_flag(c.status, MEDUSA_FLAG_NONFINITE);
      *reinterpret_cast<uint2*>(block + slot * (c.dh / 2) + grp * 8) = codes;
      block[8 * c.dh + slot * groups + grp] = scale;
    } else if (FMT == MEDUSA_BF16) {
      store16(static_cast<bf16*>(part ? c.v : c.k) + plain_offset(c, unit, in, h) + grp * 16, true, f);
    } else {
      store16(static_cast<float*>(part ? c.v : c.k) + plain_offset(c, unit, in, h) + grp * 16, true, f);
    }
  }
}

// len_out where it is len itself: after the rows, which are placed by the old lengths.
__global__ void kv_length_kernel(CacheView c, ItemMap m) {
  pdl_wait();
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < c.B; b += gridDim.x * blockDim.x)
    c.len_out[b] = min(clamp_len(c, c.len[b]) + item_count(m, b), c.capacity);
}

template <typename T>
static cudaError_t append_go(const AppendArgs& a, int format, cudaStream_t st) {
  const long n = (long)a.m.rows * 2 * a.c.Hkv * (a.c.dh / 16);
  const long want = (n + 255) / 256;
  const int blocks = (int)(want < 1 ? 1 : want < (1 << 20) ? want : (1 << 20));
  auto kern = format == MEDUSA_KV4 ? kv_append_kernel<T, MEDUSA_KV4>
              : format == MEDUSA_BF16 ? kv_append_kernel<T, MEDUSA_BF16> : kv_append_kernel<T, MEDUSA_F32>;
  return launch_kernel(kern, dim3(blocks), dim3(256), 0, st, 1, a);
}

cudaError_t launch_kv_append(const AppendArgs& a, int src_dtype, int format, cudaStream_t st) {
  cudaError_t e = src_dtype == MEDUSA_F32 ? append_go<float>(a, format, st) : append_go<bf16>(a, format, st);
  if (e != cudaSuccess || a.c.len_out != a.c.len) return e;
  return launch_kernel(kv_length_kernel, dim3((a.c.B + 255) / 256), dim3(256), 0, st, 1, a.c, a.m);
}

template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ ReadArgs a) {
  const CacheView& c = a.c;
  const int groups = c.dh / 16;
  const long n = (long)a.m.rows * 2 * c.Hkv * groups;
  for (long e = (long)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (long)gridDim.x * blockDim.x) {
    const int grp = (int)(e % groups);
    long r = e / groups;
    const int h = (int)(r % c.Hkv);
    r /= c.Hkv;
    const int part = (int)(r & 1);
    const int i = (int)(r >> 1);
    const int2 it = item_of(a.m, c.B, i);
    if (it.x < 0) continue;
    const long t = (long)it.y + (a.first ? a.first[it.x] : 0);
    const bool lead = part == 0 && h == 0 && grp == 0;
    if (t < 0 || t >= clamp_len(c, c.len[it.x])) {
      if (lead) set_flag(c.status, MEDUSA_FLAG_KV_CAPACITY);
      continue;
    }
    long unit;
    int in;
    if (!unit_of(c, it.x, (int)t, unit, in)) {
      if (lead) set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
      continue;
    }
    float f[16];
    if (FMT == MEDUSA_KV4) {
      const uint8_t* block = static_cast<const uint8_t*>(part ? c.v : c.k) + kv4_offset(c, unit, in, h);
      const int slot = in % KV4_SLOTS;
      kv4_decode(*reinterpret_cast<const uint2*>(block + slot * (c.dh / 2) + grp * 8),
                 block[8 * c.dh + slot * groups + grp], part ? c.gv : c.gk, f);
    } else if (FMT == MEDUSA_BF16) {
      load16(static_cast<const bf16*>(part ? c.v : c.k) + plain_offset(c, unit, in, h) + grp * 16, true, f);
    } else {
      load16(static_cast<const float*>(part ? c.v : c.k) + plain_offset(c, unit, in, h) + grp * 16, true, f);
    }
    T* dst = part ? static_cast<T*>(a.v) + i * a.v_row + h * a.v_head : static_cast<T*>(a.k) + i * a.k_row + h * a.k_head;
    store16(dst + grp * 16, a.vec, f);
  }
}

template <typename T>
static cudaError_t read_go(const ReadArgs& a, int format, cudaStream_t st) {
  const long n = (long)a.m.rows * 2 * a.c.Hkv * (a.c.dh / 16);
  const long want = (n + 255) / 256;
  const int blocks = (int)(want < (1 << 20) ? want : (1 << 20));
  auto kern = format == MEDUSA_KV4 ? kv_read_kernel<T, MEDUSA_KV4>
              : format == MEDUSA_BF16 ? kv_read_kernel<T, MEDUSA_BF16> : kv_read_kernel<T, MEDUSA_F32>;
  return launch_kernel(kern, dim3(blocks), dim3(256), 0, st, 1, a);
}

cudaError_t launch_kv_read(const ReadArgs& a, int dst_dtype, int format, cudaStream_t st) {
  return dst_dtype == MEDUSA_F32 ? read_go<float>(a, format, st) : read_go<bf16>(a, format, st);
}

}  // namespace medusa
