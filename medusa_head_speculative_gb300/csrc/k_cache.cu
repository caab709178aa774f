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

// Where item i goes: sequence it.x, slot t, unit and slot in it, source row.  False: nowhere
// (reported by the lead thread).
struct Target {
  int t, in;
  long unit, row;
};
__device__ __forceinline__ bool append_target(const AppendArgs& a, int i, int2 it, bool lead, Target& o) {
  const CacheView& c = a.c;
  if (it.x < 0) return false;
  const int len = c.len[it.x], base = clamp_len(c, len);
  const long t = (long)base + it.y;
  uint32_t flag = len != base ? MEDUSA_FLAG_KV_CAPACITY : 0u;
  bool ok = true;
  o.row = i;
  if (t >= c.capacity) {
    flag |= MEDUSA_FLAG_KV_CAPACITY;
    ok = false;
  } else {
    o.t = (int)t;
    if (a.index) {
      const int x = a.index[i];
      o.row = (long)it.x * a.index_rows + x;
      if (x < 0 || x >= a.index_rows) {
        flag |= MEDUSA_FLAG_ROW_RANGE;
        ok = false;
      }
    }
    if (ok && !unit_of(c, it.x, o.t, o.unit, o.in)) {
      flag |= MEDUSA_FLAG_PAGE_RANGE;
      ok = false;
    }
  }
  if (flag && lead) set_flag(c.status, flag);
  return ok;
}
// The item's row of angles (null: not turned).
__device__ __forceinline__ const float* append_angles(const AppendArgs& a, int i, int t, bool lead) {
  if (!a.turn) return nullptr;
  const int pos = a.pos ? a.pos[i] : t;
  if (pos >= 0 && pos < a.t.max_pos) return a.t.cs + (long)pos * a.t.rot;
  if (lead) set_flag(a.c.status, MEDUSA_FLAG_POS_RANGE);
  return nullptr;
}
// 16 elements of head h from element 16 grp on into the cache.
template <int FMT>
__device__ __forceinline__ void put16(const CacheView& c, bool values, const Target& o, int h, int grp, float (&f)[16]) {
  if (FMT == MEDUSA_KV4) {
    uint8_t* block = static_cast<uint8_t*>(values ? c.v : c.k) + kv4_offset(c, o.unit, o.in, h);
    const int slot = o.in % KV4_SLOTS;
    uint2 codes;
    uint8_t scale;
    if (!kv4_encode(f, values ? c.gv : c.gk, codes, scale)) set_flag(c.status, MEDUSA_FLAG_NONFINITE);
    *reinterpret_cast<uint2*>(block + slot * (c.dh / 2) + grp * 8) = codes;
    block[8 * c.dh + slot * (c.dh / 16) + grp] = scale;
  } else if (FMT == MEDUSA_BF16) {
    store16(static_cast<bf16*>(values ? c.v : c.k) + plain_offset(c, o.unit, o.in, h) + grp * 16, true, f);
  } else {
    store16(static_cast<float*>(values ? c.v : c.k) + plain_offset(c, o.unit, o.in, h) + grp * 16, true, f);
  }
}
__device__ __forceinline__ void append_lengths(const CacheView& c, const ItemMap& m, long tid, long threads) {
  if (c.len_out == c.len) return;
  for (long b = tid; b < c.B; b += threads)
    c.len_out[b] = min(clamp_len(c, c.len[b]) + item_count(m, (int)b), c.capacity);
}

// 16 angles of a row of the table from pair p0 on.
__device__ __forceinline__ void load_angles(const float* cs, int p0, int h, float (&c)[16], float (&s)[16]) {
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const float4 x = *reinterpret_cast<const float4*>(cs + p0 + e), y = *reinterpret_cast<const float4*>(cs + h + p0 + e);
    c[e] = x.x; c[e + 1] = x.y; c[e + 2] = x.z; c[e + 3] = x.w;
    s[e] = y.x; s[e + 1] = y.y; s[e + 2] = y.z; s[e + 3] = y.w;
  }
}

// Aligned rows whose rotation pairs whole groups of 16 elements (HALF with rot a multiple of
// 32, or INTERLEAVED with rot one of 16, or none): a warp takes one item's keys or its values,
// found once for the warp, and its lanes go over the heads' groups; with HALF a lane takes a
// group and its partner, so that every key and angle is read once.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_append_vec_kernel(const __grid_constant__ AppendArgs a) {
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, groups = c.dh / 16, h2 = a.t.rot / 2;
  append_lengths(c, a.m, (long)blockIdx.x * blockDim.x + threadIdx.x, (long)gridDim.x * blockDim.x);
  const long wid = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int i = (int)(wid >> 1);
  const bool values = wid & 1;
  if (i >= a.m.rows) return;
  const int2 it = item_of_warp(a.m, c.B, i);
  Target o;
  const bool lead = lane == 0 && !values;
  if (!append_target(a, i, it, lead, o)) return;
  const T* src = values ? static_cast<const T*>(a.v) + o.row * a.v_row : static_cast<const T*>(a.k) + o.row * a.k_row;
  const long head = values ? a.v_head : a.k_head;
  const float* cs = values ? nullptr : append_angles(a, i, o.t, lead);
  const bool half = cs && a.t.layout == MEDUSA_ROPE_HALF;
  // tasks of a head: pairs of groups, then single groups
  const int pairs = half ? a.t.rot / 32 : 0, tasks = half ? groups - pairs : groups;
  const int n = c.Hkv * tasks;
  for (int e = lane; e < n; e += 32) {
    const int h = e / tasks, u = e - h * tasks;
    const T* row = src + h * head;
    const int g0 = u < pairs ? u : pairs + u;
    float f[16];
    load16(row + g0 * 16, true, f);
    if (u < pairs) {
      float f2[16], cc[16], ss[16];
      load16(row + g0 * 16 + h2, true, f2);
      load_angles(cs, g0 * 16, h2, cc, ss);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float x1 = f[k], x2 = f2[k];
        f[k] = __fsub_rn(__fmul_rn(x1, cc[k]), __fmul_rn(x2, ss[k]));
        f2[k] = __fadd_rn(__fmul_rn(x2, cc[k]), __fmul_rn(x1, ss[k]));
      }
      put16<FMT>(c, values, o, h, g0 + pairs, f2);
    } else if (cs && !half && g0 * 16 < a.t.rot) {
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float ck = cs[g0 * 8 + k / 2], sk = cs[h2 + g0 * 8 + k / 2], x1 = f[k], x2 = f[k + 1];
        f[k] = __fsub_rn(__fmul_rn(x1, ck), __fmul_rn(x2, sk));
        f[k + 1] = __fadd_rn(__fmul_rn(x2, ck), __fmul_rn(x1, sk));
      }
    }
    put16<FMT>(c, values, o, h, g0, f);
  }
}

// Any alignment and any rotation: one thread per (item, keys or values, head, 16 elements).
template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  const CacheView& c = a.c;
  const int groups = c.dh / 16;
  const long tid = (long)blockIdx.x * blockDim.x + threadIdx.x;
  append_lengths(c, a.m, tid, (long)gridDim.x * blockDim.x);
  const long n = (long)a.m.rows * 2 * c.Hkv * groups;
  for (long e = tid; e < n; e += (long)gridDim.x * blockDim.x) {
    const int grp = (int)(e % groups);
    long r = e / groups;
    const int h = (int)(r % c.Hkv);
    r /= c.Hkv;
    const bool values = r & 1;
    const int i = (int)(r >> 1);
    Target o;
    const bool lead = !values && h == 0 && grp == 0;
    if (!append_target(a, i, item_of(a.m, c.B, i), lead, o)) continue;
    float f[16];
    if (values) {
      load16(static_cast<const T*>(a.v) + o.row * a.v_row + h * a.v_head + grp * 16, a.vec, f);
    } else {
      const float* cs = append_angles(a, i, o.t, lead);
      load_turned(static_cast<const T*>(a.k) + o.row * a.k_row + h * a.k_head, grp * 16, a.vec, a.t, cs, f);
    }
    put16<FMT>(c, values, o, h, grp, f);
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
  if (a.vec && (!a.turn || a.t.rot % (a.t.layout == MEDUSA_ROPE_HALF ? 32 : 16) == 0)) {
    auto kern = format == MEDUSA_KV4 ? kv_append_vec_kernel<T, MEDUSA_KV4>
                : format == MEDUSA_BF16 ? kv_append_vec_kernel<T, MEDUSA_BF16> : kv_append_vec_kernel<T, MEDUSA_F32>;
    const unsigned ctas = (unsigned)(((long)a.m.rows * 2 + 7) / 8);
    return launch_kernel(kern, dim3(ctas ? ctas : 1), dim3(256), 0, st, 1, a);
  }
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

// A warp takes one place's keys or its values, found once for the warp; its lanes go over the
// heads' groups of 16 elements, UNROLL at a time with all loads before the first use.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int UNROLL = FMT == MEDUSA_KV4 ? 4 : 1;
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, groups = c.dh / 16;
  const long wid = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int i = (int)(wid >> 1);
  const bool values = wid & 1;
  if (i >= a.m.rows) return;
  const int2 it = item_of_warp(a.m, c.B, i);
  if (it.x < 0) return;
  const long t = (long)it.y + (a.first ? a.first[it.x] : 0);
  uint32_t flag = 0;
  long unit = 0;
  int in = 0;
  if (t < 0 || t >= clamp_len(c, c.len[it.x])) flag = MEDUSA_FLAG_KV_CAPACITY;
  else if (!unit_of(c, it.x, (int)t, unit, in)) flag = MEDUSA_FLAG_PAGE_RANGE;
  if (flag) {
    if (lane == 0) set_flag(c.status, flag);
    return;
  }
  T* dst = values ? static_cast<T*>(a.v) + i * a.v_row : static_cast<T*>(a.k) + i * a.k_row;
  const long head = values ? a.v_head : a.k_head;
  const void* pool = values ? c.v : c.k;
  const float g = values ? c.gv : c.gk;
  const int n = c.Hkv * groups, slot = in % KV4_SLOTS;
  const uint8_t* block0 = static_cast<const uint8_t*>(pool) + kv4_offset(c, unit, in, 0);
  const long step = (long)((c.page_table ? c.page_size : c.capacity) / KV4_SLOTS) * kv4_block(c.dh);   // to the next head
  for (int e0 = lane; e0 < n; e0 += 32 * UNROLL) {
    uint2 codes[UNROLL];
    uint8_t scale[UNROLL];
    if (FMT == MEDUSA_KV4) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int e = e0 + 32 * u, h = e / groups, grp = e - h * groups;
        if (e >= n) break;
        const uint8_t* block = block0 + h * step;
        codes[u] = *reinterpret_cast<const uint2*>(block + slot * (c.dh / 2) + grp * 8);
        scale[u] = block[8 * c.dh + slot * groups + grp];
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int e = e0 + 32 * u, h = e / groups, grp = e - h * groups;
      if (e >= n) break;
      float f[16];
      if (FMT == MEDUSA_KV4) kv4_decode(codes[u], scale[u], g, f);
      else if (FMT == MEDUSA_BF16) load16(static_cast<const bf16*>(pool) + plain_offset(c, unit, in, h) + grp * 16, true, f);
      else load16(static_cast<const float*>(pool) + plain_offset(c, unit, in, h) + grp * 16, true, f);
      store16(dst + h * head + grp * 16, a.vec, f);
    }
  }
}

template <typename T>
static cudaError_t read_go(const ReadArgs& a, int format, cudaStream_t st) {
  const unsigned ctas = (unsigned)(((long)a.m.rows * 2 + 7) / 8);
  auto kern = format == MEDUSA_KV4 ? kv_read_kernel<T, MEDUSA_KV4>
              : format == MEDUSA_BF16 ? kv_read_kernel<T, MEDUSA_BF16> : kv_read_kernel<T, MEDUSA_F32>;
  return launch_kernel(kern, dim3(ctas), dim3(256), 0, st, 1, a);
}

cudaError_t launch_kv_read(const ReadArgs& a, int dst_dtype, int format, cudaStream_t st) {
  return dst_dtype == MEDUSA_F32 ? read_go<float>(a, format, st) : read_go<bf16>(a, format, st);
}

}  // namespace medusa
