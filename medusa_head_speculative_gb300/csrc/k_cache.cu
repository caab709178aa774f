// Appending rows to a KV cache, with the keys' rotation and the 4-bit rounding on the way,
// and reading slots back ("MEDUSA 精读" section 3: only the accepted path stays in the cache;
// section 6: the cache is paged).  Formats and rules: include/medusa.h.
//
// Appending: y = rotate(x, position), then y as it is, or of 16 elements s = e4m3(max|y| / (6 g)) and
// e2m1(y / (g s)) each (kvcache.cuh).  Reading: e2m1 e4m3 g.  A long call is bound by what it moves, but
// for 4-bit appends, which wait for loads: no unit is full (49 % of the issue slots, 27 % of the warps, 53 %
// of the copy rate), with one task fetched ahead and the angles loaded where they are used.  A short call is
// bound by the chain of loads that finds a row's place.  Measured: 32,000 rows of 40 heads of 128 bf16
// elements, keys (turned) and values, into a 4-bit cache (839 MB, 124 us at copy bandwidth) 221 us, 3.8 TB/s;
// 98,000 rows of 8 heads read back as bf16 (519 MB, 76 us) 89 us, 5.8 TB/s; one row in each of 16 sequences
// 3.3 us.
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
  load_n(row + d0, vec, f);
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
// 8 or 16 elements into the cache: at points to them in a plain cache, in a 4-bit one to their
// codes, with sc at their group's scale.
template <int FMT, int N>
__device__ __forceinline__ void put(const CacheView& c, const Kv4Divisors& d, void* at, uint8_t* sc, const float (&f)[N]) {
  if constexpr (FMT == MEDUSA_KV4) {
    uint2 codes;
    uint8_t scale;
    if (!kv4_encode(f, d, codes, scale)) set_flag(c.status, MEDUSA_FLAG_NONFINITE);
    *static_cast<uint2*>(at) = codes;
    *sc = scale;
  } else if constexpr (FMT == MEDUSA_BF16) {
    store_n(static_cast<bf16*>(at), true, f);
  } else {
    store_n(static_cast<float*>(at), true, f);
  }
}
// The block's tables of divisors, for keys and values (4-bit format only).
template <int FMT, int N> __device__ __forceinline__ void fill_divisors(const CacheView& c, float2 (&t)[2][N]) {
  if constexpr (FMT == MEDUSA_KV4) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) t[i >> 7][i & 127] = kv4_divisor(i & 127, i >> 7 ? c.gv : c.gk);
    __syncthreads();
  }
}
template <int N> __device__ __forceinline__ Kv4Divisors divisors_of(const CacheView& c, const float2 (&t)[2][N], bool values) {
  const float six = 6.f * (values ? c.gv : c.gk);
  return {t[values ? 1 : 0], six, __frcp_rn(six), __float_as_uint(448.f * six)};
}
// Byte offset of slot `in` of a unit, head 0: its first element, or its block's first byte.
template <int FMT> __device__ __forceinline__ long slot_bytes(const CacheView& c, long unit, int in) {
  return FMT == MEDUSA_KV4 ? kv4_offset(c, unit, in, 0) : plain_offset(c, unit, in, 0) * (FMT == MEDUSA_BF16 ? 2 : 4);
}
// Bytes from a head to the next.
template <int FMT> __device__ __forceinline__ long head_bytes(const CacheView& c) {
  return FMT == MEDUSA_KV4 ? (long)((c.page_table ? c.page_size : c.capacity) / KV4_SLOTS) * kv4_block(c.dh)
                           : (long)c.dh * (FMT == MEDUSA_BF16 ? 2 : 4);
}
__device__ __forceinline__ int append_length(const CacheView& c, const ItemMap& m, int b) {
  return (int)min((long)clamp_len(c, c.len[b]) + item_count(m, b, c.status), (long)c.capacity);
}
__device__ __forceinline__ void append_lengths(const CacheView& c, const ItemMap& m, long tid, long threads) {
  if (c.len_out == c.len) return;
  for (long b = tid; b < c.B; b += threads)
    c.len_out[b] = append_length(c, m, (int)b);
}

// How warps share rows x (keys, values): a warp takes `places` rows of one kind and every
// slices-th 32 tasks of them, tasks being numbered (head, row, piece of a head): four rows of a
// 4-bit cache fill whole sectors of codes and of scales.
constexpr int KV_PLACES = 8, KV_SHARE_ELEMS = 8192, KV_APPEND_WARPS = 4;
struct WarpShare {
  int places, slices;
};
// Many rows: as many a warp as make 8192 elements of each kind, eight at most, so that finding them
// (three dependent loads, one lane a row) is paid once; few rows: a row over several warps.
// Appending 32,000 rows in 4 bits, us: 8 heads of 128, eight rows a warp 50, four 54, one 70 (blocks of
// eight warps); 40 heads, one 214, eight 256.  8192 rows of 8 heads: several 13, a row over several 18.
// 4096 rows: 11.3 and 11.0.
static WarpShare warp_share(long rows, int row_elems, int tasks) {
  const long wave = 152l * 48;                         // warps that keep the GPU busy
  if (rows * 2 >= 2 * wave) {
    const int places = KV_SHARE_ELEMS / row_elems;
    return {places < 1 ? 1 : places < KV_PLACES ? places : KV_PLACES, 1};
  }
  const int most = (tasks + 31) / 32;
  const long want = wave / (rows * 2 > 0 ? rows * 2 : 1);
  return {1, (int)(want < 1 ? 1 : want < most ? want : most)};
}
// A warp's place in that numbering: task e0 + lane, then every step-th.
struct TaskWalk {
  int u, j, h, du, dj, dh, tasks, places;
  __device__ __forceinline__ TaskWalk(int e, int step, int tasks_, int places_) : tasks(tasks_), places(places_) {
    u = e % tasks;
    j = e / tasks % places;
    h = e / tasks / places;
    du = step % tasks;
    dj = step / tasks % places;
    dh = step / tasks / places;
  }
  __device__ __forceinline__ void next() {
    u += du;
    j += dj;
    h += dh;
    if (u >= tasks) { u -= tasks; ++j; }
    if (j >= places) { j -= places; ++h; }
  }
};
// A row found: its elements outside the cache, its slot in it (head 0: elements, or codes and
// scales), its angles.  Heads are less than 2^31 bytes apart everywhere (checked by the caller).
struct PlaceInfo {
  char* rows;             // null: no such row
  char* at;
  char* sc;
  const float* cs;
};
template <int FMT>
__device__ __forceinline__ PlaceInfo place_info(const CacheView& c, const void* pool, long unit, int in) {
  PlaceInfo p;
  p.rows = nullptr;
  p.cs = nullptr;
  p.at = const_cast<char*>(static_cast<const char*>(pool)) + slot_bytes<FMT>(c, unit, in);
  p.sc = p.at + 8 * c.dh + in % KV4_SLOTS * (c.dh / 16);
  if (FMT == MEDUSA_KV4) p.at += in % KV4_SLOTS * (c.dh / 2);
  return p;
}

// Two pairs turned: (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), each operation rounded by itself.
__device__ __forceinline__ void turn2(F2 c, F2 s, float* x1, float* x2) {
  const F2 a = f2(x1[0], x1[1]), b = f2(x2[0], x2[1]);
  unf2(fma2(mul2(b, s), f2(-1.f, -1.f), mul2(a, c)), x1[0], x1[1]);
  unf2(add2(mul2(b, c), mul2(a, s)), x2[0], x2[1]);
}
template <int N> struct Raw16 {
  uint4 v[N];
};
template <typename T, int N> __device__ __forceinline__ void load_raw(const char* p, Raw16<N * sizeof(T) / 16>& r) {
#pragma unroll
  for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
}
template <typename T, int N> __device__ __forceinline__ void unpack_raw(const Raw16<N * sizeof(T) / 16>& r, float (&f)[N]) {
  constexpr int E = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < N / E; ++i) {
    float t[E];
    unpack16(r.v[i], t);
#pragma unroll
    for (int e = 0; e < E; ++e) f[E * i + e] = t[e];
  }
}

// Aligned rows whose rotation pairs whole groups of 16 elements (HALF with rot a multiple of
// 32, or INTERLEAVED with rot one of 16, or none).  A task is N elements of a head, with HALF
// together with their partners, so that every key and angle is read once: a group of 16 for the
// 4-bit format, 8 for the others (whole 16 or 32 bytes written by neighbouring lanes).  The next
// task's elements are under way while one is encoded.  Blocks of four warps, five to an SM: 96
// registers, which the encoding needs (three blocks of eight: 80, with spills, 57 us where this takes 50;
// four to an SM, 62).  Copying three tasks ahead to shared memory instead was slower (61).
template <typename T, int FMT>
__global__ void __launch_bounds__(KV_APPEND_WARPS * 32, 5) kv_append_vec_kernel(const __grid_constant__ AppendArgs a, const WarpShare ws) {
  constexpr int N = FMT == MEDUSA_KV4 ? 16 : 8, ES = FMT == MEDUSA_F32 ? 4 : 2;
  using Raw = Raw16<N * sizeof(T) / 16>;
  __shared__ PlaceInfo info[KV_APPEND_WARPS][KV_PLACES];
  __shared__ float2 table[2][FMT == MEDUSA_KV4 ? 128 : 1];
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h2 = a.t.rot / 2;
  fill_divisors<FMT>(c, table);
  append_lengths(c, a.m, (long)blockIdx.x * blockDim.x + threadIdx.x, (long)gridDim.x * blockDim.x);
  long wid = (long)blockIdx.x * KV_APPEND_WARPS + warp;
  const int slice = (int)(wid % ws.slices);
  wid /= ws.slices;
  const bool values = wid & 1;
  if ((wid >> 1) * ws.places >= a.m.rows) return;
  const int i0 = (int)(wid >> 1) * ws.places;
  if (lane < ws.places) {
    const bool lead = !values && slice == 0;
    PlaceInfo p{};
    Target o;
    if (lane < a.m.rows - i0 && append_target(a, i0 + lane, item_of(a.m, c.B, i0 + lane), lead, o)) {
      p = place_info<FMT>(c, values ? c.v : c.k, o.unit, o.in);
      p.rows = const_cast<char*>(static_cast<const char*>(values ? a.v : a.k)) +
               o.row * (values ? a.v_row : a.k_row) * (long)sizeof(T);
      if (!values) p.cs = append_angles(a, i0 + lane, o.t, lead);
    }
    info[warp][lane] = p;
  }
  __syncwarp();
  const int head_b = (int)((values ? a.v_head : a.k_head) * (long)sizeof(T)), step = (int)head_bytes<FMT>(c);
  // tasks of a row's head: pairs of pieces (rows that are not turned copy both), then single ones
  const bool half = a.turn && !values && a.t.layout == MEDUSA_ROPE_HALF;
  const int pairs = half ? h2 / N : 0, tasks = c.dh / N - pairs;
  const Kv4Divisors dv = divisors_of(c, table, values);
  TaskWalk w(32 * slice + lane, 32 * ws.slices, tasks, ws.places);
  Raw ahead, ahead2;
  auto fetch = [&]() {                     // the task's elements, if there is such a task
    while (w.h < c.Hkv && !info[warp][w.j].rows) w.next();
    if (w.h >= c.Hkv) return;
    const char* x = info[warp][w.j].rows + (long)w.h * head_b + N * (int)sizeof(T) * (w.u < pairs ? w.u : w.u + pairs);
    load_raw<T, N>(x, ahead);
    if (w.u < pairs) load_raw<T, N>(x + h2 * sizeof(T), ahead2);
  };
  fetch();
  while (w.h < c.Hkv) {
    const PlaceInfo& p = info[warp][w.j];
    const bool paired = w.u < pairs;
    const int d0 = N * (paired ? w.u : w.u + pairs);
    char* at = p.at + (long)w.h * step + (FMT == MEDUSA_KV4 ? d0 / 2 : d0 * ES);
    uint8_t* sc = reinterpret_cast<uint8_t*>(p.sc) + (long)w.h * step + d0 / 16;      // 4-bit only
    const float* cs = p.cs;
    float f[N], g[N];
    unpack_raw<T, N>(ahead, f);
    if (paired) unpack_raw<T, N>(ahead2, g);
    w.next();
    fetch();
    if (paired) {
      if (cs) {
#pragma unroll
        for (int k4 = 0; k4 < N; k4 += 4) {
          float ck[4], sk[4];
          load_n(cs + d0 + k4, true, ck);
          load_n(cs + h2 + d0 + k4, true, sk);
#pragma unroll
          for (int k = 0; k < 4; k += 2) turn2(f2(ck[k], ck[k + 1]), f2(sk[k], sk[k + 1]), f + k4 + k, g + k4 + k);
        }
      }
      put<FMT, N>(c, dv, at + (FMT == MEDUSA_KV4 ? h2 / 2 : h2 * ES), sc + h2 / 16, g);
    } else if (cs && !half && d0 < a.t.rot) {
      float ck[N / 2], sk[N / 2];
      load_n(cs + d0 / 2, true, ck);
      load_n(cs + h2 + d0 / 2, true, sk);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const float x1 = f[k], x2 = f[k + 1];
        f[k] = __fsub_rn(__fmul_rn(x1, ck[k / 2]), __fmul_rn(x2, sk[k / 2]));
        f[k + 1] = __fadd_rn(__fmul_rn(x2, ck[k / 2]), __fmul_rn(x1, sk[k / 2]));
      }
    }
    put<FMT, N>(c, dv, at, sc, f);
  }
}

// Any alignment and any rotation: one thread per (item, keys or values, head, 16 elements).
template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 table[2][FMT == MEDUSA_KV4 ? 128 : 1];
  const CacheView& c = a.c;
  fill_divisors<FMT>(c, table);
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
      load_n(static_cast<const T*>(a.v) + o.row * a.v_row + h * a.v_head + grp * 16, a.vec, f);
    } else {
      const float* cs = append_angles(a, i, o.t, lead);
      load_turned(static_cast<const T*>(a.k) + o.row * a.k_row + h * a.k_head, grp * 16, a.vec, a.t, cs, f);
    }
    char* at = static_cast<char*>(values ? c.v : c.k) + slot_bytes<FMT>(c, o.unit, o.in) + h * head_bytes<FMT>(c);
    const int slot = o.in % KV4_SLOTS;
    uint8_t* sc = reinterpret_cast<uint8_t*>(at) + 8 * c.dh + slot * groups + grp;
    at += FMT == MEDUSA_KV4 ? slot * (c.dh / 2) + grp * 8 : grp * (FMT == MEDUSA_BF16 ? 32 : 64);
    put<FMT, 16>(c, divisors_of(c, table, values), at, sc, f);
  }
}

// len_out where it is len itself: after the rows, which are placed by the old lengths.
__global__ void kv_length_kernel(CacheView c, ItemMap m) {
  pdl_wait();
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < c.B; b += gridDim.x * blockDim.x)
    c.len_out[b] = append_length(c, m, b);
}

// The kernel for aligned rows against the other (4-bit, 8 heads of 128, us): 16 rows 3.7 / 4.5, 4096 rows
// 10.9 / 15.4, 32,000 rows 50 / 103.
template <typename T>
static cudaError_t append_go(const AppendArgs& a, int format, cudaStream_t st) {
  if (a.vec && (!a.turn || a.t.rot % (a.t.layout == MEDUSA_ROPE_HALF ? 32 : 16) == 0)) {
    auto kern = format == MEDUSA_KV4 ? kv_append_vec_kernel<T, MEDUSA_KV4>
                : format == MEDUSA_BF16 ? kv_append_vec_kernel<T, MEDUSA_BF16> : kv_append_vec_kernel<T, MEDUSA_F32>;
    const WarpShare ws = warp_share(a.m.rows, a.c.Hkv * a.c.dh, a.c.Hkv * (a.c.dh / (format == MEDUSA_KV4 ? 16 : 8)));
    const long warps = ((long)a.m.rows + ws.places - 1) / ws.places * 2 * ws.slices;
    return launch_kernel(kern, dim3((unsigned)(warps < 1 ? 1 : (warps + KV_APPEND_WARPS - 1) / KV_APPEND_WARPS)), dim3(KV_APPEND_WARPS * 32), 0, st, 1, a, ws);
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

// A task is 16 bytes of the result; a lane has UNROLL of them under way.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ ReadArgs a, const WarpShare ws) {
  constexpr int N = 16 / sizeof(T), UNROLL = 4, ES = FMT == MEDUSA_F32 ? 4 : 2;
  __shared__ PlaceInfo info[8][KV_PLACES];
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long b = (long)blockIdx.x * blockDim.x + threadIdx.x; b < c.B; b += (long)gridDim.x * blockDim.x)
    item_count(a.m, (int)b, c.status);      // reports what is out of range
  long wid = (long)blockIdx.x * 8 + warp;
  const int slice = (int)(wid % ws.slices);
  wid /= ws.slices;
  const bool values = wid & 1;
  if ((wid >> 1) * ws.places >= a.m.rows) return;
  const int i0 = (int)(wid >> 1) * ws.places;
  if (lane < ws.places) {
    PlaceInfo p{};
    const int2 it = lane < a.m.rows - i0 ? item_of(a.m, c.B, i0 + lane) : make_int2(-1, 0);
    if (it.x >= 0) {
      const long t = (long)it.y + (a.first ? a.first[it.x] : 0);
      long unit;
      int in;
      uint32_t flag = 0;
      if (t < 0 || t >= clamp_len(c, c.len[it.x])) flag = MEDUSA_FLAG_KV_CAPACITY;
      else if (!unit_of(c, it.x, (int)t, unit, in)) flag = MEDUSA_FLAG_PAGE_RANGE;
      if (flag) {
        if (!values && slice == 0) set_flag(c.status, flag);
      } else {
        p = place_info<FMT>(c, values ? c.v : c.k, unit, in);
        p.rows = static_cast<char*>(values ? a.v : a.k) + (long)(i0 + lane) * (values ? a.v_row : a.k_row) * (long)sizeof(T);
      }
    }
    info[warp][lane] = p;
  }
  __syncwarp();
  const int head_b = (int)((values ? a.v_head : a.k_head) * (long)sizeof(T)), step = (int)head_bytes<FMT>(c);
  const float g = values ? c.gv : c.gk;
  TaskWalk w(32 * slice + lane, 32 * ws.slices, c.dh / N, ws.places);
  while (w.h < c.Hkv) {
    uint32_t codes[UNROLL];
    uint8_t scale[UNROLL];
    float f[UNROLL][N];
    T* dst[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u, w.next()) {
      dst[u] = nullptr;
      if (w.h >= c.Hkv) continue;
      const PlaceInfo& p = info[warp][w.j];
      if (!p.rows) continue;
      const int d0 = w.u * N;
      const char* at = p.at + (long)w.h * step;
      dst[u] = reinterpret_cast<T*>(p.rows + (long)w.h * head_b) + d0;
      if (FMT == MEDUSA_KV4) {
        codes[u] = N == 8 ? *reinterpret_cast<const uint32_t*>(at + d0 / 2) : *reinterpret_cast<const uint16_t*>(at + d0 / 2);
        scale[u] = static_cast<uint8_t>(p.sc[(long)w.h * step + d0 / 16]);
      } else if (FMT == MEDUSA_BF16) {
        load_n(reinterpret_cast<const bf16*>(at + d0 * ES), N == 8, f[u]);
      } else {
        load_n(reinterpret_cast<const float*>(at + d0 * ES), true, f[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (!dst[u]) continue;
      if (FMT == MEDUSA_KV4) kv4_decode<N>(codes[u], scale[u], g, f[u]);
      store_n(dst[u], a.vec, f[u]);
    }
  }
}

template <typename T>
static cudaError_t read_go(const ReadArgs& a, int format, cudaStream_t st) {
  const WarpShare ws = warp_share(a.m.rows, a.c.Hkv * a.c.dh, a.c.Hkv * a.c.dh * (int)sizeof(T) / 16);
  const long warps = ((long)a.m.rows + ws.places - 1) / ws.places * 2 * ws.slices;
  auto kern = format == MEDUSA_KV4 ? kv_read_kernel<T, MEDUSA_KV4>
              : format == MEDUSA_BF16 ? kv_read_kernel<T, MEDUSA_BF16> : kv_read_kernel<T, MEDUSA_F32>;
  return launch_kernel(kern, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, 1, a, ws);
}

cudaError_t launch_kv_read(const ReadArgs& a, int dst_dtype, int format, cudaStream_t st) {
  return dst_dtype == MEDUSA_F32 ? read_go<float>(a, format, st) : read_go<bf16>(a, format, st);
}

}  // namespace medusa
