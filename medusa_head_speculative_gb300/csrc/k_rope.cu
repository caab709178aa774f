// Rotary positions: the table of cosines and sines, and the rotation of query / key rows
// ("Medusa: Simple LLM Inference Acceleration Framework with Multiple Decoding Heads" §3.4
// Tree Attention Step 4: a node's position is the prefix length plus its depth).
//
// y1 = x1 c - x2 s, y2 = x2 c + x1 s with every product and sum rounded by itself (no fused
// multiply-add), so that the result depends on the inputs alone and not on how a kernel
// groups the operations: medusa_kv_append quantises the same values.
//
// Bound by what it moves.  Measured: 16,381 rows of 40 heads of 128 bf16 elements, 64 of them turned
// (340 MB, 50 us at copy bandwidth) 57 us, 5.9 TB/s; 65 rows of 64 heads 2.1 us (latency).  Units of 16
// bytes where alignment and rot allow, of 8 for the bf16 rows that allow only these (halves of 36
// elements, 16,384 rows of 40 heads: 98 us), single elements for the rest (394 us there).
#include "cache.h"
#include "common.cuh"
#include "launch.cuh"

namespace medusa {

__global__ void rope_fill_kernel(float* cs, const double* freq, int rot, int max_pos, double attn) {
  const int h = rot / 2;
  const long n = (long)max_pos * h;
  for (long e = (long)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (long)gridDim.x * blockDim.x) {
    const long p = e / h;
    const int i = (int)(e - p * h);
    double s, c;
    sincos((double)p * freq[i], &s, &c);
    cs[p * rot + i] = (float)(c * attn);
    cs[p * rot + h + i] = (float)(s * attn);
  }
}

cudaError_t launch_rope_fill(float* cs, const double* freq, int rot, int max_pos, double attn, cudaStream_t st) {
  const long n = (long)max_pos * (rot / 2);
  const int blocks = (int)((n + 255) / 256 < 152 * 16 ? (n + 255) / 256 : 152 * 16);
  return launch_kernel(rope_fill_kernel, dim3(blocks), dim3(256), 0, st, 1, cs, freq, rot, max_pos, attn);
}

__device__ __forceinline__ void turn(float c, float s, float x1, float x2, float& y1, float& y2) {
  y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
}
// N elements of a row, loaded and stored in one access of 8 or 16 bytes.
template <typename T, int N> struct RowUnit {
  static constexpr int WORDS = N * sizeof(T) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
  }
  __device__ __forceinline__ void unpack(float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      f[i] = __uint_as_float(sizeof(T) == 4 ? w[i] : i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void pack(const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(f[i]);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
  }
};

// Rows in units of N elements, 16 or 8 bytes (grid y: the part).  A thread takes one unit (HALF: N
// elements and their partners rot/2 further on; INTERLEAVED: N; past rot: N to copy) of HPT heads
// of one row, which share its cosines and sines, all loads before the first use.  Neighbouring
// threads take neighbouring units, then neighbouring heads.
template <typename T, int LAYOUT, int HPT, int N>
__global__ void __launch_bounds__(256) rope_vec_kernel(const __grid_constant__ RopeArgs a) {
  const medusa_rope_rows& p = a.part[blockIdx.y];
  const int h = a.t.rot / 2, turned = LAYOUT == MEDUSA_ROPE_HALF ? h / N : a.t.rot / N;
  const bool place = p.x == p.y;
  const int units = turned + (place ? 0 : (a.dh - a.t.rot) / N);
  const int groups = (p.heads + HPT - 1) / HPT;
  const unsigned long long e = (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int u = (int)(e % units);
  const int hg = (int)(e / units % groups);
  const long r = (long)(e / units / groups);
  if (r >= a.rows) return;
  const T* x = static_cast<const T*>(p.x) + r * p.x_row;
  T* y = static_cast<T*>(p.y) + r * p.y_row;
  const int at = u < turned ? u * N : a.t.rot + (u - turned) * N;
  RowUnit<T, N> v[HPT][2];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int hd = hg + i * groups;
    if (hd >= p.heads) break;
    v[i][0].load(x + hd * p.x_head + at);
    if (LAYOUT == MEDUSA_ROPE_HALF && u < turned) v[i][1].load(x + hd * p.x_head + at + h);
  }
  if (u < turned) {
    const int pos = a.pos[r];
    const bool ok = pos >= 0 && pos < a.t.max_pos;
    if (!ok && u == 0 && hg == 0) set_flag(a.t.status, MEDUSA_FLAG_POS_RANGE);
    constexpr int M = LAYOUT == MEDUSA_ROPE_HALF ? N : N / 2;   // angles of a unit
    float c[M], s[M];
    if (ok) {
      const float* cs = a.t.cs + (long)pos * a.t.rot + u * M;
#pragma unroll
      for (int i = 0; i < M; i += 2) {
        const float2 c2 = *reinterpret_cast<const float2*>(cs + i), s2 = *reinterpret_cast<const float2*>(cs + h + i);
        c[i] = c2.x;
        c[i + 1] = c2.y;
        s[i] = a.inverse ? -s2.x : s2.x;
        s[i + 1] = a.inverse ? -s2.y : s2.y;
      }
#pragma unroll
      for (int i = 0; i < HPT; ++i) {
        float f[N], g[N];
        v[i][0].unpack(f);
        if (LAYOUT == MEDUSA_ROPE_HALF) {
          v[i][1].unpack(g);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            float y1, y2;
            turn(c[k], s[k], f[k], g[k], y1, y2);
            f[k] = y1;
            g[k] = y2;
          }
          v[i][1].pack(g);
        } else {
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            float y1, y2;
            turn(c[k / 2], s[k / 2], f[k], f[k + 1], y1, y2);
            f[k] = y1;
            f[k + 1] = y2;
          }
        }
        v[i][0].pack(f);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int hd = hg + i * groups;
    if (hd >= p.heads) break;
    v[i][0].store(y + hd * p.y_head + at);
    if (LAYOUT == MEDUSA_ROPE_HALF && u < turned) v[i][1].store(y + hd * p.y_head + at + h);
  }
}

// Any alignment and any even rot: one thread per (row, head, pair) and passed-through element.
template <typename T>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  const int h = a.t.rot / 2, units = h + (a.dh - a.t.rot);
  const long n = (long)a.rows * a.heads * units;
  for (long e = (long)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (long)gridDim.x * blockDim.x) {
    const int u = (int)(e % units);
    const long rh = e / units;
    int hd = (int)(rh % a.heads);
    const long r = rh / a.heads;
    int pi = 0;
    while (hd >= a.part[pi].heads) hd -= a.part[pi++].heads;
    const medusa_rope_rows& p = a.part[pi];
    const T* x = static_cast<const T*>(p.x) + r * p.x_row + hd * p.x_head;
    T* y = static_cast<T*>(p.y) + r * p.y_row + hd * p.y_head;
    const int pos = a.pos[r];
    const bool ok = pos >= 0 && pos < a.t.max_pos;
    if (!ok && u == 0) set_flag(a.t.status, MEDUSA_FLAG_POS_RANGE);
    if (u >= h) {
      y[a.t.rot + u - h] = x[a.t.rot + u - h];
      continue;
    }
    const int i1 = a.t.layout == MEDUSA_ROPE_HALF ? u : 2 * u;
    const int i2 = a.t.layout == MEDUSA_ROPE_HALF ? u + h : 2 * u + 1;
    const float x1 = to_f32(x[i1]), x2 = to_f32(x[i2]);
    float y1 = x1, y2 = x2;
    if (ok) {
      const float c = a.t.cs[(long)pos * a.t.rot + u], s = a.t.cs[(long)pos * a.t.rot + h + u];
      turn(c, a.inverse ? -s : s, x1, x2, y1, y2);
    }
    y[i1] = from_f32<T>(y1);
    y[i2] = from_f32<T>(y2);
  }
}

template <typename T, int LAYOUT, int HPT, int N>
static cudaError_t rope_vec(const RopeArgs& a, cudaStream_t st) {
  long most = 0;
  for (int i = 0; i < a.n_parts; ++i) {
    const medusa_rope_rows& p = a.part[i];
    const int turned = LAYOUT == MEDUSA_ROPE_HALF ? a.t.rot / 2 / N : a.t.rot / N;
    const int units = turned + (p.x == p.y ? 0 : (a.dh - a.t.rot) / N);
    const long n = (long)a.rows * units * ((p.heads + HPT - 1) / HPT);
    most = n > most ? n : most;
  }
  const dim3 grid((unsigned)((most + 255) / 256), (unsigned)a.n_parts);
  return launch_kernel(rope_vec_kernel<T, LAYOUT, HPT, N>, grid, dim3(256), 0, st, 1, a);
}

// Whether all rows can be taken in units of n elements.
template <typename T> static bool units_fit(const RopeArgs& a, int n) {
  const size_t bytes = n * sizeof(T);
  bool fit = a.dh % n == 0 && a.t.rot % n == 0 && (a.t.layout != MEDUSA_ROPE_HALF || a.t.rot / 2 % n == 0);
  for (int i = 0; i < a.n_parts; ++i) {
    const medusa_rope_rows& p = a.part[i];
    fit = fit && reinterpret_cast<uintptr_t>(p.x) % bytes == 0 && reinterpret_cast<uintptr_t>(p.y) % bytes == 0 &&
          p.x_row % n == 0 && p.x_head % n == 0 && p.y_row % n == 0 && p.y_head % n == 0;
  }
  return fit;
}
// Heads of a thread share its angles' loads, but too few threads leave the GPU idle.  40 heads of
// 128 bf16 elements, 1 / 2 / 4 heads a thread (us): HALF 65 rows 2.0 / 2.3 / 2.9, 512 rows 3.5 / 3.4 /
// 3.9, 4096 rows 14.5 / 12.1 / 13.3; INTERLEAVED 65 rows 2.0 / 2.0 / 2.3, 512 rows 4.1 / 3.4 / 3.3, 4096
// rows 21.8 / 14.2 / 11.1.
template <typename T, int N> static cudaError_t rope_units(const RopeArgs& a, cudaStream_t st) {
  const bool many = (long)a.rows * a.heads * a.dh >= 2l << 20;
  constexpr int H = MEDUSA_ROPE_HALF, I = MEDUSA_ROPE_INTERLEAVED;
  if (a.t.layout == H) return many ? rope_vec<T, H, 2, N>(a, st) : rope_vec<T, H, 1, N>(a, st);
  return many ? rope_vec<T, I, 4, N>(a, st) : rope_vec<T, I, 1, N>(a, st);
}

template <typename T>
static cudaError_t rope_go(const RopeArgs& a, cudaStream_t st) {
  constexpr int N = 16 / sizeof(T);
  if (units_fit<T>(a, N)) return rope_units<T, N>(a, st);
  if constexpr (N == 8) {                  // partial rotations whose halves are no whole 16 bytes
    if (units_fit<T>(a, 4)) return rope_units<T, 4>(a, st);
  }
  const long n = (long)a.rows * a.heads * (a.dh - a.t.rot / 2);
  const int blocks = (int)((n + 255) / 256 < 1 << 20 ? (n + 255) / 256 : 1 << 20);
  return launch_kernel(rope_kernel<T>, dim3(blocks), dim3(256), 0, st, 1, a);
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st) {
  return dtype == MEDUSA_F32 ? rope_go<float>(a, st) : rope_go<bf16>(a, st);
}

}  // namespace medusa
