// Attention over a 4-bit KV cache ("Medusa: Simple LLM Inference Acceleration Framework with
// Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5, over the format of
// include/medusa.h).
//
// A CTA takes one sequence, one KV head and eight of the rows (node x query head of the
// group) that share it; each warp has one row and runs over the cached slots 32 at a time, one
// slot a lane, with a running maximum and sum, then over the tree keys its row sees.
#include "cache.h"
#include "common.cuh"
#include "kvcache.cuh"
#include "launch.cuh"

namespace medusa {

constexpr int KS_ROWS = 8;

template <typename T, int DH>
__global__ void __launch_bounds__(256) kv4_attn_simple_kernel(const __grid_constant__ Kv4AttnArgs a) {
  constexpr int C = DH / 32;
  __shared__ float ks[32][DH + 1], vs[32][DH], qs[KS_ROWS][DH];
  const CacheView& c = a.c;
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.n1 * a.G, r = blockIdx.x * KS_ROWS + warp;
  const bool live = r < R;
  const int node = live ? r / a.G : 0, hq = g * a.G + (live ? r % a.G : 0);
  const T* q = static_cast<const T*>(a.q) + ((long)b * a.n1 + node) * a.q_row + hq * a.q_head;
  for (int i = 0; i < C; ++i) qs[warp][lane + 32 * i] = to_f32(q[lane + 32 * i]);
  const int len = clamp_len(c, c.len[b]);
  float m = -INFINITY, l = 0.f, o[C];
  for (int i = 0; i < C; ++i) o[i] = 0.f;
  for (int t0 = 0; t0 < len; t0 += 32) {
    __syncthreads();
    for (int e = tid; e < 32 * 2 * (DH / 16); e += 256) {
      const int part = e & 1, grp = (e >> 1) % (DH / 16), j = (e >> 1) / (DH / 16), t = t0 + j;
      float f[16];
      for (int x = 0; x < 16; ++x) f[x] = 0.f;
      long unit;
      int in;
      if (t < len) {
        if (unit_of(c, b, t, unit, in)) {
          const uint8_t* block = static_cast<const uint8_t*>(part ? c.v : c.k) + kv4_offset(c, unit, in, g);
          const int slot = in % KV4_SLOTS;
          kv4_decode(*reinterpret_cast<const uint2*>(block + slot * (DH / 2) + grp * 8),
                     block[8 * DH + slot * (DH / 16) + grp], part ? c.gv : c.gk, f);
        } else {
          set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
        }
      }
      for (int x = 0; x < 16; ++x) (part ? &vs[j][grp * 16] : &ks[j][grp * 16])[x] = f[x];
    }
    __syncthreads();
    float s = -INFINITY;
    if (t0 + lane < len) {
      s = 0.f;
      for (int d = 0; d < DH; ++d) s = fmaf(qs[warp][d], ks[lane][d], s);
      s *= a.scale;
    }
    const float mn = fmaxf(m, warp_max(s)), al = __expf(m - mn), p = __expf(s - mn);
    l = l * al + warp_sum(p);
    m = mn;
    for (int i = 0; i < C; ++i) o[i] *= al;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      for (int i = 0; i < C; ++i) o[i] = fmaf(pj, vs[j][lane + 32 * i], o[i]);
    }
  }
  if (!live) return;
  if (a.tk) {
    for (int j = 0; j < a.n1; ++j) {
      const bool see = a.mask ? (a.mask[(long)node * 8 + (j >> 5)] >> (j & 31)) & 1u : j <= node;
      if (!see) continue;
      const long off = (((long)b * a.n1 + j) * c.Hkv + g) * DH;
      float s = 0.f;
      for (int i = 0; i < C; ++i)
        s = fmaf(qs[warp][lane + 32 * i], to_f32(static_cast<const T*>(a.tk)[off + lane + 32 * i]), s);
      s = warp_sum(s) * a.scale;
      const float mn = fmaxf(m, s), al = __expf(m - mn), p = __expf(s - mn);
      l = l * al + p;
      m = mn;
      for (int i = 0; i < C; ++i)
        o[i] = fmaf(p, to_f32(static_cast<const T*>(a.tv)[off + lane + 32 * i]), o[i] * al);
    }
  }
  T* y = static_cast<T*>(a.o) + ((long)b * a.n1 + node) * a.o_row + hq * a.o_head;
  for (int i = 0; i < C; ++i) y[lane + 32 * i] = from_f32<T>(l > 0.f ? o[i] / l : 0.f);
}

size_t kv4_workspace(int, int, int, int, int, int) { return 256; }

template <typename T>
static cudaError_t attn_go(const Kv4AttnArgs& a, cudaStream_t st) {
  const dim3 grid((a.n1 * a.G + KS_ROWS - 1) / KS_ROWS, a.c.Hkv, a.c.B);
  auto kern = a.c.dh == 128 ? kv4_attn_simple_kernel<T, 128>
              : a.c.dh == 64 ? kv4_attn_simple_kernel<T, 64> : kv4_attn_simple_kernel<T, 32>;
  return launch_kernel(kern, grid, dim3(256), 0, st, 1, a);
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int dtype, void*, int, cudaStream_t st) {
  return dtype == MEDUSA_F32 ? attn_go<float>(a, st) : attn_go<bf16>(a, st);
}

}  // namespace medusa
