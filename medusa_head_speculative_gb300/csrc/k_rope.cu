// Rotary positions: the table of cosines and sines, and the rotation of query / key rows
// ("Medusa: Simple LLM Inference Acceleration Framework with Multiple Decoding Heads" §3.4
// Tree Attention Step 4: a node's position is the prefix length plus its depth).
//
// y1 = x1 c - x2 s, y2 = x2 c + x1 s with every product and sum rounded by itself (no fused
// multiply-add), so that the result depends on the inputs alone and not on how a kernel
// groups the operations: medusa_kv_append quantises the same values.
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

// One thread per (row, head, pair) and per passed-through element pair.
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
      const float c = a.t.cs[(long)pos * a.t.rot + u];
      const float s0 = a.t.cs[(long)pos * a.t.rot + h + u], s = a.inverse ? -s0 : s0;
      y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
      y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    }
    y[i1] = from_f32<T>(y1);
    y[i2] = from_f32<T>(y2);
  }
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st) {
  const long n = (long)a.rows * a.heads * (a.dh - a.t.rot / 2);
  const int blocks = (int)((n + 255) / 256 < 1 << 20 ? (n + 255) / 256 : 1 << 20);
  return launch_kernel(dtype == MEDUSA_F32 ? rope_kernel<float> : rope_kernel<bf16>, dim3(blocks), dim3(256), 0, st,
                       1, a);
}

}  // namespace medusa
