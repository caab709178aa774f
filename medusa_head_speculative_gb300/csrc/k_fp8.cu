// Rounding rows and weights to 8 bits and reading them back (the format of include/medusa.h).
//
// Both directions are bound by memory: round reads x once and writes 1 byte an element, read the
// reverse.  A warp has one group of 128 elements, 4 a lane, so that a group's maximum is one integer
// reduction over the warp and loads and stores are whole 128- to 512-byte lines; FP8_ILP groups are in
// flight a warp.  Weights: a CTA has one 128 x 128 block in registers, 16 rows a warp.
//
// Measured (one GB300): 13824 x 5120 float weights rounded and read back 121 us, 5.8 TB/s of 708 MB (copy: 6.8); 520 x
// 5120 bf16 rows 7.3 us for the two launches, of which 2.4 are their bytes.
#include "fp8.cuh"
#include "launch.cuh"

namespace medusa {

constexpr int FP8_ILP = 4;

__device__ __forceinline__ uint32_t top_of(const float (&x)[4]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) t = max(t, __float_as_uint(x[i]) & 0x7fffffffu);
  return t;
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_round_rows_kernel(Fp8RoundArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t groups = (uint32_t)a.rows * a.kb, warps = gridDim.x * 8;
  const T* x = static_cast<const T*>(a.x);
  for (uint32_t g0 = blockIdx.x * 8 + (threadIdx.x >> 5); g0 < groups; g0 += warps * FP8_ILP) {
    float v[FP8_ILP][4];
    uint32_t row[FP8_ILP], col[FP8_ILP];
#pragma unroll
    for (int i = 0; i < FP8_ILP; ++i) {
      const uint32_t g = g0 + i * warps;
      row[i] = g / a.kb;
      col[i] = (g - row[i] * a.kb) * kFp8Group + lane * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = 0.f;
      if (g < groups && col[i] < a.k) load4(x + row[i] * a.x_row + col[i], a.vec, v[i]);
    }
#pragma unroll
    for (int i = 0; i < FP8_ILP; ++i) {
      const uint32_t g = g0 + i * warps;
      if (g >= groups) break;
      const Fp8Scale s = fp8_scale(__reduce_max_sync(0xffffffffu, top_of(v[i])));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] *= s.inv;
      if (col[i] < a.k)
        *reinterpret_cast<uint32_t*>(a.codes + (long)row[i] * a.k + col[i]) = s.finite ? fp8_codes(v[i]) : FP8_NANS;
      if (lane == 0) {
        a.scales[g] = s.s;
        if (!s.finite) set_flag(a.status, MEDUSA_FLAG_NONFINITE);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_round_blocks_kernel(Fp8RoundArgs a) {
  __shared__ uint32_t tops[8];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nb = blockIdx.x / a.kb, kb = blockIdx.x - nb * a.kb;
  const int row0 = nb * kFp8Group + warp, col = kb * kFp8Group + lane * 4;
  const T* x = static_cast<const T*>(a.x);
  float v[16][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = 0.f;
    if (row0 + 8 * i < a.rows && col < a.k) load4(x + (row0 + 8 * i) * a.x_row + col, a.vec, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, top_of(v[i]));
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, tops[i]);
  const Fp8Scale s = fp8_scale(top);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] *= s.inv;
    if (row0 + 8 * i < a.rows && col < a.k)
      *reinterpret_cast<uint32_t*>(a.codes + (long)(row0 + 8 * i) * a.k + col) = s.finite ? fp8_codes(v[i]) : FP8_NANS;
  }
  if (threadIdx.x == 0) {
    a.scales[blockIdx.x] = s.s;
    if (!s.finite) set_flag(a.status, MEDUSA_FLAG_NONFINITE);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_read_kernel(Fp8ReadArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t groups = (uint32_t)a.rows * a.kb, warps = gridDim.x * 8;
  T* y = static_cast<T*>(a.y);
  for (uint32_t g0 = blockIdx.x * 8 + (threadIdx.x >> 5); g0 < groups; g0 += warps * FP8_ILP) {
    uint32_t c[FP8_ILP], row[FP8_ILP], col[FP8_ILP];
    float s[FP8_ILP];
#pragma unroll
    for (int i = 0; i < FP8_ILP; ++i) {
      const uint32_t g = g0 + i * warps;
      row[i] = g / a.kb;
      const uint32_t j = g - row[i] * a.kb;
      col[i] = j * kFp8Group + lane * 4;
      c[i] = 0;
      s[i] = 0.f;
      if (g < groups && col[i] < a.k) {
        c[i] = *reinterpret_cast<const uint32_t*>(a.codes + (long)row[i] * a.k + col[i]);
        s[i] = a.scales[(long)(row[i] / a.block) * a.kb + j];
      }
    }
#pragma unroll
    for (int i = 0; i < FP8_ILP; ++i) {
      if (g0 + i * warps >= groups || col[i] >= a.k) continue;
      float v[4];
      fp8_values(c[i], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= s[i];
      save4(y + (long)row[i] * a.y_row + col[i], a.vec, v);
    }
  }
}

// Blocks of 8 warps: all that an SM holds, at most.
static int group_blocks(int rows, int kb, int num_sms) {
  const long per = 8 * FP8_ILP, groups = (long)rows * kb, blocks = (groups + per - 1) / per, most = 8L * num_sms;
  return (int)(blocks < most ? blocks : most);
}

cudaError_t launch_fp8_round(const Fp8RoundArgs& a, int dtype, int block, int num_sms, cudaStream_t st) {
  const bool f32 = dtype == MEDUSA_F32;
  if (block == 1)
    return launch_kernel(f32 ? fp8_round_rows_kernel<float> : fp8_round_rows_kernel<bf16>, dim3(group_blocks(a.rows, a.kb, num_sms)),
                         dim3(256), 0, st, 1, a);
  const int nb = (a.rows + kFp8Group - 1) / kFp8Group;
  return launch_kernel(f32 ? fp8_round_blocks_kernel<float> : fp8_round_blocks_kernel<bf16>, dim3((unsigned)nb * a.kb),
                       dim3(256), 0, st, 1, a);
}
cudaError_t launch_fp8_read(const Fp8ReadArgs& a, int dtype, int num_sms, cudaStream_t st) {
  return launch_kernel(dtype == MEDUSA_F32 ? fp8_read_kernel<float> : fp8_read_kernel<bf16>,
                       dim3(group_blocks(a.rows, a.kb, num_sms)), dim3(256), 0, st, 1, a);
}

}  // namespace medusa
