// Products of rows and weights in 8 bits (the format of include/medusa.h):
//   y[r][n] = sum_j xs[r][j] ws[n / 128][j] sum_{k in group j} x[r][k] w[n][k]   (+ add), or the gated pair.
// Codes are decoded to shared memory; a thread has 4 x 4 results of a 64 x 64 tile.
#include "fp8.cuh"
#include "launch.cuh"

namespace medusa {

constexpr int LT = 64, LP = kFp8Group + 4;

template <typename T, int NW>
__global__ void __launch_bounds__(256) fp8_linear_kernel(Fp8LinearArgs a) {
  extern __shared__ float sm[];
  float* xs = sm;                                  // [64][132]
  float* wt = sm + LT * LP;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n0 = blockIdx.x * LT;
  const long r0 = (long)blockIdx.y * LT;
  float acc[NW][4][4] = {};
  for (int j = 0; j < a.kb; ++j) {
    const int kn = min(kFp8Group, a.k - j * kFp8Group);
    for (int h = 0; h < NW; ++h) {
      __syncthreads();
      for (int e = tid; e < LT * 32; e += 256) {
        const int r = e / 32, c = e % 32 * 4;
        float v[4] = {};
        if (h == 0) {
          if (r0 + r < a.rows && c < kn) fp8_values(*reinterpret_cast<const uint32_t*>(a.x + (r0 + r) * a.x_row + j * kFp8Group + c), v);
          *reinterpret_cast<float4*>(xs + r * LP + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
        float u[4] = {};
        if (n0 + r < a.n && c < kn) fp8_values(*reinterpret_cast<const uint32_t*>(a.w[h] + (long)(n0 + r) * a.k + j * kFp8Group + c), u);
        *reinterpret_cast<float4*>(wt + r * LP + c) = make_float4(u[0], u[1], u[2], u[3]);
      }
      __syncthreads();
      float p[4][4] = {};
      for (int c = 0; c < kn; c += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(xs + (ty + 16 * i) * LP + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 w = *reinterpret_cast<const float4*>(wt + (tx + 16 * q) * LP + c);
            p[i][q] = fmaf(x.x, w.x, fmaf(x.y, w.y, fmaf(x.z, w.z, fmaf(x.w, w.w, p[i][q]))));
          }
        }
      const float sw = a.ws[h][(long)(n0 / kFp8Group) * a.kb + j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long r = r0 + ty + 16 * i;
        const float s = r < a.rows ? a.xs[r * a.kb + j] * sw : 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[h][i][q] = fmaf(p[i][q], s, acc[h][i][q]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const long r = r0 + ty + 16 * i;
      const int n = n0 + tx + 16 * q;
      if (r >= a.rows || n >= a.n) continue;
      float y = acc[0][i][q];
      if (NW == 2) y = y / (1.f + expf(-y)) * acc[NW - 1][i][q];
      if (a.add) y += to_f32(static_cast<const T*>(a.add)[r * a.add_row + n]);
      static_cast<T*>(a.y)[r * a.y_row + n] = from_f32<T>(y);
    }
}

template <typename T, int NW> static cudaError_t linear_go(const Fp8LinearArgs& a, cudaStream_t st) {
  const size_t smem = 2 * LT * LP * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(fp8_linear_kernel<T, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(fp8_linear_kernel<T, NW>, dim3((a.n + LT - 1) / LT, (a.rows + LT - 1) / LT), dim3(256), smem, st, 1, a);
}
cudaError_t launch_fp8_linear(const Fp8LinearArgs& a, int dtype, void* part, int num_sms, cudaStream_t st) {
  if (dtype == MEDUSA_F32) return a.w[1] ? linear_go<float, 2>(a, st) : linear_go<float, 1>(a, st);
  return a.w[1] ? linear_go<bf16, 2>(a, st) : linear_go<bf16, 1>(a, st);
}

}  // namespace medusa
