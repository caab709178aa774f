// Launch interfaces of the 8-bit projections (internal; the public API is include/medusa.h, whose
// description of the format holds here).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/medusa.h"

namespace medusa {

constexpr int kFp8Group = 128;                    // elements of a row's scale, rows and columns of a block's

struct Fp8RoundArgs {
  const void* x; long x_row;
  uint8_t* codes; float* scales;
  int rows, k, kb;                                // kb = ceil(k / 128)
  int vec;                                        // 4 elements of x are one aligned load
  uint32_t* status;
};
cudaError_t launch_fp8_round(const Fp8RoundArgs& a, int dtype, int block, int num_sms, cudaStream_t st);
struct Fp8ReadArgs {
  const uint8_t* codes; const float* scales;
  void* y; long y_row;
  int rows, k, kb, block, vec;
};
cudaError_t launch_fp8_read(const Fp8ReadArgs& a, int dtype, int num_sms, cudaStream_t st);

struct Fp8LinearArgs {
  const uint8_t* x; const float* xs; long x_row;  // codes and scales [rows][kb]
  const uint8_t* w[2]; const float* ws[2];        // weights, and the pair's second (or NULL)
  const void* add; long add_row;
  void* y; long y_row;
  int rows, n, k, kb;
  uint32_t* status;
  unsigned long long test_wait_ns;                // failure-path tests only (0 otherwise): a wait that runs out
};
// How a call of so many rows is cut up: tiles of 128 rows by `columns` results, `whole` of them each one CTA's, `shared` added
// up from several CTAs' partials.
struct Fp8Tiles {
  int columns, whole, shared;
};
Fp8Tiles fp8_linear_tiles(int rows, int n, int kb, bool gated, int num_sms);
// Bytes of partials (`part`) a call may need.
size_t fp8_linear_partials(int max_rows, int n, int kb, int num_sms);
cudaError_t launch_fp8_linear(const Fp8LinearArgs& a, int dtype, void* part, int num_sms, cudaStream_t st);

}  // namespace medusa
