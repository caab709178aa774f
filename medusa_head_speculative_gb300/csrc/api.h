// What the C entry points of the handles share (rotations, caches, 8-bit products): small checks, and
// reading a status word.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/medusa.h"

namespace medusa {

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline size_t elem(int dtype) { return dtype == MEDUSA_F32 ? 4 : 2; }
inline bool is_dtype(int t) { return t == MEDUSA_F32 || t == MEDUSA_BF16; }
// A handle's memory lives on the device that was current when it was made.
inline bool here(int device) {
  int d = -1;
  return cudaGetDevice(&d) == cudaSuccess && d == device;
}
// Whether no two of rows x heads pieces of dh elements, row and head elements apart, share an element: results
// that lie on one another would be written in any order.
inline bool lie_apart(long long rows, long long row, long long heads, long long head, int dh) {
  if ((rows > 1 && row < dh) || (heads > 1 && head < dh)) return false;
  if (rows <= 1 || heads <= 1) return true;
  if (row >= (__int128)(heads - 1) * head + dh || head >= (__int128)(rows - 1) * row + dh) return true;
  for (long long i = 1; i < heads; ++i) {          // neither within the other's gaps: piece by piece
    const __int128 at = (__int128)i * head, j = at / row;
    if ((j < rows && at - j * row < dh) || (j + 1 < rows && (j + 1) * row - at < dh)) return false;
  }
  return true;
}
inline medusa_status done(cudaError_t e) { return e == cudaSuccess ? MEDUSA_OK : MEDUSA_ERR_CUDA; }

inline medusa_status read_status(uint32_t* word, void* stream, uint32_t* flags) {
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, S(stream)) != cudaSuccess ||
      cudaMemsetAsync(word, 0, sizeof(v), S(stream)) != cudaSuccess || cudaStreamSynchronize(S(stream)) != cudaSuccess)
    return MEDUSA_ERR_CUDA;
  *flags = v;
  return v ? MEDUSA_ERR_DEVICE : MEDUSA_OK;
}

}  // namespace medusa
