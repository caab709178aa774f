// What the two kernels of 4-bit cache attention share: how the work is dealt out, and where
// partials go (k_kv4_attn.cu: few rows a head; k_kv4_tree.cu: many).
#pragma once
#include <cuda_fp16.h>

#include "cache.h"
#include "common.cuh"
#include "kvcache.cuh"
#include "launch.cuh"

namespace medusa {

struct Kv4Work {
  Kv4AttnArgs a;
  int R, rb, nrb;                     // rows of a head, rows of a block, row blocks
  float* part_o;                      // [slots][rb][dh]
  float2* part_ml;                    // [slots][rb] (reference in base-2 units, sum)
  int2* span;                         // [B * Hkv * nrb]: first slot and one past the last
};

constexpr int KD_CHUNK = 128;         // cached slots of a chunk

// Scores are scaled to base-2 units.  P is taken against a reference 2^KD_TOP below a half's
// range: a row's reference starts KD_BACK (log2) below its running maximum and is raised, O
// rescaled, only once a score passes it by KD_TOP.  Small probabilities then stay normal halves
// down to 2^(-14 - back) of the largest; with two halves for P (float inputs) that floor
// matters most, so the reference lies lower and moves more often.
constexpr float KD_TOP = 15.f;
template <bool SPLIT> constexpr float KD_BACK = SPLIT ? 13.f : 7.f;

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) { return h2u(__floats2half2_rn(lo, hi)); }

// down: 2^-e, which brings a row whose largest element is top into [1, 2).  Returned: what its scores,
// taken with that row and with keys without gk, are multiplied by (base-2 units): 2^e scale gk log2(e).
// Put together from exponents, as the product of its parts can leave a float's range where it does
// not, and kept within 2^-126 .. 2^107: not 0 and not infinite for any row, and with |score| < 2^20 (128 x
// 2 x 448 x 6) neither is a product.  A factor of 0 would turn a masked score's -infinity into NaN.
__device__ __forceinline__ float row_scale(const Kv4AttnArgs& a, float top, float& down) {
  const int eb = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23), 1), 253) : 127;
  down = __uint_as_float((uint32_t)(254 - eb) << 23);
  return __uint_as_float(__float_as_uint(a.factor_m) + ((uint32_t)min(max(eb - 127 + a.factor_e, -126), 107) << 23));
}

// Contiguous bytes (multiples of 16) to shared memory by the copy engine.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}

// Chunks of sequence b.
__device__ __forceinline__ int kd_chunks(const CacheView& c, int b) {
  return (clamp_len(c, c.len[b]) + KD_CHUNK - 1) / KD_CHUNK;
}
// All chunks of the call, and where the walk through them stands at chunk w: sequence b, its
// triple q of Hkv * nrb, chunk j, and nb chunks of b.
struct KdCursor {
  int b, q, j, nb;
};
__device__ __forceinline__ long kd_total(const CacheView& c, int per) {
  long sum = 0;
  for (int b = threadIdx.x & 31; b < c.B; b += 32) sum += kd_chunks(c, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * per;
}
__device__ __forceinline__ KdCursor kd_seek(const CacheView& c, int per, long w) {
  const int lane = threadIdx.x & 31;
  long before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int mine = b0 + lane < c.B ? kd_chunks(c, b0 + lane) : 0;
    long upto = mine;                              // chunks of the sequences b0 .. b0 + lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, (before + upto) * per > w);
    if (hit || b0 + 32 >= c.B) {
      const int l = hit ? __ffs(hit) - 1 : 31;
      const int nb = __shfl_sync(0xffffffffu, mine, l);
      const long first = (before + __shfl_sync(0xffffffffu, upto, l) - nb) * per;
      KdCursor k;
      k.b = b0 + l;
      k.nb = max(nb, 1);
      const long in = w - first;
      k.q = (int)(in / k.nb);
      k.j = (int)(in - (long)k.q * k.nb);
      return k;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}
__device__ __forceinline__ void kd_next(const CacheView& c, int per, KdCursor& k) {
  if (++k.j < k.nb) return;
  k.j = 0;
  if (++k.q < per) return;
  k.q = 0;
  do {
    ++k.b;
    k.nb = k.b < c.B ? kd_chunks(c, k.b) : 1;
  } while (k.nb == 0);
}

// Many rows a head on the tensor cores (k_kv4_tree.cu): bf16, dh 64 or 128.
bool kv4_tree_takes(int dtype, int dh, int R);
void kv4_tree_blocks(int R, int* rb, int* nrb);
cudaError_t launch_kv4_tree(const Kv4Work& w, int num_sms, cudaStream_t st);

}  // namespace medusa
