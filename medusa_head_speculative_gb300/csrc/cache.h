// Launch interfaces of the rotary and KV-cache kernels (internal; the public API is
// include/medusa.h, whose descriptions of the formats and rules hold here).
#pragma once
#include <cuda_runtime.h>

#include "../../include/medusa.h"

namespace medusa {

// ---- rotary positions
struct RopeTable {
  const float* cs;        // device [max_pos][rot]: rot/2 cosines, then rot/2 sines
  int rot, max_pos, layout;
  uint32_t* status;
};
// Fills cs from rot/2 frequencies (device doubles).
cudaError_t launch_rope_fill(float* cs, const double* freq, int rot, int max_pos, double attn, cudaStream_t st);

constexpr int kRopeParts = 4;
struct RopeArgs {
  RopeTable t;
  const int32_t* pos;
  int rows, dh, n_parts, heads, inverse;          // heads: of all parts together
  medusa_rope_rows part[kRopeParts];
};
cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st);

// ---- caches
struct CacheView {
  void* k; void* v;
  const int32_t* page_table; const int32_t* len; int32_t* len_out;
  int B, Hkv, dh, capacity, page_size, pages_per_seq, num_pages;   // page_size 0: contiguous
  float gk, gv;                                                    // KV4: k_scale, v_scale
  uint32_t* status;
};
// Which items belong to which sequence (medusa_kv_rows: packed or padded).
struct ItemMap {
  int rows, per_seq;
  const int32_t* start; const int32_t* count;
};
struct AppendArgs {
  CacheView c;
  ItemMap m;
  const void* k; const void* v;
  long k_row, k_head, v_row, v_head;
  const int32_t* index; int index_rows;
  const int32_t* pos;
  int turn;                                       // 1: t is given
  RopeTable t;
  int vec;                                        // rows move in 16-byte units
};
cudaError_t launch_kv_append(const AppendArgs& a, int src_dtype, int format, cudaStream_t st);
struct ReadArgs {
  CacheView c;
  ItemMap m;
  void* k; void* v;
  long k_row, k_head, v_row, v_head;
  const int32_t* first;
  int vec;
};
cudaError_t launch_kv_read(const ReadArgs& a, int dst_dtype, int format, cudaStream_t st);

// ---- attention over a 4-bit cache
struct Kv4AttnArgs {
  CacheView c;
  const void* q; void* o;
  long q_row, q_head, o_row, o_head;
  const void* tk; const void* tv;
  const uint32_t* mask;
  int n1, Hq, G;                                  // G = Hq / Hkv query heads per KV head
  float scale;                                    // of the scores, without gk
  float factor_m;                                 // scale gk log2(e) = factor_m 2^factor_e, factor_m in [1, 2)
  int factor_e;
  unsigned long long test_wait_ns;                // failure-path tests only (0 otherwise): a wait that runs out
};
cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int dtype, void* ws, int num_sms, cudaStream_t st);
size_t kv4_workspace(int B, int Hq, int Hkv, int dh, int max_nodes, int num_sms);

}  // namespace medusa
