// Launch interface of attention over a shared prefix (internal; the public API is include/medusa.h).
#pragma once
#include "cache.h"

namespace medusa {

struct PrefixArgs {
  CacheView own, shared;
  const void* q; void* o;
  long q_row, q_head, o_row, o_head;
  const void* tk; const void* tv;                 // the call's own rows [B][n1][Hkv][dh], or NULL
  const uint32_t* mask;                           // [n1][8]; NULL: row j <= n
  int n1, Hq, G;                                  // G = Hq / Hkv query heads per KV head
  float scale2;                                   // of the scores, times log2(e)
  uint32_t* status;                               // own's
  unsigned long long test_wait_ns;                // failure-path tests only (0 otherwise): a wait that runs out
};
// Whether a kernel with limited waits takes such heads (bf16 rows on the tensor cores).
bool prefix_tc_takes(int dtype, int dh);
// Bytes of workspace for calls of up to max_nodes rows a sequence.
size_t prefix_workspace(int B, int Hq, int Hkv, int dh, int max_nodes, int num_sms);
cudaError_t launch_prefix_attention(const PrefixArgs& a, int dtype, void* ws, int num_sms, cudaStream_t st);

}  // namespace medusa
