// How the work of attention over a shared prefix is dealt out, shared by its kernels.
//
// For each row (sequence b, node n, query head) the softmax runs over three ranges of keys: the shared
// prefix, the sequence's own slots, and the call's own rows.  Keys go in chunks of 128, and a chunk is
// multiplied with a block of query rows of its key head:
//   shared items  (head g, row block): the rows of ALL sequences of a head in one line, row (b n1 + n) G + h,
//                 so that a chunk of the prefix is read once for a block of up to 256 rows of any sequences
//   own items     (sequence b, head g, row block): b's slots, then the call's rows of b
// Each CTA works on one of the two kinds (the kinds differ in their row blocks) and takes an even share of
// that kind's units in one line, item after item.  An item's units are PxWork::item for its queries and its
// partial, which take about as long as so many chunks, and then its chunks; for every item of which a CTA has chunks
// it writes a partial (o, reference, sum) to a slot of its own, and the joining kernel adds an item's
// partials up in order.
// Lengths are read on the device, so all of this is counted there, the same way by every warp.
#pragma once
#include "common.cuh"
#include "kvcache.cuh"
#include "prefix.h"

namespace medusa {

constexpr int PX_KEYS = 128;                      // keys of a chunk

// Counted by the main kernel for the joining one.
struct PxPlan {
  long ws, wo;                                    // units of the shared and of the own items
  int cs, co;                                     // CTAs that work on them
  int ns;                                         // chunks of a shared item
};
struct PxWork {
  PrefixArgs a;
  int R, rows;                                    // rows of a head: a sequence's, all
  int rbs, nrbs, rbo, nrbo;                       // rows of a block and blocks of a head: shared, own
  int cost_s, cost_o;                             // of a chunk
  int item;                                       // what an item costs besides, in chunks
  int tree;                                       // chunks of the call's own rows
  int ctas;
  float* o_s; float2* ml_s;                       // partials of shared items [slot][rbs][dh], [slot][rbs]
  float* o_o; float2* ml_o;
  PxPlan* plan;
  long* first;                                    // [B]: units of the sequences before b (for one head and block)
};

__device__ __forceinline__ int px_chunks(const PxWork& w, int b) {
  return (clamp_len(w.a.own, w.a.own.len[b]) + PX_KEYS - 1) / PX_KEYS + w.tree;
}
__device__ __forceinline__ int px_units(const PxWork& w, int chunks) { return chunks > 0 ? chunks + w.item : 0; }
// All lanes of a warp; writes the plan and `first` when asked to.
__device__ __forceinline__ PxPlan px_plan(const PxWork& w, bool write) {
  const int lane = threadIdx.x & 31, B = w.a.own.B;
  long sum = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int mine = b0 + lane < B ? px_units(w, px_chunks(w, b0 + lane)) : 0;
    long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (write && b0 + lane < B) w.first[b0 + lane] = sum + upto - mine;
    sum += __shfl_sync(0xffffffffu, upto, 31);
  }
  PxPlan p;
  p.ns = (clamp_len(w.a.shared, w.a.shared.len[0]) + PX_KEYS - 1) / PX_KEYS;
  p.ws = (long)px_units(w, p.ns) * w.a.own.Hkv * w.nrbs;
  p.wo = sum * w.a.own.Hkv * w.nrbo;
  const float s = (float)p.ws * w.cost_s, t = (float)(sum * w.a.own.Hkv * w.nrbo) * w.cost_o;
  p.cs = p.ws == 0 ? 0 : p.wo == 0 ? w.ctas : min(max((int)(w.ctas * (s / (s + t)) + 0.5f), 1), w.ctas - 1);
  p.co = w.ctas - p.cs;
  p.cs = (int)min((long)p.cs, p.ws);
  p.co = (int)min((long)p.co, p.wo);
  if (write && lane == 0) *w.plan = p;
  return p;
}

// One stretch of an item's chunks: j .. j + n - 1.
struct PxSeg {
  int b, g, rb, j, n;
  long slot;
};
// A CTA's walk through its chunks.
struct PxWalk {
  bool shared;
  int c, item, b, nb, j, per;                     // nb, j: units of an item, and the next one
  long left;
};
__device__ __forceinline__ PxWalk px_start(const PxWork& w, const PxPlan& p, int cta) {
  PxWalk k;
  k.shared = cta < p.cs;
  k.c = k.shared ? cta : cta - p.cs;
  const int n = k.shared ? p.cs : p.co;
  k.left = 0;
  k.b = 0;
  k.item = k.j = 0;
  k.nb = max(px_units(w, p.ns), 1);
  k.per = w.a.own.Hkv * (k.shared ? w.nrbs : w.nrbo);
  if (k.c >= n) return k;
  const long total = k.shared ? p.ws : p.wo;
  const long w0 = total * k.c / n;
  k.left = total * (k.c + 1) / n - w0;
  if (k.shared) {
    k.item = (int)(w0 / k.nb);
    k.j = (int)(w0 - (long)k.item * k.nb);
    return k;
  }
  const int lane = threadIdx.x & 31, B = w.a.own.B;
  long before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int mine = b0 + lane < B ? px_units(w, px_chunks(w, b0 + lane)) : 0;
    long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, (before + upto) * k.per > w0);
    if (hit || b0 + 32 >= B) {
      const int l = hit ? __ffs(hit) - 1 : 31;
      k.nb = max(__shfl_sync(0xffffffffu, mine, l), 1);
      const long in = w0 - (before + __shfl_sync(0xffffffffu, upto - mine, l)) * k.per;
      k.b = b0 + l;
      k.item = (int)(in / k.nb);
      k.j = (int)(in - (long)k.item * k.nb);
      return k;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}
__device__ __forceinline__ bool px_next(const PxWork& w, PxWalk& k, PxSeg& s) {
  const int nrb = k.shared ? w.nrbs : w.nrbo;
  do {
    if (k.left <= 0) return false;
    s.b = k.b;
    s.g = k.item / nrb;
    s.rb = k.item - s.g * nrb;
    s.j = max(k.j - w.item, 0);
    const int n = (int)min((long)(k.nb - k.j), k.left);
    s.n = max(k.j + n - w.item, 0) - s.j;        // (0: the share ends before the item's chunks)
    s.slot = (long)k.c + (k.shared ? (long)k.item : (long)k.b * k.per + k.item);
    k.left -= n;
    k.j = 0;
    if (++k.item == k.per && !k.shared && k.left > 0) {
      k.item = 0;
      do {
        ++k.b;
        k.nb = px_units(w, px_chunks(w, k.b));       // (what is left lies in a later sequence)
      } while (k.nb == 0);
    }
  } while (s.n == 0);
  return true;
}

// Query row r of a block: its node row (b n1 + n), node n and query head; < 0 rows are none.
struct PxRow {
  long node_row;
  int n, head;
  bool ok;
};
__device__ __forceinline__ PxRow px_row(const PxWork& w, bool shared, const PxSeg& s, int r) {
  const int gr = s.rb * (shared ? w.rbs : w.rbo) + r;
  PxRow x;
  x.ok = r < (shared ? w.rbs : w.rbo) && gr < (shared ? w.rows : w.R);
  const int node = gr / w.a.G;
  x.head = s.g * w.a.G + gr - node * w.a.G;
  x.node_row = shared ? node : (long)s.b * w.a.n1 + node;
  x.n = shared ? 0 : node;                        // (only the call's own rows ask for it)
  return x;
}
// 32 bits of which of the call's own rows 32 i .. 32 i + 31 node n sees.
__device__ __forceinline__ uint32_t px_sees(const PrefixArgs& a, int n, int i) {
  const int rest = a.n1 - 32 * i;                 // (mask bits from n1 on name no row)
  if (rest <= 0) return 0u;
  const uint32_t there = rest >= 32 ? 0xffffffffu : (1u << rest) - 1u;
  if (a.mask) return a.mask[(long)n * 8 + i] & there;
  const int upto = n - 32 * i;
  return (upto < 0 ? 0u : upto >= 31 ? 0xffffffffu : (2u << upto) - 1u) & there;
}

// bf16 rows on the tensor cores (k_prefix_tc.cu): dh 64 or 128.
cudaError_t launch_prefix_tc(const PxWork& w, cudaStream_t st);

}  // namespace medusa
