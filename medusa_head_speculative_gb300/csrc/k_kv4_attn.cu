// Attention over a 4-bit KV cache ("Medusa: Simple LLM Inference Acceleration Framework with
// Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5, over the format of
// include/medusa.h), for few query rows a key/value head: single tokens and small trees.
//
// Rows: the n1 nodes x G query heads that share a key/value head, up to 8 or 16 at a time (a
// "row block").  Work: every (sequence, head, row block) has ceil(len / 128) chunks of 128 cached
// slots; all chunks of the call in that order are dealt out evenly, CTA i of n taking the
// chunks [W i / n, W (i + 1) / n), n at most W, whatever sequences they belong to (the lengths are read on
// the GPU).  A CTA that leaves a (sequence, head, row block) writes its unnormalised partial
// (o, max, sum) to slot i + p, p the index of the triple: both grow along the work, so slots
// are never shared, and one triple's slots lie together.  kv4_combine_kernel joins them, adds
// the call's own tree rows and rounds once.
//
// In a CTA each of four warps takes 32 slots of a chunk: two blocks of the format, each in one
// piece, so each warp keeps its own ring of blocks filled by the copy engine.  With few rows a
// 128-row tcgen05 tile would be mostly padding; the products here go through warp-wide
// 16 x 8 x 16 MMAs whose operands are decoded straight into registers, never written to shared
// memory.  The cache is the 16-row operand and the queries the 8-column one, so 8 rows waste
// nothing and cost half the registers: S^T = K Q^T (a lane's 16 bytes are 32 elements of one
// key; the order of the head's elements is free as long as Q has the same), then O^T += V^T P^T
// with P^T turned into a column operand by one 8 x 8 register transpose a key tile, and the
// codes of two keys put side by side before they are decoded.  e2m1 * e4m3 is exact in a half,
// so K and V lose nothing; P is rounded to a half (11 bits), queries are scaled row by row by
// a power of two into a half's range, which is exact for bf16 but for elements 2^-17 below the
// row's largest.  Float queries and their P go as two halves (22 bits) in two MMAs.
//
// Measured: one row of each of 32 heads over 1024 slots (4.7 MB) 7.0 us, one launch, latency; 16
// sequences x 8 heads x 4 rows over 4100-8192 slots each (115 MB, 17 us at copy bandwidth) 32.7 us.
// There a chunk takes 943 cycles of an SM, 790 at copy bandwidth; some 600 are the decoding's
// conversions, multiplications and nibble moves (half-rate instructions), the rest of the time goes
// into starting, the last partial chunks and joining (about 10 us together).
#include "cache.h"
#include "common.cuh"
#include "kv4_attn.cuh"
#include "kvcache.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace medusa {

constexpr int KD_WARPS = 4, KD_ROWS = 16, KD_STAGES = 2;
template <int NR> constexpr int KD_CTAS = NR == 1 ? 4 : 3;     // resident CTAs per SM (registers, shared memory)
constexpr int KD_CTAS_MOST = 4;
constexpr int KD_CLUSTER = 8;         // CTAs of a cluster that share one triple (small calls)
constexpr int KD_SMALL_CTAS = 3, KD_SMALL_SLOTS = 8192;   // see kd_small()
constexpr int KD_KEYS = 2 * KV4_SLOTS;              // slots a warp takes at a time: two blocks
static_assert(KD_CHUNK == KD_WARPS * KD_KEYS, "a chunk is the warps' slots");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Q as column operands: for MMA step s and 8-row tile n, lane (g, t) holds row 8 n + g, elements
// e, e + 1 and e + 2, e + 3 with e = t dh/4 + 4 s; kept in shared memory as the lanes read it.
template <typename T, int DH, int NR, bool SPLIT>
__device__ __forceinline__ void kd_load_q(const Kv4Work& w, int b, int g, int rb, uint32_t* qf, float* rs) {
  // one warp two rows at a time: 16 lanes a row, DH / 16 elements a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, li = lane & 15;
  constexpr int N = DH / 16;
  for (int r0 = warp * 2; r0 < 8 * NR; r0 += 2 * KD_WARPS) {
    const int r = r0 + half, gr = rb * w.rb + r;
    float x[N];
    float top = 0.f;
    const bool ok = r < w.rb && gr < w.R;
    const int node = ok ? gr / w.a.G : 0, hq = g * w.a.G + (ok ? gr - node * w.a.G : 0);
    const T* q = static_cast<const T*>(w.a.q) + ((long)b * w.a.n1 + node) * w.a.q_row + hq * w.a.q_head + li * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = ok ? to_f32(q[i]) : 0.f;
      top = fmaxf(top, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float down;
    const float factor = row_scale(w.a, top, down);
    if (li == 0) rs[r] = factor;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const int e = li * N + i, t = e / (DH / 4), in = e % (DH / 4), s = in >> 2, hi = (in >> 1) & 1;
      const float x0 = x[i] * down, x1 = x[i + 1] * down;
      const __half2 p = __floats2half2_rn(x0, x1);
      const int at = (((s * NR + (r >> 3)) * 32 + (r & 7) * 4 + t) << 1) + hi;
      qf[at] = h2u(p);
      if (SPLIT) {
        const float2 f = __half22float2(p);
        qf[DH / 16 * NR * 64 + at] = half_pair(x0 - f.x, x1 - f.y);
      }
    }
  }
}
// Thread-block cluster: all of its threads meet; 1, 2 or 4 floats of CTA `rank`'s shared memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int N> __device__ __forceinline__ void peer_load(uint32_t addr, uint32_t rank, float (&v)[N]) {
  asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  if constexpr (N == 4)
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 4, 2 or 1 elements of a lane as loaded: bf16 pairs stay packed until they are used.
template <typename T, int N> struct LaneRow {
  uint32_t u[(N * sizeof(T) + 3) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N * sizeof(T) == 16) *reinterpret_cast<uint4*>(u) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (N * sizeof(T) == 8) *reinterpret_cast<uint2*>(u) = *reinterpret_cast<const uint2*>(p);
    else if constexpr (N * sizeof(T) == 4) u[0] = *reinterpret_cast<const uint32_t*>(p);
    else u[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    else return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
};

// N = 1, 2 or 4 consecutive elements of a lane.
template <int N> __device__ __forceinline__ void store_f(float* p, const float (&f)[N]) {
  if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  else p[0] = f[0];
}
template <int N> __device__ __forceinline__ void store_f(bf16* p, const float (&f)[N]) {
  if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
  else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = pack2(f[0], f[1]);
  else p[0] = from_f32<bf16>(f[0]);
}

// One warp finishes a query row: the prefix's (o, reference, sum) from join(m, l, o), the call's own
// rows the row sees added in float, and the quotient rounded once.  A row of a candidate tree sees its
// ancestors only (at most 9), so going through the set bits beats a masked product with all n1; a chunk
// without a mask, whose rows see up to 256, pays for it row by row (8 x 256 rows of 32 heads over 3000
// slots: 650 us, 133 without the call's own rows).
// The first four visible rows' keys and values are loaded before join, which waits for loads too.
template <typename T, int DH, typename Join>
__device__ __forceinline__ void finish_row(const Kv4Work& w, int b, int node, int hq, Join join) {
  constexpr int C = DH / 32;
  const Kv4AttnArgs& a = w.a;
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, bn = b * a.n1 + node;
  const int g = hq / a.G;
  // lane i < 8: word i of the row's visible bits
  uint32_t mine = 0;
  if (a.tk && lane < (a.n1 + 31) / 32) {
    const int first = 32 * lane;
    mine = a.mask ? a.mask[(long)node * 8 + lane]
                  : (node >= first + 31 ? 0xffffffffu : node < first ? 0u : (2u << (node - first)) - 1u);
    if (a.n1 < first + 32) mine &= (1u << (a.n1 - first)) - 1u;
  }
  LaneRow<T, C> q;
  if (a.tk) q.load(static_cast<const T*>(a.q) + (long)bn * a.q_row + hq * a.q_head + lane * C);
  int wd = 0;
  uint32_t bits = __shfl_sync(0xffffffffu, mine, 0);
  auto next_row = [&]() {                  // the next visible row, -1: none
    while (!bits && ++wd < 8) bits = __shfl_sync(0xffffffffu, mine, wd);
    if (!bits) return -1;
    const int j = 32 * wd + __ffs(bits) - 1;
    bits &= bits - 1;
    return j;
  };
  const long tree0 = ((long)b * a.n1 * c.Hkv + g) * DH + lane * C;
  const int tree_row = c.Hkv * DH;
  LaneRow<T, C> tk[4], tv[4];
  int seen = 0;                            // of the four, how many there are
  auto load_rows = [&]() {
    seen = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = next_row();
      if (j < 0) continue;
      const long off = tree0 + (long)j * tree_row;
      tk[u].load(static_cast<const T*>(a.tk) + off);
      tv[u].load(static_cast<const T*>(a.tv) + off);
      seen = u + 1;
    }
  };
  if (a.tk) load_rows();
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
  join(m, l, o);
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] *= c.gv;
  if (a.tk) {
    const float scale = a.scale * 1.4426950408889634f;
#pragma unroll 1
    while (seen > 0) {
      float sc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        sc[u] = 0.f;
        if (u < seen) {
#pragma unroll
          for (int i = 0; i < C; ++i) sc[u] = fmaf(q[i], tk[u][i], sc[u]);
        }
      }
      // The four sums over the warp: lanes trade rows until each eight of them have one (10 shuffles for 20)
      const bool h16 = lane & 16, h8 = lane & 8;
      const float s0 = (h16 ? sc[2] : sc[0]) + __shfl_xor_sync(0xffffffffu, h16 ? sc[0] : sc[2], 16);
      const float s1 = (h16 ? sc[3] : sc[1]) + __shfl_xor_sync(0xffffffffu, h16 ? sc[1] : sc[3], 16);
      float sum = (h8 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, h8 ? s0 : s1, 8);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
      for (int u = 0; u < 4; ++u) sc[u] = __shfl_sync(0xffffffffu, sum, 8 * u);
      float mn = m;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        sc[u] = u < seen ? sc[u] * scale : -INFINITY;
        mn = fmaxf(mn, sc[u]);
      }
      const float f = ex2_approx(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] *= f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u >= seen) continue;
        const float p = ex2_approx(sc[u] - mn);
        l += p;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = fmaf(p, tv[u][i], o[i]);
      }
      load_rows();
    }
  }
  T* y = static_cast<T*>(a.o) + (long)bn * a.o_row + hq * a.o_head + lane * C;
  const float inv = l == 0.f ? 0.f : 1.f / l;            // nothing seen: 0; a NaN stays one
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
  store_f<C>(y, o);
}

template <typename T, int DH, int NR, bool SPLIT, bool CLUSTER>
__global__ void __launch_bounds__(KD_WARPS * 32, KD_CTAS<NR>) kv4_rows_kernel(const __grid_constant__ Kv4Work w) {
  constexpr int BLK = kv4_block(DH), STEPS = DH / 16, MT = DH / 16;   // MT: 16-element tiles of O^T
  constexpr int QW = STEPS * NR * 64 * (SPLIT ? 2 : 1);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[KD_WARPS][KD_STAGES], never;
  __shared__ __align__(16) uint32_t qf[QW];
  __shared__ float rs[8 * NR];
  __shared__ float2 ml[KD_WARPS][8 * NR];
  __shared__ float2 whole[CLUSTER ? 8 * NR : 1];       // the CTA's (reference, sum)
  const CacheView& c = w.a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int per = c.Hkv * w.nrb;
  uint8_t* ring = smem + warp * KD_STAGES * 4 * BLK;
  float* merge = reinterpret_cast<float*>(smem + KD_WARPS * KD_STAGES * 4 * BLK);   // [2 warps][rb][DH + 4]
  constexpr int ML = DH + 4;
  long w0, w1;
  KdCursor k;
  if constexpr (CLUSTER) {
    // block (triple, rank): the ranks of a cluster share one triple's chunks
    k.b = blockIdx.x / per;
    k.q = blockIdx.x - k.b * per;
    k.nb = kd_chunks(c, k.b);
    w0 = k.nb * blockIdx.y / KD_CLUSTER;
    w1 = k.nb * (blockIdx.y + 1) / KD_CLUSTER;
    k.j = (int)w0;
  } else {
    const long W = kd_total(c, per);
    // every CTA that takes part has at least one chunk, so a triple's slots have no gaps
    const long ctas = W < (long)gridDim.x ? W : (long)gridDim.x;
    pdl_trigger();
    if (blockIdx.x >= ctas) return;
    w0 = W * blockIdx.x / ctas;
    w1 = W * (blockIdx.x + 1) / ctas;
    k = kd_seek(c, per, w0);
  }
  if (lane == 0)
    for (int s = 0; s < KD_STAGES; ++s) mbar_init(smem_u32(&bars[warp][s]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  const uint64_t pol = policy_evict_first();

  // ---- this warp's blocks, in order: the copies run up to KD_STAGES ahead.  Lane 2 i + x knows
  // where block x of the warp's chunk win0 + i lies (head 0's) and issues its copies.
  KdCursor pc = k;
  int left = (int)(w1 - w0);               // chunks to copy
  int issued = 0, taken = 0, drain = 0;
  int win_b = -1, win0 = 0, plen = 0, head = pc.q / w.nrb;
  long my_blk = 0;
  const int upp = (c.page_table ? c.page_size : c.capacity) / KV4_SLOTS;
  bool dead = false;
  auto copy_next = [&]() {
    // skips chunks whose part of 32 slots lies past the length
    while (left > 0) {
      if (win_b != pc.b || pc.j < win0 || pc.j >= win0 + 16) {
        plen = clamp_len(c, c.len[pc.b]);
        win_b = pc.b;
        win0 = pc.j;
        const int t = (win0 + (lane >> 1)) * KD_CHUNK + warp * KD_KEYS + (lane & 1) * KV4_SLOTS;
        if (t < plen) {
          long unit;
          int in;
          if (!unit_of(c, pc.b, t, unit, in)) {
            set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
            unit = 0;
          }
          my_blk = unit * c.Hkv * upp + in / KV4_SLOTS;
        }
      }
      const int t0 = pc.j * KD_CHUNK + warp * KD_KEYS;
      const bool any = t0 < plen;
      if (any) {
        const bool both = t0 + KV4_SLOTS < plen;
        if ((lane >> 1) == pc.j - win0 && (both || !(lane & 1))) {
          const int st = issued % KD_STAGES;
          const uint32_t bar = smem_u32(&bars[warp][st]), dst = smem_u32(ring + st * 4 * BLK) + (lane & 1) * BLK;
          const long off = (my_blk + (long)head * upp) * BLK;
          if (!(lane & 1)) mbar_expect_tx(bar, both ? 4 * BLK : 2 * BLK);
          bulk_load(dst, static_cast<const uint8_t*>(c.k) + off, BLK, bar, pol);
          bulk_load(dst + 2 * BLK, static_cast<const uint8_t*>(c.v) + off, BLK, bar, pol);
        }
        ++issued;
      }
      if (--left > 0) {
        const int q0 = pc.q, b0 = pc.b;
        kd_next(c, per, pc);
        if (pc.q != q0 || pc.b != b0) head = pc.q / w.nrb;
      }
      if (any) return;
    }
  };
  for (int s = 0; s < KD_STAGES; ++s) copy_next();

  if constexpr (CLUSTER) {
    if (w0 == w1 && tid < w.rb) whole[tid] = make_float2(-INFINITY, -1.f);   // no chunks, no sums
  }
  if constexpr (!CLUSTER) {                // failure-path tests; in the one-launch form it would cost 0.12 us
    if (w.a.test_wait_ns && warp == 0) {
      if (lane == 0) mbar_init(smem_u32(&never), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      __syncwarp();
      dead = !__all_sync(0xffffffffu, mbar_wait(smem_u32(&never), 0, w.a.test_wait_ns));
    }
  }
  long wi = w0;
  while (wi < w1) {
    // ---- one (sequence, head, row block)
    const int b = k.b, q = k.q, g = q / w.nrb, rb = q - g * w.nrb;
    const int len = clamp_len(c, c.len[b]);
    const long n = min((long)(k.nb - k.j), w1 - wi);
    const int j0 = k.j;
    kd_load_q<T, DH, NR, SPLIT>(w, b, g, rb, qf, rs);
    __syncthreads();
    // a lane has the rows 8 x + 2 t4 + {0, 1} of each row tile x
    float f[NR][2], m[NR][2], l[NR][2], o[MT][NR][4];
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[x][e] = rs[8 * x + 2 * t4 + e];
        m[x][e] = -INFINITY;
        l[x][e] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int x = 0; x < NR; ++x) o[i][x][0] = o[i][x][1] = o[i][x][2] = o[i][x][3] = 0.f;
    for (int j = j0; j < j0 + (int)n; ++j) {
      const int t0 = j * KD_CHUNK + warp * KD_KEYS;
      if (t0 >= len) break;
      const int st = taken % KD_STAGES;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][st]), (taken / KD_STAGES) & 1, TC_TIMEOUT_NS))) {
        dead = true;
        drain = taken;
      }
      ++taken;
      if (dead) continue;
      const uint8_t* kb = ring + st * 4 * BLK;
      const uint8_t* vb = kb + 2 * BLK;
      // ---- S^T = K Q^T for two blocks of 16 keys: a lane has keys g8, g8 + 8 of each
      float s[2][NR][4];
      uint32_t kw[4][DH / 32];
      __half2 s2[4];                       // the lane's dh/4 elements have one scale (dh 128: two)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint8_t* blk = kb + (y >> 1) * BLK;
        const int key = (y & 1) * 8 + g8;
        const uint8_t* src = blk + key * (DH / 2) + t4 * (DH / 8);
        if (DH == 128) *reinterpret_cast<uint4*>(kw[y]) = *reinterpret_cast<const uint4*>(src);
        else if (DH == 64) *reinterpret_cast<uint2*>(kw[y]) = *reinterpret_cast<const uint2*>(src);
        else kw[y][0] = *reinterpret_cast<const uint32_t*>(src);
        const uint8_t* sc = blk + 8 * DH + key * (DH / 16) + t4 * DH / 64;
        if (DH == 128) s2[y] = kv4_scales(*reinterpret_cast<const uint16_t*>(sc));
        else s2[y] = __half2half2(kv4_scale(*sc));
      }
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int x = 0; x < NR; ++x) s[hb][x][0] = s[hb][x][1] = s[hb][x][2] = s[hb][x][3] = 0.f;
#pragma unroll
      for (int x = 0; x < DH / 32; ++x) {
        __half2 y[4][4];
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          kv4_pairs(kw[k4][x], y[k4]);
          const __half2 sc = x < 2 ? __low2half2(s2[k4]) : __high2half2(s2[k4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[k4][e] = __hmul2(y[k4][e], sc);
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t ka[2][4] = {{h2u(y[0][2 * z]), h2u(y[1][2 * z]), h2u(y[0][2 * z + 1]), h2u(y[1][2 * z + 1])},
                                     {h2u(y[2][2 * z]), h2u(y[3][2 * z]), h2u(y[2][2 * z + 1]), h2u(y[3][2 * z + 1])}};
#pragma unroll
          for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              const uint2 q2 = *reinterpret_cast<const uint2*>(
                  qf + part * STEPS * NR * 64 + (((2 * x + z) * NR + n) * 32 + lane) * 2);
              mma16816(s[0][n], ka[0], q2.x, q2.y);
              mma16816(s[1][n], ka[1], q2.x, q2.y);
            }
        }
      }
      // ---- softmax
      const bool tail = t0 + KD_KEYS > len;
      if (tail) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (t0 + hb * KV4_SLOTS + g8 + 8 * (e >> 1) >= len) s[hb][x][e] = -INFINITY;
      }
      float top[NR][2];
      bool raise = false;
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {       // the rows' factors are positive
          top[x][e] = fmaxf(fmaxf(s[0][x][e], s[0][x][e + 2]), fmaxf(s[1][x][e], s[1][x][e + 2])) * f[x][e];
          raise = raise || !(top[x][e] <= m[x][e] + KD_TOP);
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = top[x][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
            const float mn = fmaxf(m[x][e], v - KD_BACK<SPLIT>);
            const float fall = m[x][e] == -INFINITY ? 0.f : ex2_approx(m[x][e] - mn);
            m[x][e] = mn;
            l[x][e] *= fall;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][x][e] *= fall;
              o[i][x][e + 2] *= fall;
            }
          }
      }
      uint32_t pb[2][NR][2], pl[2][NR][2];  // P^T as column operands, and what the halves left
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            const float p0 = ex2_approx(fmaf(s[hb][x][2 * k8], f[x][0], -m[x][0]));
            const float p1 = ex2_approx(fmaf(s[hb][x][2 * k8 + 1], f[x][1], -m[x][1]));
            l[x][0] += p0;
            l[x][1] += p1;
            const __half2 h = __floats2half2_rn(p0, p1);
            pb[hb][x][k8] = transpose8(h2u(h));
            if (SPLIT) {
              const float2 hf = __half22float2(h);
              pl[hb][x][k8] = transpose8(half_pair(p0 - hf.x, p1 - hf.y));
            }
          }
      // ---- O^T += V^T P^T: lane's keys 2 t4, + 1, + 8, + 9 of each block, elements from g8 DH/8 on
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const uint8_t* blk = vb + hb * BLK;
        uint32_t vw[4][DH > 64 ? 2 : 1];
        __half vh[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 2 * t4 + (x & 1) + 8 * (x >> 1);
          const uint8_t* src = blk + key * (DH / 2) + g8 * (DH / 16);
          if (DH == 128) *reinterpret_cast<uint2*>(vw[x]) = *reinterpret_cast<const uint2*>(src);
          else if (DH == 64) vw[x][0] = *reinterpret_cast<const uint32_t*>(src);
          else vw[x][0] = *reinterpret_cast<const uint16_t*>(src);
          vh[x] = kv4_scale(blk[8 * DH + key * (DH / 16) + g8 * DH / 128]);
          if (tail && t0 + hb * KV4_SLOTS + key >= len) vh[x] = __float2half(0.f);   // p is 0 there: keep 0 * NaN out
        }
        const __half2 v0 = __halves2half2(vh[0], vh[1]), v1 = __halves2half2(vh[2], vh[3]);
#pragma unroll
        for (int x = 0; x < (DH > 64 ? 2 : 1); ++x) {
          // nibbles of two keys side by side: bytes of the even elements, then of the odd ones
          constexpr uint32_t LO = 0x0f0f0f0fu;
          __half2 e0[4], e1[4], o0[4], o1[4];
          kv4_pairs((vw[0][x] & LO) | ((vw[1][x] << 4) & ~LO), e0);
          kv4_pairs((vw[2][x] & LO) | ((vw[3][x] << 4) & ~LO), e1);
          kv4_pairs(((vw[0][x] >> 4) & LO) | (vw[1][x] & ~LO), o0);
          kv4_pairs(((vw[2][x] >> 4) & LO) | (vw[3][x] & ~LO), o1);
#pragma unroll
          for (int i = 0; i < 4 && 4 * x + i < MT; ++i) {
            const uint32_t va[4] = {h2u(__hmul2(e0[i], v0)), h2u(__hmul2(o0[i], v0)), h2u(__hmul2(e1[i], v1)),
                                    h2u(__hmul2(o1[i], v1))};
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              mma16816(o[4 * x + i][n], va, pb[hb][n][0], pb[hb][n][1]);
              if (SPLIT) mma16816(o[4 * x + i][n], va, pl[hb][n][0], pl[hb][n][1]);
            }
          }
        }
      }
      fence_proxy_async();                   // every lane has read the stage before the copy engine writes there
      __syncwarp();
      copy_next();
    }
    // ---- join the warps' partials and write the CTA's: everybody on one reference, then the
    // upper two warps' sums onto the lower two's
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], d);
        if (g8 == 0) ml[warp][8 * x + 2 * t4 + e] = make_float2(m[x][e], l[x][e]);
      }
    __syncthreads();
    auto joined = [&](int r) {               // (reference, sum) of row r over the warps
      float mn = -INFINITY, sum = 0.f;
#pragma unroll
      for (int y = 0; y < KD_WARPS; ++y) mn = fmaxf(mn, ml[y][r].x);
#pragma unroll
      for (int y = 0; y < KD_WARPS; ++y) sum += ml[y][r].x == -INFINITY ? 0.f : ex2_approx(ml[y][r].x - mn) * ml[y][r].y;
      return make_float2(mn, sum);
    };
    float fall[NR][2];
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        fall[x][e] = m[x][e] == -INFINITY ? 0.f : ex2_approx(m[x][e] - joined(8 * x + 2 * t4 + e).x);
    float* mine = merge + (warp & 1) * w.rb * ML;
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      if ((warp >> 1) == 1 - step) {
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * x + 2 * t4 + e;
            if (r >= w.rb) continue;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              float2* at = reinterpret_cast<float2*>(mine + r * ML + g8 * (DH / 8) + 2 * i);
              float2 v = make_float2(o[i][x][e] * fall[x][e], o[i][x][e + 2] * fall[x][e]);
              if (step) {
                v.x += at->x;
                v.y += at->y;
              }
              *at = v;
            }
          }
      }
      __syncthreads();
    }
    if constexpr (CLUSTER) {                 // to this CTA's own shared memory: the cluster joins it
      for (int e = tid; e < w.rb * DH; e += KD_WARPS * 32) {
        const int r = e / DH, col = e - r * DH;
        merge[r * ML + col] += merge[(w.rb + r) * ML + col];
        if (col == 0) whole[r] = joined(r);
      }
      break;
    }
    const long pair = (long)b * per + q, slot = pair + blockIdx.x;
    for (int e = tid; e < w.rb * (DH / 4); e += KD_WARPS * 32) {
      const int r = e / (DH / 4), col = (e - r * (DH / 4)) * 4;
      const float4 v0 = *reinterpret_cast<const float4*>(merge + r * ML + col);
      const float4 v1 = *reinterpret_cast<const float4*>(merge + (w.rb + r) * ML + col);
      *reinterpret_cast<float4*>(w.part_o + (slot * w.rb + r) * DH + col) =
          make_float4(v0.x + v1.x, v0.y + v1.y, v0.z + v1.z, v0.w + v1.w);
      if (col == 0) w.part_ml[slot * w.rb + r] = joined(r);
    }
    if (tid == 0) {
      if (j0 == 0) w.span[pair].x = (int)slot;
      if (j0 + n == k.nb) w.span[pair].y = (int)slot + 1;
    }
    __syncthreads();                         // before the next triple's queries and partials
    wi += n;
    k.j += (int)n - 1;
    if (wi < w1) kd_next(c, per, k);
  }
  if (dead) {
    set_flag(c.status, MEDUSA_FLAG_TIMEOUT);
    for (; drain < issued; ++drain)          // copies in flight (bounded)
      mbar_wait(smem_u32(&bars[warp][drain % KD_STAGES]), (drain / KD_STAGES) & 1, TC_TIMEOUT_NS / 16);
  }
  if constexpr (CLUSTER) {
    // every CTA of the cluster comes here: the rows are dealt out over its warps
    constexpr int C = DH / 32;
    cluster_sync();
    const int r = blockIdx.y * KD_WARPS + warp, g = k.q / w.nrb, gr = (k.q - g * w.nrb) * w.rb + r;
    if (r < w.rb && gr < w.R) {
      const int node = gr / w.a.G;
      finish_row<T, DH>(w, k.b, node, g * w.a.G + gr - node * w.a.G, [&](float& m, float& l, float (&o)[C]) {
        float2 y[KD_CLUSTER];
        float v[KD_CLUSTER][C];
#pragma unroll
        for (int x = 0; x < KD_CLUSTER; ++x) {
          peer_load(smem_u32(&whole[r]), x, reinterpret_cast<float(&)[2]>(y[x]));
          peer_load(smem_u32(merge + r * ML + lane * C), x, v[x]);
          m = fmaxf(m, y[x].x);
        }
#pragma unroll
        for (int x = 0; x < KD_CLUSTER; ++x) {
          if (y[x].y < 0.f) continue;          // a CTA without chunks: its sums were never written
          const float f = ex2_approx(y[x].x - m);
          l += f * y[x].y;
#pragma unroll
          for (int i = 0; i < C; ++i) o[i] = fmaf(f, v[x][i], o[i]);
        }
      });
    }
    cluster_sync();                          // nobody leaves while its shared memory is read
  }
}

// Joins the partials: one warp a query row.  What its loads depend on comes in two rounds: query,
// span and mask first, then the first partials and the first visible rows.  Bound by its
// instructions where the call brings rows of its own (two thirds of the issue slots; 20,800 rows, of
// which each sees up to six: 17 us, without such rows 8), else by latency (2.6 us for 512 rows).  Two or
// more rows a warp, 16 bytes a lane, took 1 to 2 us off the trees and put 0.2 to 0.4 on small calls.  SB partials in a
// round: few slots a row (many rows a head) need few registers, many need them.
template <typename T, int DH, int SB>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const __grid_constant__ Kv4Work w) {
  constexpr int C = DH / 32;
  const Kv4AttnArgs& a = w.a;
  const CacheView& c = a.c;
  // block (sequence and node, query heads)
  const int lane = threadIdx.x & 31;
  const int hq = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (hq >= a.Hq) return;
  const int bn = blockIdx.x, b = bn / a.n1, node = bn - b * a.n1;
  const int g = hq / a.G, r = node * a.G + hq - g * a.G;
  const int rb = w.nrb == 1 ? 0 : r / w.rb, in = r - rb * w.rb;
  const int len = clamp_len(c, c.len[b]);
  finish_row<T, DH>(w, b, node, hq, [&](float& m, float& l, float (&o)[C]) {
    pdl_wait();                            // the partials come from the kernel before
    if (len > 0) {
      const int2 sp = w.span[((long)b * c.Hkv + g) * w.nrb + rb];
#pragma unroll 1
      for (int s0 = sp.x; s0 < sp.y; s0 += SB) {
        float2 y[SB];
        LaneRow<float, C> v[SB];
#pragma unroll
        for (int u = 0; u < SB; ++u) {
          const long at = (long)min(s0 + u, sp.y - 1) * w.rb + in;
          y[u] = w.part_ml[at];
          v[u].load(w.part_o + (at * DH + lane * C));
        }
        float mn = m;                      // stays -inf only where every score was NaN: so is the sum, then
#pragma unroll
        for (int u = 0; u < SB; ++u) mn = fmaxf(mn, y[u].x);
        const float f = ex2_approx(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] *= f;
#pragma unroll
        for (int u = 0; u < SB; ++u) {
          if (s0 + u >= sp.y) continue;    // the last partial once more
          const float h = ex2_approx(y[u].x - mn);
          l += y[u].y * h;
#pragma unroll
          for (int i = 0; i < C; ++i) o[i] = fmaf(v[u][i], h, o[i]);
        }
      }
    }
  });
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// Row blocks, and how many CTAs a launch can have, of R rows a head.
static void blocks_of(int dtype, int dh, int R, int num_sms, int* rb, int* nrb, int* ctas) {
  if (kv4_tree_takes(dtype, dh, R)) {
    kv4_tree_blocks(R, rb, nrb);
    *ctas = num_sms;
  } else {
    *rb = R < KD_ROWS ? R : KD_ROWS;
    *nrb = (R + *rb - 1) / *rb;
    *ctas = num_sms * KD_CTAS_MOST;
  }
}

size_t kv4_workspace(int B, int Hq, int Hkv, int dh, int max_nodes, int num_sms) {
  size_t most = 0;
  for (int dtype : {MEDUSA_F32, MEDUSA_BF16})
    for (int R = Hq / Hkv, n = 1; n <= max_nodes; ++n, R += Hq / Hkv) {
      int rb, nrb, ctas;
      blocks_of(dtype, dh, R, num_sms, &rb, &nrb, &ctas);
      const size_t pairs = (size_t)B * Hkv * nrb, slots = ctas + pairs;
      const size_t s = up256(slots * rb * dh * 4) + up256(slots * rb * 8) + up256(pairs * 8);
      most = s > most ? s : most;
    }
  return most;
}

// Few triples in caches that are not long: a cluster of eight CTAs each, joined through
// distributed shared memory in the same launch.  All clusters have to be resident together, at
// three CTAs an SM.  Single tokens, dh 128, one launch against two (us): 32 triples, 64 slots
// 5.4 against 7.3, 2048 slots 7.3 / 9.8, 8192 slots 14.7 / 16.5; 8 triples, 8192 slots 12.6 / 14.7,
// but 16384 slots 20.5 / 18.3 (64 CTAs of a possible 608); 56 triples, 64 slots 6.0 / 6.6, 8192 slots
// 20.8 / 21.6, 16384 slots 37.0 / 34.1; 80 triples, which take two rounds, 9.9 / 6.6.
static bool kd_small(const Kv4Work& w, int num_sms) {
  return !w.a.test_wait_ns && (long)w.a.c.B * w.a.c.Hkv * w.nrb * KD_CLUSTER <= (long)num_sms * KD_SMALL_CTAS && w.a.c.capacity <= KD_SMALL_SLOTS;
}
template <typename T, int DH, int NR, bool SPLIT>
static cudaError_t rows_go(const Kv4Work& w, int num_sms, cudaStream_t st) {
  const size_t ring = (size_t)KD_WARPS * KD_STAGES * 4 * kv4_block(DH);
  const size_t smem = ring + (size_t)2 * w.rb * (DH + 4) * 4, most = ring + (size_t)2 * 8 * NR * (DH + 4) * 4;
  static unsigned long long done = 0, done_small = 0;
  if (kd_small(w, num_sms)) {
    auto kern = kv4_rows_kernel<T, DH, NR, SPLIT, true>;
    const cudaError_t e = allow_smem(kern, most, &done_small);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3((unsigned)(w.a.c.B * w.a.c.Hkv * w.nrb), KD_CLUSTER), dim3(KD_WARPS * 32), smem, st,
                         KD_CLUSTER, w);
  }
  auto kern = kv4_rows_kernel<T, DH, NR, SPLIT, false>;
  const cudaError_t e = allow_smem(kern, most, &done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(num_sms * KD_CTAS<NR>), dim3(KD_WARPS * 32), smem, st, 1, w);
}
template <typename T, int SB> static cudaError_t combine(const Kv4Work& w, cudaStream_t st) {
  const int warps = w.a.Hq < 8 ? w.a.Hq : 8;
  const dim3 grid((unsigned)w.a.c.B * w.a.n1, (unsigned)((w.a.Hq + warps - 1) / warps));
  auto kern = w.a.c.dh == 32   ? kv4_combine_kernel<T, 32, SB>
              : w.a.c.dh == 64 ? kv4_combine_kernel<T, 64, SB>
                               : kv4_combine_kernel<T, 128, SB>;
  return launch_kernel(kern, grid, dim3(32 * warps), 0, st, 1, w);
}
template <typename T, bool SPLIT>
static cudaError_t rows_dh(const Kv4Work& w, int num_sms, cudaStream_t st) {
  const bool one = w.rb <= 8;
  switch (w.a.c.dh) {
    case 32: return one ? rows_go<T, 32, 1, SPLIT>(w, num_sms, st) : rows_go<T, 32, 2, SPLIT>(w, num_sms, st);
    case 64: return one ? rows_go<T, 64, 1, SPLIT>(w, num_sms, st) : rows_go<T, 64, 2, SPLIT>(w, num_sms, st);
    default: return one ? rows_go<T, 128, 1, SPLIT>(w, num_sms, st) : rows_go<T, 128, 2, SPLIT>(w, num_sms, st);
  }
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int dtype, void* ws, int num_sms, cudaStream_t st) {
  Kv4Work w{};
  w.a = a;
  w.R = a.n1 * a.G;
  int ctas;
  blocks_of(dtype, a.c.dh, w.R, num_sms, &w.rb, &w.nrb, &ctas);
  const size_t slots = ctas + (size_t)a.c.B * a.c.Hkv * w.nrb;
  char* p = static_cast<char*>(ws);
  w.part_o = reinterpret_cast<float*>(p);
  p += up256(slots * w.rb * a.c.dh * 4);
  w.part_ml = reinterpret_cast<float2*>(p);
  p += up256(slots * w.rb * 8);
  w.span = reinterpret_cast<int2*>(p);
  const bool tree = kv4_tree_takes(dtype, a.c.dh, w.R);
  cudaError_t e = tree ? launch_kv4_tree(w, num_sms, st)
                  : dtype == MEDUSA_F32 ? rows_dh<float, true>(w, num_sms, st) : rows_dh<bf16, false>(w, num_sms, st);
  if (e != cudaSuccess || (!tree && kd_small(w, num_sms))) return e;
  // Partials a round of the joining kernel, 2 against 8, by how many a row has on average (us): 19
  // partials (8 heads, 8192 slots) 26.3 / 23.6, 4.8 30.9 / 30.1, 3.8 22.0 / 21.6; 1.2 (16 x 8 heads of 172
  // rows) 134 / 144, 0.5 (8 x 40 heads of 65 rows) 88 / 98.
  if (ctas >= 3l * a.c.B * a.c.Hkv * w.nrb) return dtype == MEDUSA_F32 ? combine<float, 8>(w, st) : combine<bf16, 8>(w, st);
  return dtype == MEDUSA_F32 ? combine<float, 2>(w, st) : combine<bf16, 2>(w, st);
}

}  // namespace medusa
