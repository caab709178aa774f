// Attention over a 4-bit KV cache ("Medusa: Simple LLM Inference Acceleration Framework with
// Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5, over the format of
// include/medusa.h), for few query rows a key/value head: single tokens and small trees.
//
// Rows: the n1 nodes x G query heads that share a key/value head, 16 at a time (a "row
// block").  Work: every (sequence, head, row block) has ceil(len / 64) chunks of 64 cached
// slots; all chunks of the call in that order are dealt out evenly, CTA i of n taking the
// chunks [W i / n, W (i + 1) / n), n at most W, whatever sequences they belong to (the lengths are read on
// the GPU).  A CTA that leaves a (sequence, head, row block) writes its unnormalised partial
// (o, max, sum) to slot i + p, p the index of the triple: both grow along the work, so slots
// are never shared, and one triple's slots lie together.  kv4_combine_kernel joins them, adds
// the call's own tree rows and rounds once.
//
// In a CTA each of four warps takes 16 slots of a chunk: one block of the format, which lies
// in one piece, so each warp keeps its own ring of blocks filled by the copy engine.  With
// few rows a 128-row tcgen05 tile would be mostly padding; the products here go through
// warp-wide 16 x 8 x 16 MMAs whose operands are decoded straight into registers, never
// written to shared memory: S = Q K^T with K as the column operand (a lane's 16 bytes are 32
// elements of one key; the order of the head's elements is free as long as Q has the same),
// then O += P V with S's own register layout as the row operand and pairs of keys packed per
// element as the column operand.  e2m1 * e4m3 is exact in a half, so K and V lose nothing;
// P is rounded to a half (11 bits), queries are scaled row by row by a power of two into a
// half's range, which is exact for bf16 but for elements 2^-17 below the row's largest.  Float
// queries and their P go as two halves (22 bits) in two MMAs.
#include "cache.h"
#include "common.cuh"
#include "kvcache.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace medusa {

constexpr int KD_WARPS = 4, KD_ROWS = 16, KD_CHUNK = KD_WARPS * KV4_SLOTS, KD_STAGES = 4, KD_CTAS = 3;
// P is taken against a reference 2^KD_TOP below a half's range: a row's reference starts KD_BACK
// (log2) below its running maximum and is raised, O rescaled, only once a score passes it by
// KD_TOP.  Small probabilities then stay normal halves down to 2^(-14 - back) of the largest; with
// two halves for P (float inputs) that floor matters most, so the reference lies lower and
// moves more often.
constexpr float KD_TOP = 15.f;
template <bool SPLIT> constexpr float KD_BACK = SPLIT ? 13.f : 7.f;

struct Kv4Work {
  Kv4AttnArgs a;
  int R, rb, nrb;                     // rows of a head, rows of a block, row blocks
  float* part_o;                      // [slots][rb][dh]
  float2* part_ml;                    // [slots][rb] (reference in base-2 units, sum)
  int2* span;                         // [B * Hkv * nrb]: first slot and one past the last
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) { return h2u(__floats2half2_rn(lo, hi)); }

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

// Q as row operands: a[s] holds, for MMA step s, rows g and g + 8 and elements e, e + 1 and
// e + 2, e + 3 with e = t dh/4 + 4 s; kept in shared memory as the lanes read it.
template <typename T, int DH, bool SPLIT>
__device__ __forceinline__ void kd_load_q(const Kv4Work& w, int b, int g, int rb, uint32_t* qf, float* rs) {
  // one warp two rows at a time: 16 lanes a row, DH / 16 elements a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, li = lane & 15;
  constexpr int N = DH / 16;
  for (int r0 = warp * 2; r0 < KD_ROWS; r0 += 2 * KD_WARPS) {
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
    // 2^-e with the row's largest element in [2^e, 2^(e+1)), and 2^e for the scores
    const int eb = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23), 1), 253) : 127;
    const float down = __uint_as_float((uint32_t)(254 - eb) << 23), up = __uint_as_float((uint32_t)eb << 23);
    if (li == 0) rs[r] = up * (w.a.scale * w.a.c.gk) * 1.4426950408889634f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const int e = li * N + i, t = e / (DH / 4), in = e % (DH / 4), s = in >> 2, hi = (in >> 1) & 1;
      const float x0 = x[i] * down, x1 = x[i + 1] * down;
      const __half2 p = __floats2half2_rn(x0, x1);
      const int at = ((s * 32 + (r & 7) * 4 + t) << 2) + (hi << 1) + (r >> 3);
      qf[at] = h2u(p);
      if (SPLIT) {
        const float2 f = __half22float2(p);
        qf[DH / 16 * 128 + at] = half_pair(x0 - f.x, x1 - f.y);
      }
    }
  }
}

template <typename T, int DH, bool SPLIT>
__global__ void __launch_bounds__(KD_WARPS * 32, KD_CTAS) kv4_rows_kernel(const __grid_constant__ Kv4Work w) {
  constexpr int BLK = kv4_block(DH), STEPS = DH / 16, NT = DH / 8;
  constexpr int QW = STEPS * 128 * (SPLIT ? 2 : 1);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[KD_WARPS][KD_STAGES];
  __shared__ uint32_t qf[QW];
  __shared__ float rs[KD_ROWS];
  __shared__ float2 ml[KD_WARPS][KD_ROWS];
  const CacheView& c = w.a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int per = c.Hkv * w.nrb;
  uint8_t* ring = smem + warp * KD_STAGES * 2 * BLK;
  float* merge = reinterpret_cast<float*>(smem + KD_WARPS * KD_STAGES * 2 * BLK);   // [warps][rb][DH + 4]
  constexpr int ML = DH + 4;
  const long W = kd_total(c, per);
  // every CTA that takes part has at least one chunk, so a triple's slots have no gaps
  const long ctas = W < (long)gridDim.x ? W : (long)gridDim.x;
  pdl_trigger();
  if (blockIdx.x >= ctas) return;
  const long w0 = W * blockIdx.x / ctas, w1 = W * (blockIdx.x + 1) / ctas;
  if (lane == 0)
    for (int s = 0; s < KD_STAGES; ++s) mbar_init(smem_u32(&bars[warp][s]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  const uint64_t pol = policy_evict_first();

  // ---- this warp's blocks, in order: the copies run up to KD_STAGES ahead
  KdCursor pc = kd_seek(c, per, w0), k = pc;
  long pw = w0;                            // next chunk to copy
  int issued = 0, taken = 0, drain = 0;
  int win_b = -1, win0 = 0, my_page = 0;   // page ids of 32 of the warp's blocks from win0 on
  bool dead = false;
  auto copy_next = [&]() {
    // skips chunks whose part of 16 slots lies past the length
    while (pw < w1) {
      const int t0 = pc.j * KD_CHUNK + warp * KV4_SLOTS;
      const bool any = t0 < clamp_len(c, c.len[pc.b]);
      if (any) {
        long blk;
        const int g = pc.q / w.nrb;
        if (c.page_table) {
          if (win_b != pc.b || pc.j < win0 || pc.j >= win0 + 32) {
            win_b = pc.b;
            win0 = pc.j;
            const int t = t0 + lane * KD_CHUNK;
            my_page = 0;
            if (t < clamp_len(c, c.len[pc.b])) {
              my_page = c.page_table[(long)pc.b * c.pages_per_seq + t / c.page_size];
              if (my_page < 0 || my_page >= c.num_pages) {
                set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
                my_page = 0;
              }
            }
          }
          const long page = __shfl_sync(0xffffffffu, my_page, pc.j - win0);
          blk = (page * c.Hkv + g) * (c.page_size / KV4_SLOTS) + t0 % c.page_size / KV4_SLOTS;
        } else {
          blk = ((long)pc.b * c.Hkv + g) * (c.capacity / KV4_SLOTS) + t0 / KV4_SLOTS;
        }
        if (lane == 0) {
          const int s = issued % KD_STAGES;
          const uint32_t bar = smem_u32(&bars[warp][s]), dst = smem_u32(ring + s * 2 * BLK);
          mbar_expect_tx(bar, 2 * BLK);
          bulk_load(dst, static_cast<const uint8_t*>(c.k) + blk * BLK, BLK, bar, pol);
          bulk_load(dst + BLK, static_cast<const uint8_t*>(c.v) + blk * BLK, BLK, bar, pol);
        }
        ++issued;
      }
      ++pw;
      if (pw < w1) kd_next(c, per, pc);
      if (any) return;
    }
  };
  for (int s = 0; s < KD_STAGES; ++s) copy_next();

  long wi = w0;
  while (wi < w1) {
    // ---- one (sequence, head, row block)
    const int b = k.b, q = k.q, g = q / w.nrb, rb = q - g * w.nrb;
    const int len = clamp_len(c, c.len[b]);
    const long n = min((long)(k.nb - k.j), w1 - wi);
    const int j0 = k.j;
    kd_load_q<T, DH, SPLIT>(w, b, g, rb, qf, rs);
    __syncthreads();
    uint32_t qa[STEPS][4];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      *reinterpret_cast<uint4*>(qa[s]) = *reinterpret_cast<const uint4*>(qf + (s * 32 + lane) * 4);
    const float rs0 = rs[g8], rs1 = rs[g8 + 8];
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    for (int j = j0; j < j0 + (int)n; ++j) {
      const int t0 = j * KD_CHUNK + warp * KV4_SLOTS;
      if (t0 >= len) break;
      const int st = taken % KD_STAGES;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][st]), (taken / KD_STAGES) & 1, TC_TIMEOUT_NS))) {
        dead = true;
        drain = taken;
      }
      ++taken;
      if (dead) continue;
      const uint8_t* kb = ring + st * 2 * BLK;
      const uint8_t* vb = kb + BLK;
      // ---- S = Q K^T for 16 keys
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        const int key = nt * 8 + g8;
        uint32_t kw[DH / 32];
        const uint8_t* src = kb + key * (DH / 2) + t4 * (DH / 8);
        if (DH == 128) *reinterpret_cast<uint4*>(kw) = *reinterpret_cast<const uint4*>(src);
        else if (DH == 64) *reinterpret_cast<uint2*>(kw) = *reinterpret_cast<const uint2*>(src);
        else kw[0] = *reinterpret_cast<const uint32_t*>(src);
        const uint8_t* sc = kb + 8 * DH + key * (DH / 16);
#pragma unroll
        for (int x = 0; x < DH / 32; ++x) {
          const __half2 s2 = __half2half2(kv4_scale(sc[(t4 * (DH / 4) + 8 * x) / 16]));
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t b0 = h2u(__hmul2(kv4_pair((kw[x] >> (16 * y)) & 0xffu), s2));
            const uint32_t b1 = h2u(__hmul2(kv4_pair((kw[x] >> (16 * y + 8)) & 0xffu), s2));
            mma16816(s[nt], qa[2 * x + y], b0, b1);
            if (SPLIT) {
              uint32_t ql[4];
              *reinterpret_cast<uint4*>(ql) =
                  *reinterpret_cast<const uint4*>(qf + STEPS * 128 + ((2 * x + y) * 32 + lane) * 4);
              mma16816(s[nt], ql, b0, b1);
            }
          }
        }
      }
      // ---- softmax: a lane has rows g8 (0, 1) and g8 + 8 (2, 3), keys 2 t4 + {0, 1} of each tile
      const bool tail = t0 + KV4_SLOTS > len;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = !tail || t0 + nt * 8 + 2 * t4 + e < len;
          s[nt][e] = in ? s[nt][e] * rs0 : -INFINITY;
          s[nt][2 + e] = in ? s[nt][2 + e] * rs1 : -INFINITY;
        }
      }
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      if (__any_sync(0xffffffffu, x0 > m0 + KD_TOP || x1 > m1 + KD_TOP)) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
        }
        const float n0 = fmaxf(m0, x0 - KD_BACK<SPLIT>), n1 = fmaxf(m1, x1 - KD_BACK<SPLIT>);
        const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - n0), f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[i][0] *= f0; o[i][1] *= f0;
          o[i][2] *= f1; o[i][3] *= f1;
        }
      }
      uint32_t pa[4], pl[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float p0 = ex2_approx(s[nt][0] - m0), p1 = ex2_approx(s[nt][1] - m0);
        const float p2 = ex2_approx(s[nt][2] - m1), p3 = ex2_approx(s[nt][3] - m1);
        l0 += p0 + p1;
        l1 += p2 + p3;
        const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
        pa[2 * nt] = h2u(h0);
        pa[2 * nt + 1] = h2u(h1);
        if (SPLIT) {
          const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
          pl[2 * nt] = half_pair(p0 - f0.x, p1 - f0.y);
          pl[2 * nt + 1] = half_pair(p2 - f1.x, p3 - f1.y);
        }
      }
      // ---- O += P V: lane's keys 2 t4, + 1, + 8, + 9, elements g8 DH/8 + i
      uint32_t vw[4][DH > 64 ? 2 : 1];
      __half2 vs[2];
      __half vh[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = 2 * t4 + (x & 1) + 8 * (x >> 1);
        const uint8_t* src = vb + key * (DH / 2) + g8 * (DH / 16);
        if (DH == 128) *reinterpret_cast<uint2*>(vw[x]) = *reinterpret_cast<const uint2*>(src);
        else if (DH == 64) vw[x][0] = *reinterpret_cast<const uint32_t*>(src);
        else vw[x][0] = *reinterpret_cast<const uint16_t*>(src);
        vh[x] = kv4_scale(vb[8 * DH + key * (DH / 16) + g8 * DH / 128]);
        if (tail && t0 + key >= len) vh[x] = __float2half(0.f);     // p is 0 there: keep 0 * NaN out
      }
      vs[0] = __halves2half2(vh[0], vh[1]);
      vs[1] = __halves2half2(vh[2], vh[3]);
#pragma unroll
      for (int i = 0; i < NT; i += 2) {
        __half2 y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] = kv4_pair((vw[x][i / 8] >> (4 * (i & 7))) & 0xffu);
        const uint32_t a0 = h2u(__hmul2(__lows2half2(y[0], y[1]), vs[0])), a1 = h2u(__hmul2(__lows2half2(y[2], y[3]), vs[1]));
        const uint32_t c0 = h2u(__hmul2(__highs2half2(y[0], y[1]), vs[0])), c1 = h2u(__hmul2(__highs2half2(y[2], y[3]), vs[1]));
        mma16816(o[i], pa, a0, a1);
        mma16816(o[i + 1], pa, c0, c1);
        if (SPLIT) {
          mma16816(o[i], pl, a0, a1);
          mma16816(o[i + 1], pl, c0, c1);
        }
      }
      __syncwarp();                          // every lane has read the stage
      copy_next();
    }
    // ---- join the warps' partials and write the CTA's
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (t4 == 0) {
      ml[warp][g8] = make_float2(m0, l0);
      ml[warp][g8 + 8] = make_float2(m1, l1);
    }
    float* mine = merge + warp * w.rb * ML;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      // columns 2 t4, 2 t4 + 1 of tile i are elements (2 t4) DH/8 + i and (2 t4 + 1) DH/8 + i
      if (g8 < w.rb) {
        mine[g8 * ML + 2 * t4 * (DH / 8) + i] = o[i][0];
        mine[g8 * ML + (2 * t4 + 1) * (DH / 8) + i] = o[i][1];
      }
      if (g8 + 8 < w.rb) {
        mine[(g8 + 8) * ML + 2 * t4 * (DH / 8) + i] = o[i][2];
        mine[(g8 + 8) * ML + (2 * t4 + 1) * (DH / 8) + i] = o[i][3];
      }
    }
    __syncthreads();
    const long pair = (long)b * per + q, slot = pair + blockIdx.x;
    for (int e = tid; e < w.rb * (DH / 4); e += KD_WARPS * 32) {
      const int r = e / (DH / 4), col = (e - r * (DH / 4)) * 4;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int x = 0; x < KD_WARPS; ++x) m = fmaxf(m, ml[x][r].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < KD_WARPS; ++x) {
        const float2 y = ml[x][r];
        if (y.x == -INFINITY) continue;
        const float f = ex2_approx(y.x - m);
        l += f * y.y;
        const float4 v = *reinterpret_cast<const float4*>(merge + (x * w.rb + r) * ML + col);
        acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
      }
      *reinterpret_cast<float4*>(w.part_o + (slot * w.rb + r) * DH + col) = acc;
      if (col == 0) w.part_ml[slot * w.rb + r] = make_float2(m, l);
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
}

// One warp a query row: joins the prefix's partials (o, max, sum), adds the call's own rows the
// row sees, one at a time in float, and rounds the quotient once.  A tree row sees its
// ancestors only (at most 9), so going through the set bits beats a masked product with all n1.
template <typename T, int DH>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const __grid_constant__ Kv4Work w) {
  constexpr int C = DH / 32;
  pdl_wait();
  const Kv4AttnArgs& a = w.a;
  const CacheView& c = a.c;
  const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long)c.B * a.n1 * a.Hq) return;
  const int lane = threadIdx.x & 31;
  const int hq = (int)(row % a.Hq);
  const long bn = row / a.Hq;
  const int node = (int)(bn % a.n1), b = (int)(bn / a.n1);
  const int g = hq / a.G, r = node * a.G + hq - g * a.G;
  const int rb = r / w.rb, in = r - rb * w.rb;
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
  if (clamp_len(c, c.len[b]) > 0) {
    const int2 sp = w.span[((long)b * c.Hkv + g) * w.nrb + rb];
    for (int s = sp.x; s < sp.y; ++s) {
      const long at = (long)s * w.rb + in;
      const float2 y = w.part_ml[at];
      float v[C];
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = w.part_o[at * DH + lane * C + i];
      const float mn = fmaxf(m, y.x);
      if (mn == -INFINITY) continue;
      const float f = ex2_approx(m - mn), h = ex2_approx(y.x - mn);
      m = mn;
      l = l * f + y.y * h;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = o[i] * f + v[i] * h;
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] *= c.gv;
  if (a.tk) {
    const T* q = static_cast<const T*>(a.q) + bn * a.q_row + hq * a.q_head + lane * C;
    float x[C];
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = to_f32(q[i]) * (a.scale * 1.4426950408889634f);
    for (int wd = 0; wd < (a.n1 + 31) / 32; ++wd) {
      uint32_t bits = a.mask ? a.mask[(long)node * 8 + wd]
                             : (node >= 32 * wd + 31 ? 0xffffffffu : node < 32 * wd ? 0u : (2u << (node - 32 * wd)) - 1u);
      if (a.n1 < 32 * wd + 32) bits &= (1u << (a.n1 - 32 * wd)) - 1u;
      while (bits) {
        const int j = 32 * wd + __ffs(bits) - 1;
        bits &= bits - 1;
        const long off = (((long)b * a.n1 + j) * c.Hkv + g) * DH + lane * C;
        const T* kp = static_cast<const T*>(a.tk) + off;
        const T* vp = static_cast<const T*>(a.tv) + off;
        float s = 0.f, v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
          s = fmaf(x[i], to_f32(kp[i]), s);
          v[i] = to_f32(vp[i]);
        }
        s = warp_sum(s);
        const float mn = fmaxf(m, s), f = ex2_approx(m - mn), p = ex2_approx(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = fmaf(p, v[i], o[i] * f);
      }
    }
  }
  T* y = static_cast<T*>(a.o) + bn * a.o_row + hq * a.o_head + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) y[i] = from_f32<T>(l > 0.f ? o[i] / l : 0.f);
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static size_t kd_slots(int B, int Hkv, int nrb, int num_sms) { return (size_t)num_sms * KD_CTAS + (size_t)B * Hkv * nrb; }

size_t kv4_workspace(int B, int Hq, int Hkv, int dh, int max_nodes, int num_sms) {
  size_t most = 0;
  // the largest over the rows a call may have: the slots of 16 rows, or fewer rows in one
  for (int R = Hq / Hkv, n = 1; n <= max_nodes; ++n, R += Hq / Hkv) {
    const int rb = R < KD_ROWS ? R : KD_ROWS, nrb = (R + rb - 1) / rb;
    const size_t slots = kd_slots(B, Hkv, nrb, num_sms);
    const size_t s = up256(slots * rb * dh * 4) + up256(slots * rb * 8) + up256((size_t)B * Hkv * nrb * 8);
    most = s > most ? s : most;
  }
  return most;
}

template <typename T, int DH, bool SPLIT>
static cudaError_t rows_go(const Kv4Work& w, int num_sms, cudaStream_t st) {
  const size_t smem = (size_t)KD_WARPS * KD_STAGES * 2 * kv4_block(DH) + (size_t)KD_WARPS * w.rb * (DH + 4) * 4;
  auto kern = kv4_rows_kernel<T, DH, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if ((e = launch_kernel(kern, dim3(num_sms * KD_CTAS), dim3(KD_WARPS * 32), smem, st, 1, w)) != cudaSuccess) return e;
  const long rows = (long)w.a.c.B * w.a.n1 * w.a.Hq;
  return launch_kernel(kv4_combine_kernel<T, DH>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, 1, w);
}
template <typename T, bool SPLIT>
static cudaError_t rows_dh(const Kv4Work& w, int num_sms, cudaStream_t st) {
  switch (w.a.c.dh) {
    case 32: return rows_go<T, 32, SPLIT>(w, num_sms, st);
    case 64: return rows_go<T, 64, SPLIT>(w, num_sms, st);
    default: return rows_go<T, 128, SPLIT>(w, num_sms, st);
  }
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int dtype, void* ws, int num_sms, cudaStream_t st) {
  Kv4Work w{};
  w.a = a;
  w.R = a.n1 * a.G;
  w.rb = w.R < KD_ROWS ? w.R : KD_ROWS;
  w.nrb = (w.R + w.rb - 1) / w.rb;
  const size_t slots = kd_slots(a.c.B, a.c.Hkv, w.nrb, num_sms);
  char* p = static_cast<char*>(ws);
  w.part_o = reinterpret_cast<float*>(p);
  p += up256(slots * w.rb * a.c.dh * 4);
  w.part_ml = reinterpret_cast<float2*>(p);
  p += up256(slots * w.rb * 8);
  w.span = reinterpret_cast<int2*>(p);
  return dtype == MEDUSA_F32 ? rows_dh<float, true>(w, num_sms, st) : rows_dh<bf16, false>(w, num_sms, st);
}

}  // namespace medusa
