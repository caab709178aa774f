// Products of rows and weights in 8 bits (the format of include/medusa.h) on the tcgen05 tensor cores:
//   y[r][n] = sum_j xs[r][j] ws[n / 128][j] sum_{k in group j} x[r][k] w[n][k]   (+ add), or the gated pair
// silu(x w^T) (x up^T).
//
// A group's scales differ from the next one's, so tensor memory can hold the sum of one group only: the sums
// of a group of 128 (4 MMAs of 32, kind::f8f6f4, float) go to one of two accumulators, and while the next
// group is multiplied, promoting warps read it and add scale times sum to their registers.  Rows are the
// MMA's M (128, a thread's row is its TMEM lane, so that a scale is one number a thread), weight rows its N:
// BN = 256 or 128 columns; a gated tile has 128 columns of either matrix.
//
//   warp 0 (one lane)  copies: rows and weights of a group, 128 bytes a row, through a ring of stages
//   warp 1 (one lane)  MMAs
//   warps 2, 3         scales of the tile's rows and weights, for each group, into a ring in shared memory (read
//                      by the promoting threads themselves, a row each, they took 256 cycles of the L1 a group)
//   warps 4-7, 8-11    promote half the columns each, then write y (or a partial); four warpgroups with a quarter
//                      each are no faster
//
// One CTA per SM.  The work is dealt out by groups: whole tiles while there is one for every CTA, the tiles
// that are left (with few rows: all) as an even share of their groups in one line, so that weights stream
// evenly over the SMs; a CTA that has a part of a tile's groups writes a partial of its own, and a second
// kernel adds a tile's partials up in order and finishes it.
//
// Measured (one GB300, calls in a graph): 8192 x 5120 x 13824 with a residual 581 us (2.0 PFLOP/s), 520 x 15360 x 5120 51 us
// (1.59), gated 688 x 14336 x 4096 99 us (1.63), gated 8 x 13824 x 5120 33 us (4.3 TB/s of weights, 6.6 while they stream),
// 1 x 4096 x 4096 11 us with the rounding before and the joining behind it.  What bounds the large ones: a group takes
// 700 to 950 cycles, its MMAs 512 (8192 multiply-adds a cycle: 256 groups in line, with a commit each or with one); the
// accumulator's way to the promoting warps and back is seen in between (510 cycles to promote), and residuals of 8192 rows
// wait for memory at a tile's end.
//
// Every wait is bounded; on expiry MEDUSA_FLAG_TIMEOUT is set, the CTA stops taking work, drains the copies
// it issued and frees its tensor memory.
#include <algorithm>
#include <cfloat>

#include "f32x2.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace medusa {

constexpr int FL_PROMOTE = 2, FL_THREADS = 128 * (1 + FL_PROMOTE), FL_MAXST = 8;
constexpr uint32_t FL_ROW = 128;                    // bytes of a row in a stage
constexpr int FL_SC = 8;                            // groups in the ring of scales: 128 rows' and two of weights each
// Registers a thread: 168 at launch (384 x 168 = 64512), then 72 for copies and MMAs and 208 to promote:
// 72 + 2 x 208 = 488 <= 3 x 168.
constexpr int FL_REG_ISSUE = 72, FL_REG_PROMOTE = 208;

struct FlArgs {
  CUtensorMap tx, tw[2];                            // rows: box {128, abox}; weights: box {128, 128}
  Fp8LinearArgs a;
  int abox, stages;                                 // rows of a copy (a multiple of 8), ring depth
  uint32_t ring;                                    // bytes of the rings
  int mt, nt;                                       // tiles
  int whole, ctas;                                  // tiles taken whole, CTAs
  int shares;                                       // CTAs that share the groups of the other tiles
  float* part;                                      // [slot][128][BN]
  int rows_last;                                    // weights are read once (mt == 1)
};

// FULL: a stage has landed.  DONE: its products are in an accumulator, and the stage is free (one barrier and one commit
// for both).  TE: an accumulator has been read.  SF, SE: scales have been written, read.  END: every MMA is done.  NEVER:
// nothing arrives (tests).
enum { FB_FULL = 0, FB_DONE = FL_MAXST, FB_TE = 2 * FL_MAXST, FB_SF = FB_TE + 2, FB_SE = FB_SF + FL_SC,
       FB_END = FB_SE + FL_SC, FB_NEVER = FB_END + 1, FB_COUNT = FB_NEVER + 1 };
// A place in the ring of stages (a division by its depth would take longer than what it is needed for).
struct FlRing {
  int st, ph;
  __device__ __forceinline__ void next(int depth) {
    if (++st == depth) {
      st = 0;
      ph ^= 1;
    }
  }
};

__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 D, e4m3 A and B, both K-major, M x N.
constexpr uint32_t idesc_e4m3(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// 16 columns of this thread's TMEM lane.  Until the wait the registers are not there yet: the wait takes them as
// its operands too, so that nothing that reads them can come before it.
__device__ __forceinline__ void fl_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void fl_ld_wait(uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
        "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}

// One stretch of a tile's groups: j .. j + n - 1.
struct FlSeg {
  int m, n0, j, n;                                  // tile row, first weight row
  long slot;                                        // partial; < 0: the whole tile
};
struct FlWalk {
  int tile;                                         // of the whole ones
  long w, w1;                                       // groups of the others
};
// Tile row and column of tile t.  Tiles that run at a time are neighbours: up to FL_GROUP rows of tiles by as many
// columns as there are CTAs for, so that they share rows and weights in the L2 (8192 x 5120 x 13824: 651 MB from memory of
// 268, with all rows of a column first 1204).
constexpr int FL_GROUP = 16;
__device__ __forceinline__ int2 fl_tile(const FlArgs& g, int t) {
  const int first = t / (FL_GROUP * g.nt) * FL_GROUP, rows = min(FL_GROUP, g.mt - first), in = t - first * g.nt;
  return make_int2(first + in % rows, in / rows);
}
__device__ __forceinline__ FlWalk fl_start(const FlArgs& g) {
  const long total = (long)(g.mt * g.nt - g.whole) * g.a.kb;
  if ((int)blockIdx.x >= g.shares) return {(int)blockIdx.x, 0, 0};
  return {(int)blockIdx.x, total * blockIdx.x / g.shares, total * (blockIdx.x + 1) / g.shares};
}
template <int OC> __device__ __forceinline__ bool fl_next(const FlArgs& g, FlWalk& k, FlSeg& s) {
  int t;
  if (k.tile < g.whole) {
    t = k.tile;
    k.tile += g.ctas;
    s.j = 0;
    s.n = g.a.kb;
    s.slot = -1;
  } else {
    if (k.w >= k.w1) return false;
    const int i = (int)(k.w / g.a.kb);
    t = g.whole + i;
    s.j = (int)(k.w - (long)i * g.a.kb);
    s.n = (int)min((long)(g.a.kb - s.j), k.w1 - k.w);
    s.slot = s.n == g.a.kb ? -1 : (long)blockIdx.x + i;
    k.w += s.n;
  }
  const int2 at = fl_tile(g, t);
  s.m = at.x;
  s.n0 = at.y * OC;
  return true;
}

// A group's sums reach 448^2 128 = 2^24.6, so where the product of a row's and a weight scale is no normal float it has lost
// bits that the result needs.  The sum takes one after the other then, the larger one first: it is below
// 2^-126 / 2^-149 = 2^23 and cannot make the sum overflow.
struct FlScale {
  float first, then;
};
__device__ __forceinline__ FlScale fl_apart(float x, float w) {
  if (fabsf(x * w) >= FLT_MIN || x == 0.f || w == 0.f) return {1.f, x * w};
  return fabsf(x) > fabsf(w) ? FlScale{x, w} : FlScale{w, x};
}
// Whether a scale may bring that about (of two without a small one the product is 2^-126 at least).
__device__ __forceinline__ bool fl_small(float s) { return fabsf(s) < 0x1p-63f && s != 0.f; }

// silu(x) u down to x = FL_FAR, from where on 1 + e^-x passes 2^126 (__fdividef gives 0 there, and e^-x an infinity soon).
// There silu(x) = x e^x, which may be no normal float where the product with u is one: it is taken in quarters.
constexpr float FL_FAR = -87.f;
__device__ __forceinline__ float gate_near(float x, float u) { return __fdividef(x, 1.f + expf(-x)) * u; }
__device__ __forceinline__ float gate_far(float x, float u) {
  const float t = expf(0.25f * x);
  return (x * t * t) * (u * t * t);
}
__device__ __forceinline__ float gate(float x, float u) { return x < FL_FAR ? gate_far(x, u) : gate_near(x, u); }

// Four residuals (columns n .. n + 3 of row r), and four results; vec: aligned, and all four exist.
template <typename T> __device__ __forceinline__ void fl_add4(const Fp8LinearArgs& a, long r, int n, bool vec, float (&x)[4]) {
  const T* src = static_cast<const T*>(a.add) + r * a.add_row + n;
  if (vec) {
    load4(src, true, x);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = n + e < a.n ? to_f32(src[e]) : 0.f;
  }
}
template <typename T> __device__ __forceinline__ void fl_save4(const Fp8LinearArgs& a, long r, int n, bool vec, const float (&y)[4]) {
  T* dst = static_cast<T*>(a.y) + r * a.y_row + n;
  if (vec) {
    save4(dst, true, y);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.n) dst[e] = from_f32<T>(y[e]);
  }
}

// A warp's 32 rows x 16 columns, a row a lane (v), turned in shared memory (`turn`, 2 KB of the warp) so that four
// lanes have a row's 16 columns, four each, and a store writes whole sectors (a row a lane: 32 sectors a store, 8 bytes
// of each; 27,000 cycles a tile of 128 x 256).  The 16-byte units of a row change places by its number, so that
// neither way meets a bank twice.  f(step, row, column, four values) for each.
template <typename F> __device__ __forceinline__ void fl_turn(float4* turn, int lane, const float2 (&v)[8], F f) {
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    turn[lane * 4 + (u ^ ((lane >> 1) & 3))] = make_float4(v[2 * u].x, v[2 * u].y, v[2 * u + 1].x, v[2 * u + 1].y);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2);
    const float4 x = turn[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
    float y[4] = {x.x, x.y, x.z, x.w};
    f(i, row, (lane & 3) * 4, y);
  }
}
template <typename T> __device__ __forceinline__ bool fl_vec(const Fp8LinearArgs& a) {
  const uintptr_t n = 4 * sizeof(T);
  return (uintptr_t)a.y % n == 0 && a.y_row % 4 == 0 && (uintptr_t)a.add % n == 0 && a.add_row % 4 == 0;
}

template <typename T, int BN, bool GATED>
__global__ void __launch_bounds__(FL_THREADS, 1) fp8_linear_kernel(const __grid_constant__ FlArgs g) {
  constexpr int OC = GATED ? BN / 2 : BN;            // results of a tile's row
  constexpr int HC = BN / FL_PROMOTE;                // columns a promoting thread adds up
  constexpr int GQ = HC / 32;                        // gated: 16 columns' steps of either matrix
  constexpr uint32_t WB = BN * FL_ROW;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[FB_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ float s_x[FL_SC][128], s_w[FL_SC][2];   // scales
  __shared__ int2 s_small[FL_SC];                    // whether there is a small one among them (of either warp's)
  __shared__ int s_issued, s_waited, s_abort;
  const Fp8LinearArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ST = g.stages;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ws = base, xs = base + ST * WB;     // the rows' ring comes last: an MMA reads 128 rows from a stage
  const uint32_t xb = g.abox * FL_ROW;               // of abox, and what lies behind goes to lanes that no row has
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(bar(FB_FULL + i), 1);
      mbar_init(bar(FB_DONE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(FB_TE + i), 4 * FL_PROMOTE);
    }
    for (int i = 0; i < FL_SC; ++i) {
      mbar_init(bar(FB_SF + i), 64);
      mbar_init(bar(FB_SE + i), 4 * FL_PROMOTE);
    }
    mbar_init(bar(FB_END), 1);
    mbar_init(bar(FB_NEVER), 1);
    s_issued = s_waited = s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), 2 * BN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();                          // only once this CTA holds its TMEM
  const uint32_t tmem = tmem_slot;
  bool timed_out = false;
  auto aborted = [&]() { return *(volatile int*)&s_abort != 0; };
  FlWalk walk = fl_start(g);
  FlSeg s;
  FlRing k = {0, 0};
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FL_REG_ISSUE));
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ copies
      const uint64_t pol_w = g.rows_last ? policy_evict_first() : policy_evict_last(), pol_x = policy_evict_last();
      // weights are written by no kernel of this call: the first stages' go out before the wait for the rows
      FlWalk ahead = walk;
      int pre = 0, c = 0;
      auto load_w = [&](const FlSeg& q, int j, int st) {
        mbar_expect_tx(bar(FB_FULL + st), WB + xb);
#pragma unroll
        for (int h = 0; h < BN / 128; ++h)
          tma_load_2d(ws + st * WB + h * 128 * FL_ROW, GATED ? &g.tw[h] : &g.tw[0], j * 128, GATED ? q.n0 : q.n0 + 128 * h,
                      bar(FB_FULL + st), pol_w);
      };
      while (pre < ST && fl_next<OC>(g, ahead, s))
        for (int i = 0; i < s.n && pre < ST; ++i) load_w(s, s.j + i, pre++);
      s_issued = pre;
      pdl_wait();
      while (!timed_out && fl_next<OC>(g, walk, s)) {
        for (int i = 0; i < s.n; ++i, ++c) {
          if (c >= pre) {
            if (c >= ST && !mbar_wait(bar(FB_DONE + k.st), k.ph ^ 1, TC_TIMEOUT_NS)) { timed_out = true; break; }
            load_w(s, s.j + i, k.st);
            s_issued = c + 1;
          }
          tma_load_2d(xs + k.st * xb, &g.tx, (s.j + i) * 128, s.m * 128, bar(FB_FULL + k.st), pol_x);
          k.next(ST);
        }
        if (aborted()) break;
      }
      for (; c < pre; ++c)                           // (left early) a stage's weights are in flight: let it fill
        tma_load_2d(xs + c * xb, &g.tx, 0, 0, bar(FB_FULL + c), pol_x);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ MMAs
      const uint32_t idesc = idesc_e4m3(128, BN);
      int c = 0;
      if (a.test_wait_ns) timed_out = !mbar_wait(bar(FB_NEVER), 0, a.test_wait_ns);
      while (!timed_out && fl_next<OC>(g, walk, s)) {
        for (int i = 0; i < s.n; ++i, ++c) {
          const int buf = c & 1;
          if (!mbar_wait(bar(FB_FULL + k.st), k.ph, TC_TIMEOUT_NS)) { timed_out = true; break; }
          s_waited = c + 1;
          if (!mbar_wait(bar(FB_TE + buf), ((c >> 1) & 1) ^ 1, TC_TIMEOUT_NS)) { timed_out = true; break; }
          tc_fence_after();
          const uint64_t da = sw128_desc(xs + k.st * xb), db = sw128_desc(ws + k.st * WB);
#pragma unroll
          for (int q = 0; q < 4; ++q) umma_e4m3(tmem + buf * BN, da + 2 * q, db + 2 * q, idesc, q > 0);
          umma_commit(bar(FB_DONE + k.st));
          k.next(ST);
        }
        if (aborted()) break;
      }
      umma_commit(bar(FB_END));                      // arrives once every MMA issued above is done
    } else if (warp >= 2) {
      // ------------------------------------------------------------ scales: rows t and t + 64 of a tile a thread
      const int t = tid - 64;
      const bool quads = a.kb % 4 == 0 && ((uintptr_t)a.xs & 15) == 0;
      pdl_wait();
      int c = 0;
      while (!timed_out && fl_next<OC>(g, walk, s)) {
        const float* x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = a.xs + min((long)s.m * 128 + t + 64 * h, (long)a.rows - 1) * a.kb;
        // the weights' scales: of the two blocks of columns, or of the two matrices (one thread each)
        const int last = (a.n - 1) / 128;
        const float* w = a.ws[GATED ? t & 1 : 0] + (long)min(s.n0 / 128 + (GATED ? 0 : t & 1), last) * a.kb;
        for (int i = s.j & ~3; i < s.j + s.n && !timed_out; i += 4) {      // four groups' loads at a time
          float f[2][4], u[4] = {};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (quads) {
              const float4 v = *reinterpret_cast<const float4*>(x[h] + i);
              f[h][0] = v.x;
              f[h][1] = v.y;
              f[h][2] = v.z;
              f[h][3] = v.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) f[h][e] = x[h][min(i + e, a.kb - 1)];
            }
          }
          if (t < 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = w[min(i + e, a.kb - 1)];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (i + e < s.j || i + e >= s.j + s.n || timed_out) continue;
            const int at = c % FL_SC;
            if (!__all_sync(0xffffffffu, mbar_wait(bar(FB_SE + at), ((c / FL_SC) & 1) ^ 1, TC_TIMEOUT_NS))) {
              timed_out = true;
              continue;
            }
            s_x[at][t] = f[0][e];
            s_x[at][t + 64] = f[1][e];
            if (t < 2) s_w[at][t] = u[e];
            const int small = __any_sync(0xffffffffu, fl_small(f[0][e]) || fl_small(f[1][e]) || fl_small(u[e]));
            if (lane == 0) (warp == 2 ? s_small[at].x : s_small[at].y) = small;
            mbar_arrive(bar(FB_SF + at));
            ++c;
          }
        }
        if (aborted()) break;
      }
    }
  } else {
    // -------------------------------------------------------------- promote
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FL_REG_PROMOTE));
    const int part = (warp >> 2) - 1, wl = warp & 3;
    // columns of this thread: HC from part * HC on, or (gated) HC / 2 of either matrix
    const uint32_t lanes = tmem + ((uint32_t)(wl * 32) << 16);
    pdl_wait();
    int c = 0;
    while (!timed_out && fl_next<OC>(g, walk, s)) {
      const bool live = (long)s.m * 128 + wl * 32 < a.rows;
      float2 acc[HC / 2];
#pragma unroll
      for (int i = 0; i < HC / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int i = 0; i < s.n; ++i, ++c) {
        const int buf = c & 1, at = c % FL_SC;
        bool got = mbar_wait(bar(FB_SF + at), (c / FL_SC) & 1, TC_TIMEOUT_NS);
        const float x = s_x[at][wl * 32 + lane], w0 = s_w[at][GATED || BN == 128 ? 0 : part], w1 = GATED ? s_w[at][1] : w0;
        float s0 = x * w0, s1 = x * w1;
        const int2 small = s_small[at];
        got = got && mbar_wait(bar(FB_DONE + k.st), k.ph, TC_TIMEOUT_NS);
        if (!__all_sync(0xffffffffu, got)) {
          timed_out = true;
          break;
        }
        k.next(ST);
        tc_fence_after();
        if (live) {
          // 16 columns on their way while 16 are added up (gated: of the first matrix, then of the second)
          auto col = [&](int q) { return lanes + buf * BN + (GATED ? (q / GQ) * 128 + part * (HC / 2) + (q % GQ) * 16 : part * HC + q * 16); };
          if (small.x | small.y) {                     // (in tensor memory: a second copy of the loop below is slower by more, also where none is small)
            const FlScale f0 = fl_apart(x, w0), f1 = fl_apart(x, w1);
#pragma unroll 1
            for (int q = 0; q < HC / 16; ++q) {
              uint32_t v[16];
              float y[16];
              fl_ld16(col(q), v);
              fl_ld_wait(v);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(v[e]) * (GATED && q >= GQ ? f1.first : f0.first);
              tmem_st16(col(q), y);
            }
            s0 = f0.then;
            s1 = f1.then;
          }
          uint32_t v[2][16];
          fl_ld16(col(0), v[0]);
#pragma unroll
          for (int q = 0; q < HC / 16; ++q) {
            fl_ld_wait(v[q & 1]);
            if (q + 1 < HC / 16) fl_ld16(col(q + 1), v[(q + 1) & 1]);
            const float sc = GATED && q >= GQ ? s1 : s0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              acc[q * 8 + e] = fma2(make_float2(__uint_as_float(v[q & 1][2 * e]), __uint_as_float(v[q & 1][2 * e + 1])),
                                    make_float2(sc, sc), acc[q * 8 + e]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(FB_TE + buf));
          mbar_arrive(bar(FB_SE + at));
        }
      }
      if (timed_out || !live) continue;
      float4* turn = reinterpret_cast<float4*>(smem_raw + (base - smem_u32(smem_raw)) + g.ring) + (warp - 4) * 128;
      const int r0 = s.m * 128 + wl * 32, rows = min(32, a.rows - r0);      // (rows < 2^24)
      if (s.slot >= 0) {
#pragma unroll
        for (int q = 0; q < HC / 16; ++q) {
          float2 v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[q * 8 + e];
          float* dst = g.part + (s.slot * 128 + wl * 32) * BN + (GATED ? (q / GQ) * 128 + part * (HC / 2) + (q % GQ) * 16 : part * HC + q * 16);
          fl_turn(turn, lane, v, [&](int, int row, int c4, float (&y)[4]) {
            if (row < rows) *reinterpret_cast<float4*>(dst + row * BN + c4) = make_float4(y[0], y[1], y[2], y[3]);
          });
        }
      } else {
        constexpr int N = GATED ? HC / 2 : HC;
        const bool al = fl_vec<T>(a);
#pragma unroll
        for (int q = 0; q < N / 16; ++q) {
          const int n = s.n0 + part * N + q * 16 + (lane & 3) * 4;
          const bool vec = al && n + 4 <= a.n;
          float2 v[8];
          float lo = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = acc[q * 8 + e];
            if constexpr (GATED) {
              lo = fminf(lo, fminf(v[e].x, v[e].y));
              v[e] = make_float2(gate_near(v[e].x, acc[HC / 4 + q * 8 + e].x), gate_near(v[e].y, acc[HC / 4 + q * 8 + e].y));
            }
          }
          if (GATED && __any_sync(0xffffffffu, lo < FL_FAR)) {       // (a branch for each: gated trees 103 -> 119 us)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 x = acc[q * 8 + e], u = acc[HC / 4 + q * 8 + e];
              if (x.x < FL_FAR) v[e].x = gate_far(x.x, u.x);
              if (x.y < FL_FAR) v[e].y = gate_far(x.y, u.y);
            }
          }
          float add[4][4] = {};                        // all asked for before the first store
          if (!GATED && a.add) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = i * 8 + (lane >> 2);
              if (row < rows && n < a.n) fl_add4<T>(a, r0 + row, n, vec, add[i]);
            }
          }
          fl_turn(turn, lane, v, [&](int i, int row, int, float (&y)[4]) {
            if (row < rows && n < a.n) {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] += add[i][e];
              fl_save4<T>(a, r0 + row, n, vec, y);
            }
          });
        }
      }
    }
  }
  if (timed_out) {
    set_flag(a.status, MEDUSA_FLAG_TIMEOUT);
    *(volatile int*)&s_abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    // every MMA done, then the copies issued but never waited for (bounded)
    mbar_wait(bar(FB_END), 0, TC_TIMEOUT_NS);
    for (int c = s_waited; c < s_issued; ++c) mbar_wait(bar(FB_FULL + c % ST), (c / ST) & 1, TC_TIMEOUT_NS / 16);
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 2 * BN);
}

// Adds up the partials of the tiles that several CTAs had a part of: with W groups over C CTAs group x is
// CTA ceil((x + 1) C / W) - 1's.  A thread has four results of a row.
template <typename T, int BN, bool GATED>
__global__ void __launch_bounds__(256) fp8_join_kernel(const __grid_constant__ FlArgs g) {
  constexpr int OC = GATED ? BN / 2 : BN, Q = OC / 4, SB = 4;
  pdl_trigger();
  const Fp8LinearArgs& a = g.a;
  const int i = blockIdx.x, t = g.whole + i;
  const int2 tile = fl_tile(g, t);
  const int m = tile.x, n0 = tile.y * OC;
  const long total = (long)(g.mt * g.nt - g.whole) * a.kb, x = (long)i * a.kb;
  auto cta = [&](long w) { return ((w + 1) * g.shares + total - 1) / total - 1; };
  const long c0 = cta(x), c1 = cta(x + a.kb - 1);
  const int e = blockIdx.y * 256 + threadIdx.x, row = e / Q, col = (e - row * Q) * 4;
  const long r = (long)m * 128 + row;
  pdl_wait();
  if (c0 == c1 || row >= 128 || r >= a.rows) return;
  const float* src = g.part + ((c0 + i) * 128 + row) * BN + col;
  float y[4] = {}, u[4] = {};
  for (long c = c0; c <= c1; c += SB) {
    float4 p[SB], q[SB];
#pragma unroll
    for (int b = 0; b < SB; ++b) {
      p[b] = q[b] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + b <= c1) {
        p[b] = *reinterpret_cast<const float4*>(src + (c + b - c0) * 128 * BN);
        if (GATED) q[b] = *reinterpret_cast<const float4*>(src + (c + b - c0) * 128 * BN + 128);
      }
    }
#pragma unroll
    for (int b = 0; b < SB; ++b) {
      y[0] += p[b].x;
      y[1] += p[b].y;
      y[2] += p[b].z;
      y[3] += p[b].w;
      u[0] += q[b].x;
      u[1] += q[b].y;
      u[2] += q[b].z;
      u[3] += q[b].w;
    }
  }
  const bool vec = fl_vec<T>(a) && n0 + col + 4 <= a.n;
  if (GATED) {
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = gate(y[q], u[q]);
  } else if (a.add) {
    float add[4];
    fl_add4<T>(a, r, n0 + col, vec, add);
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] += add[q];
  }
  fl_save4<T>(a, r, n0 + col, vec, y);
}

// ------------------------------------------------------------------ host side
static bool make_map(CUtensorMap* map, const void* p, long k, long rows, long row, int box) {
  auto fn = tma_encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row};
  const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call of `rows` rows is cut up.
struct FlPlan {
  int bn, mt, nt, whole, ctas, shares;
};
static FlPlan fl_plan(int rows, int n, int kb, bool gated, int num_sms) {
  FlPlan p;
  p.mt = (rows + 127) / 128;
  // Columns of a tile.  With one row of tiles 128 share the weights more evenly as long as tiles of 256 are for less than half
  // of the CTAs, and are slower from there on; with more, 256 load each row half as often.  128 / 256, in us: 1 x 4096 x 4096
  // 10.2 / 10.6; over 15360 x 5120 (60 tiles of 256) 1 row 22.5 / 21.3, 64 24.3 / 25.8, 128 23.6 / 32.8; over 20480 x 4096 (80)
  // 25.6 / 21.7, 31.7 / 26.8, 32.8 / 24.9; over 32000 x 4096 (125) 31.0 / 28.2, 34.8 / 29.7, 34.8 / 30.2; over 48000 x 4096 (188)
  // 41.7 / 41.4, 47.1 / 48.4, 49.1 / 53.4; over 64000 x 4096 (250) 53.3 / 48.9, 58.6 / 52.9, 61.2 / 54.9; 200 x 15360 x 5120
  // 37.5 / 27.5, 520 x 4096 x 4096 28.1 / 23.0.
  p.bn = gated || p.mt > 1 || 2 * ((n + 255) / 256) >= num_sms ? 256 : 128;
  const int oc = gated ? 128 : p.bn;
  p.nt = (n + oc - 1) / oc;
  const long tiles = (long)p.mt * p.nt;
  p.whole = (int)(tiles / num_sms * num_sms);
  // The last tiles whole, too, or in shares: shares save the time in which CTAs without a tile would wait, and cost
  // partials that go through memory and a kernel that joins them.  In microseconds: a group of a tile takes 0.35,
  // or with one row of tiles, where weights are waited for, 0.36 a 16 KB of them; partials 1.5 and what their bytes
  // take at 4 TB/s.
  const long over = tiles - p.whole;
  const double group = p.mt > 1 ? 0.35 : 0.36 * p.bn / 128, rows1 = rows < 128 ? rows : 128;
  const double saved = kb * group * (1.0 - (double)over / num_sms);
  const double cost = 1.5 + 2.0 * (over + num_sms) * rows1 * p.bn * 4 / 4e6;
  if (over > 0 && saved < cost) p.whole = (int)tiles;
  const long left = tiles - p.whole;
  p.shares = (int)std::min<long>(num_sms, left * kb);
  p.ctas = p.whole ? (int)std::min<long>(num_sms, tiles) : p.shares;
  return p;
}

Fp8Tiles fp8_linear_tiles(int rows, int n, int kb, bool gated, int num_sms) {
  const FlPlan p = fl_plan(rows, n, kb, gated, num_sms);
  const int left = p.mt * p.nt - p.whole, shared = p.shares == left ? 0 : left;       // (as many CTAs as tiles: one each)
  return {p.bn, p.mt * p.nt - shared, shared};
}

size_t fp8_linear_partials(int max_rows, int n, int kb, int num_sms) {
  // tiles that are left are fewer than CTAs, and a tile has no more shares than groups
  const size_t tiles = (size_t)((max_rows + 127) / 128) * ((n + 127) / 128);
  return std::min<size_t>(2 * (size_t)num_sms, tiles * (1 + (size_t)kb)) * 128 * 256 * sizeof(float);
}

template <typename T, int BN, bool GATED> static cudaError_t linear_go(FlArgs& g, cudaStream_t st) {
  static unsigned long long allowed = 0;
  constexpr size_t turn = 4 * FL_PROMOTE * 2048, limit = 222 * 1024;
  const size_t stage = BN * FL_ROW + g.abox * FL_ROW, fixed = 1024 + (128 - g.abox) * FL_ROW;
  g.stages = (int)std::min<size_t>(FL_MAXST, (limit - fixed - turn) / stage);
  g.ring = (uint32_t)(fixed - 1024 + g.stages * stage);
  cudaError_t e = allow_smem(fp8_linear_kernel<T, BN, GATED>, limit, &allowed);
  if (e != cudaSuccess) return e;
  e = launch_kernel(fp8_linear_kernel<T, BN, GATED>, dim3(g.ctas), dim3(FL_THREADS), fixed + g.stages * stage + turn, st, 1, g);
  const int left = g.mt * g.nt - g.whole;
  if (e != cudaSuccess || left == 0 || g.shares == left) return e;      // (every CTA has one tile: no partials)
  const int rows = std::min(g.a.rows, 128);
  return launch_kernel(fp8_join_kernel<T, BN, GATED>, dim3(left, (rows * (GATED ? BN / 8 : BN / 4) + 255) / 256), dim3(256), 0, st, 1, g);
}

template <typename T> static cudaError_t linear_type(FlArgs& g, int bn, cudaStream_t st) {
  if (g.a.w[1]) return linear_go<T, 256, true>(g, st);
  return bn == 128 ? linear_go<T, 128, false>(g, st) : linear_go<T, 256, false>(g, st);
}

cudaError_t launch_fp8_linear(const Fp8LinearArgs& a, int dtype, void* part, int num_sms, cudaStream_t st) {
  const bool gated = a.w[1] != nullptr;
  const FlPlan p = fl_plan(a.rows, a.n, a.kb, gated, num_sms);
  FlArgs g{};
  g.a = a;
  g.abox = std::min(128, (a.rows + 7) / 8 * 8);
  g.mt = p.mt;
  g.nt = p.nt;
  g.whole = p.whole;
  g.ctas = p.ctas;
  g.shares = p.shares;
  g.part = static_cast<float*>(part);
  g.rows_last = p.mt == 1;
  if (!make_map(&g.tx, a.x, a.k, a.rows, a.x_row, g.abox) || !make_map(&g.tw[0], a.w[0], a.k, a.n, a.k, 128) ||
      (gated && !make_map(&g.tw[1], a.w[1], a.k, a.n, a.k, 128)))
    return cudaErrorInvalidValue;
  return dtype == MEDUSA_F32 ? linear_type<float>(g, p.bn, st) : linear_type<bf16>(g, p.bn, st);
}

}  // namespace medusa
