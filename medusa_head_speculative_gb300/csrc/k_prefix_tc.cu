// Attention over a shared prefix on the tcgen05 tensor cores: bf16, dh 64 or 128 ("Medusa: Simple LLM
// Inference Acceleration Framework with Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5; how the
// work is dealt out is in prefix.cuh).
//
// For each row r, with s_j = scale q_r . k_j over the keys j it sees: o_r = sum_j 2^(s'_j - m_r) v_j and
// l_r = sum_j 2^(s'_j - m_r), s' in base-2 units, m_r a running reference that is raised (and o rescaled)
// only once a score passes it by PT_LAZY, o and l in float, probabilities rounded to bf16 for the product: the MMA takes
// both operands in one type, and values are bf16.  Results are then 0.0023 off the 64-bit ones (relative, over listed cases), of
// which 0.0017 are their own rounding.  Probabilities as two summands of bf16, multiplied one after the other, keep 16 bits and
// give 0.0017, but the cases below take 58, 96 and 152 us for 52, 81 and 118 (calls from Python): not worth it.
//
// One CTA per SM walks through its chunks of 128 keys, an item at a time.  A block of rows is one tile of 128
// or two.  In the CTA
//
//   warps 12-15  copies of keys and values into rings of stages: whole chunks of a contiguous cache by the
//                copy engine; paged caches, last chunks and the call's own rows with 16-byte copies (a row
//                from the length on is filled with zeros).  The call's own values pass through registers:
//                a row's infinities and NaN become 0 there and the key is noted, since rows that do not
//                see it multiply it by 0; a row that does gets a NaN sum
//   warps 8, 9   MMAs of a "slot" each, with S (128 columns) and O (dh columns) in tensor memory: S = Q K^T,
//                then O += P V with P read from tensor memory and V from shared memory (MN-major)
//   warps 10, 11 copies of the queries; with one tile a block ahead
//   warps 0-3,   two softmax warpgroups, one per slot, one query row per thread: they read S,
//   4-7          exponentiate and write P over it, 32 keys at a time (all 64 of a half unrolled made the
//                warps of a CTA wait for instructions)
//
// With two tiles the slots are the tiles and share every chunk; with one both slots work on it and take
// alternate chunks, and the first warpgroup merges the second's (O, reference, sum) before it writes the
// partial (of an item's only chunk its slot writes it).
//
// Measured (one GB300), joining included: 16 x 8 heads x 172 rows over a prefix of 8192 and 64-512 slots 115 us (830
// TFLOP/s; heads of 64 99 us, 490), 8 x 40 heads x 65 rows over 2048 + 0-1024 76 us, 32 x 8 heads x 4 rows over 16384 +
// 100-1000 slots in pages of 16 49 us (2.8 TB/s).  What bounds them: with two tiles a chunk takes 5000 cycles, its MMAs 2050 and the softmax of a
// slot 2900 (instructions a warp at a time; exponentials alone 2050 for both slots); pages of 16 slots come by
// 16-byte copies, 4000 cycles a chunk; items of few chunks have their start and end besides.  Code size counts here:
// more unrolling of the copies or the softmax makes every warp slower (64 keys at a time 112 -> 129 us).
//
// A wait names a phase by its parity: a waiter has to have seen the phase before.  With one tile a slot
// sees every other chunk of the CTA, odd or even ones over all its items, and the rings are of two or four
// stages, so that a stage is always the same slot's.
// Every wait is bounded; on expiry MEDUSA_FLAG_TIMEOUT is set, the CTA stops taking work, lets its MMAs and
// copies end, also those that nobody came to wait for, and frees its tensor memory.
#include <algorithm>

#include "attn_mma.cuh"
#include "launch.cuh"
#include "prefix.cuh"
#include "tma_host.h"

namespace medusa {

constexpr int PT_ROWS = 128, PT_MAXST = 4, PT_MMA_WARP = 8, PT_QUERY_WARP = 10, PT_COPY_WARP = 12, PT_THREADS = 512;
// Registers a thread: 128 at launch (512 x 128 = 65536), then 2 x 160 + 2 x 96 = 4 x 128.
constexpr int PT_REG_SOFTMAX = 160, PT_REG_REST = 96;
static_assert(2 * PT_REG_SOFTMAX + 2 * PT_REG_REST == 4 * 128, "what the launch holds");
constexpr uint32_t PT_SLOT_COLS = 256;              // per slot: S / P [0, 128), O [128, 128 + dh)
constexpr float PT_LAZY = 8.f;

struct PtArgs {
  CUtensorMap tk[2], tv[2];                         // shared, own: dims {dh, Hkv, slots}, box {64, 1, 128}
  int tma[2];                                       // whole chunks come by them
  PxWork w;
  int nt[2], sk[2], sv[2];                          // shared, own: tiles of a block, stages of the rings
  int qb[2];                                        // blocks of queries there is room for
};

// QF / QE: query tiles (with one tile: two in turn) written / no longer read.  KF and VF: stages full.  Per slot
// and stage: SF (S written, so that the keys' stage is free as far as the slot goes), OF (P V done, the values'
// stage).  Per slot: P1 and P2 (P of the first 64 keys, of all written), O1 (P V of the first done).  One barrier for
// both who wait (with four commits a chunk's QK and PV took 1390 cycles in this kernel; such MMAs by themselves take 1024, also
// with four commits among them).  MRG / MFR: the second slot's (reference, sum) are in shared
// memory / consumed.  END: every MMA issued has completed.  NEVER: nothing arrives (tests).
enum {
  XB_QF = 0, XB_QE = 2, XB_KF = 4, XB_VF = XB_KF + PT_MAXST, XB_SF = XB_VF + PT_MAXST, XB_OF = XB_SF + 2 * PT_MAXST,
  XB_P1 = XB_OF + 2 * PT_MAXST, XB_P2 = XB_P1 + 2, XB_O1 = XB_P2 + 2, XB_MRG = XB_O1 + 2, XB_MFR = XB_MRG + 1,
  XB_END = XB_MFR + 1, XB_NEVER = XB_END + 1, XB_COUNT = XB_NEVER + 1
};

// Of chunk j (pc: chunks of cached slots, len of them): whether it is of the call's own rows, its keys, and
// whether the copy engine brings it.
__device__ __forceinline__ int pt_keys(const PrefixArgs& a, int j, int pc, int len) {
  return min((j < pc ? len : a.n1) - (j < pc ? j : j - pc) * PX_KEYS, PX_KEYS);
}
__device__ __forceinline__ bool pt_engine(const PtArgs& g, int kind, int j, int len) {
  return g.tma[kind] && (long)(j + 1) * PX_KEYS <= len;
}

// A place in a ring of stages that is walked through in steps (a division by its depth, which is no constant,
// would take longer than what it is needed for).
struct PtRing {
  int st, ph;
  __device__ __forceinline__ void next(int by, int depth) {
    st += by;
    if (st >= depth) {
      st -= depth;
      ph ^= 1;
    }
  }
};

// A value that all lanes have, as the compiler can tell: what an MMA takes comes from uniform registers, and moving
// an operand there costs as much as half an MMA (16 MMAs of a job 1800 cycles to issue, 1025 to run).
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }

template <int DH>
__global__ void __launch_bounds__(PT_THREADS, 1) prefix_tc_kernel(const __grid_constant__ PtArgs g) {
  constexpr int H = DH / 64;                         // 64-element halves of a head
  constexpr uint32_t TILE = 128 * 128;               // one half of a tile: 128 rows of 128 bytes
  constexpr uint32_t CHUNK = H * TILE;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[XB_COUNT];
  __shared__ uint32_t tmem_slot, s_bad[8][4];        // keys of the call's own rows whose values are not finite
  __shared__ int s_abort, s_copied;                  // s_copied: chunks whose copies have begun
  __shared__ float2 s_ml[PT_ROWS];                   // second slot's (reference, sum) per row
  const PxWork& w = g.w;
  const PrefixArgs& a = w.a;
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  pdl_wait();
  const PxPlan plan = px_plan(w, blockIdx.x == 0 && warp == PT_QUERY_WARP);
  if ((int)blockIdx.x >= plan.cs + plan.co) {
    pdl_trigger();
    return;
  }
  PxWalk walk = px_start(w, plan, blockIdx.x);
  const bool shared = uni(walk.shared);
  const int kind = shared ? 0 : 1, nt = g.nt[kind], SK = g.sk[kind], SV = g.sv[kind], QB = g.qb[kind];
  const CacheView& c = shared ? a.shared : a.own;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t qs = base, k0s = base + nt * QB * CHUNK, v0s = k0s + SK * CHUNK;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(XB_QF + i), 64);
      mbar_init(bar(XB_QE + i), 2);
    }
    for (int i = 0; i < PT_MAXST; ++i) {
      mbar_init(bar(XB_KF + i), 128);
      mbar_init(bar(XB_VF + i), 128);
    }
    for (int s = 0; s < 2 * PT_MAXST; ++s) {
      mbar_init(bar(XB_SF + s), 1);
      mbar_init(bar(XB_OF + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(XB_P1 + s), PT_ROWS);
      mbar_init(bar(XB_P2 + s), PT_ROWS);
      mbar_init(bar(XB_O1 + s), 1);
    }
    mbar_init(bar(XB_MRG), PT_ROWS);
    mbar_init(bar(XB_MFR), PT_ROWS);
    mbar_init(bar(XB_END), 2);
    mbar_init(bar(XB_NEVER), 1);
    s_abort = s_copied = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == PT_MMA_WARP) tmem_alloc(smem_u32(&tmem_slot), 2 * PT_SLOT_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();                          // only once this CTA holds its TMEM
  const uint32_t tmem = (uint32_t)uni((int)tmem_slot);
  bool timed_out = false;
  auto aborted = [&]() { return *(volatile int*)&s_abort != 0; };
  PxSeg s;

  if (warp >= PT_COPY_WARP) {
    // ------------------------------------------------------------ copies
    reg_fewer<PT_REG_REST>();
    constexpr int UPR = DH / 8, RPI = 32 / UPR;      // 16-byte units of a row, rows a step of the warp
    const int pw = warp - PT_COPY_WARP, unit = lane % UPR, sub = lane / UPR;
    const uint64_t pol = shared ? policy_evict_last() : policy_evict_first();
    const bool boss = pw == 0 && lane == 0;
    int x = 0, trees = 0;                            // chunks, chunks of the call's own rows so far
    PtRing ring[2] = {{0, 0}, {0, 0}};
    auto abandon = [&](bool got) { timed_out = !got; return !got; };
    while (!timed_out && px_next(w, walk, s)) {
      const int b = shared ? 0 : s.b, len = clamp_len(c, c.len[b]), pc = (len + PX_KEYS - 1) / PX_KEYS;
      // The page of the warp's row `lane` of chunk j, asked for a chunk ahead and not looked at before (a warp
      // that needs it at once waits for memory); and the row's first element (< 0: none).
      auto page_of = [&](int j) {
        const int t = j * PX_KEYS + 32 * pw + lane;
        return c.page_table && j < pc && t < len ? c.page_table[(long)b * c.pages_per_seq + t / c.page_size] : b;
      };
      auto offset = [&](int j, int page) -> long {
        const int t = (j < pc ? j : j - pc) * PX_KEYS + 32 * pw + lane;
        if (j >= pc) return t < a.n1 ? (((long)b * a.n1 + t) * c.Hkv + s.g) * DH : -1;
        if (t >= len) return -1;
        if (c.page_table && (page < 0 || page >= c.num_pages)) {
          set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
          page = 0;
        }
        return plain_offset(c, page, c.page_table ? t % c.page_size : t, s.g);
      };
      int page = page_of(s.j);
      for (int i = 0; i < s.n; ++i, ++x) {
        const int j = s.j + i;
        const bool tree = j >= pc, engine = pt_engine(g, kind, j, len);
        const long at = offset(j, page);
        if (i + 1 < s.n) page = page_of(j + 1);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const int n = part ? SV : SK, st = part ? ring[1].st : ring[0].st;
          const uint32_t full = bar((part ? XB_VF : XB_KF) + st), dst = (part ? v0s : k0s) + st * CHUNK;
          // the stage's last chunk has been multiplied by the slots that took it
          if (x >= n) {
            const int done = (part ? XB_OF : XB_SF) + st, ph = part ? ring[1].ph : ring[0].ph;
            bool got = true;
            if (nt == 2 || !(st & 1)) got = kt_warp_wait(bar(done), ph ^ 1);
            if (got && (nt == 2 || (st & 1))) got = kt_warp_wait(bar(done + PT_MAXST), ph ^ 1);
            if (abandon(got)) break;
          }
          if (engine) {
            if (boss) {
              mbar_expect_tx(full, CHUNK);
#pragma unroll
              for (int h = 0; h < H; ++h)
                tma_load_3d(dst + h * TILE, part ? &g.tv[kind] : &g.tk[kind], h * 64, s.g, b * c.capacity + j * PX_KEYS, full, pol);
            } else {
              mbar_arrive(full);
            }
            continue;
          }
          const bf16* src = static_cast<const bf16*>(tree ? (part ? a.tv : a.tk) : (part ? c.v : c.k));
          const uint32_t to = dst + (unit >> 3) * TILE;
          if (tree && part) {
            uint32_t bad = 0;
            constexpr int FLY = 8;                       // loads in flight a lane
#pragma unroll 1
            for (int y0 = 0; y0 < UPR; y0 += FLY) {
              uint4 v[FLY];
#pragma unroll
              for (int y = 0; y < FLY; ++y) {
                const long o = __shfl_sync(0xffffffffu, at, (y0 + y) * RPI + sub);
                v[y] = make_uint4(0u, 0u, 0u, 0u);
                if (o >= 0) v[y] = *reinterpret_cast<const uint4*>(src + o + unit * 8);
              }
#pragma unroll
              for (int y = 0; y < FLY; ++y) {
                const uint32_t words[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
                bool no = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  no |= (words[e] & 0x7f80u) == 0x7f80u || (words[e] & 0x7f800000u) == 0x7f800000u;
                if (no) v[y] = make_uint4(0u, 0u, 0u, 0u);
                const uint32_t hit = __ballot_sync(0xffffffffu, no);
#pragma unroll
                for (int e = 0; e < RPI; ++e)
                  if ((hit >> (e * UPR)) & ((1u << UPR) - 1u)) bad |= 1u << ((y0 + y) * RPI + e);
                const int r = 32 * pw + (y0 + y) * RPI + sub;
                st_shared16(to + r * 128 + (((unit & 7) ^ (r & 7)) << 4), v[y].x, v[y].y, v[y].z, v[y].w);
              }
            }
            if (lane == 0) s_bad[trees & 7][pw] = bad;
            fence_proxy_async();
            mbar_arrive(full);
          } else {
            if (__all_sync(0xffffffffu, at >= 0)) {
              const char* from = reinterpret_cast<const char*>(src + unit * 8);
              const uint32_t key = 32 * pw + sub;
#pragma unroll 4
              for (int y = 0; y < UPR; ++y) {
                const uint32_t r = key + y * RPI;
                const long o = __shfl_sync(0xffffffffu, at, y * RPI + sub);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + r * 128 + (((unit & 7) ^ (r & 7)) << 4)), "l"(from + 2 * o));
              }
            } else {
#pragma unroll 4
              for (int y = 0; y < UPR; ++y) {
                const int row = y * RPI + sub, r = 32 * pw + row;
                const long o = __shfl_sync(0xffffffffu, at, row);
                cp_async16(to + r * 128 + (((unit & 7) ^ (r & 7)) << 4), o >= 0 ? src + o + unit * 8 : src, o >= 0 ? 16 : 0);
              }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
          }
        }
        if (timed_out) break;
        ring[0].next(1, SK);
        ring[1].next(1, SV);
        trees += tree;
      }
      if (aborted()) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (boss) s_copied = x + timed_out;              // (given up between a chunk's keys and its values: the keys count)
  } else if (warp >= PT_MMA_WARP) {
    // ------------------------------------------------------------ MMAs of one slot
    reg_fewer<PT_REG_REST>();
    if (warp < PT_QUERY_WARP) {
      const int slot = warp - PT_MMA_WARP;
      const uint32_t lead = lane == 0;
      const uint32_t id_qk = idesc_bf16(PT_ROWS, PX_KEYS), id_half = idesc_bf16(PT_ROWS, PX_KEYS / 2);
      const uint32_t id_pv = idesc_bf16(PT_ROWS, DH) | IDESC_B_MN_MAJOR;
      // descriptors hold addresses in 16-byte units: an offset is added to them
      const uint64_t dq = sw128_desc(qs + (nt == 2 ? slot : 0) * CHUNK), dk = sw128_desc(k0s), dv = sw128_desc_mn(v0s, TILE);
      const uint32_t sp = tmem + slot * PT_SLOT_COLS, od = sp + PX_KEYS;
      const int step = nt == 2 ? 1 : 2;                  // two tiles: every chunk; one: alternate ones
      int gc = 0, qn = 0, mc = 0;         // chunks, blocks and merged blocks so far
      int done = 0, halves = 0;           // this slot's chunks with rows so far, and those of more than 64 keys
      bool dead = a.test_wait_ns && slot == 0 && !__all_sync(0xffffffffu, mbar_wait(bar(XB_NEVER), 0, a.test_wait_ns));
      int pc = 0, len = 0;                // of the item's cache
      PtRing kr = {nt == 2 ? 0 : slot, 0}, vr = kr;  // (rings have two stages at least)
      // a stage written by 16-byte copies (the generic proxy) is made visible to the MMAs
      auto wait_k = [&](int j) {
        const bool got = kt_warp_wait(bar(XB_KF + kr.st), kr.ph);
        if (!pt_engine(g, kind, j, len)) fence_proxy_async();
        return got;
      };
      auto wait_v = [&](int j) {
        const bool got = kt_warp_wait(bar(XB_VF + vr.st), vr.ph);
        if (!pt_engine(g, kind, j, len)) fence_proxy_async();
        return got;
      };
      uint64_t q = dq;                    // the block's queries
      auto two = [&](int j) { return pt_keys(a, j, pc, len) > PX_KEYS / 2; };   // whether a chunk has a second half
      auto scores = [&](int j) {
        kt_qk<H>(sp, q, dk + kr.st * (CHUNK >> 4), two(j) ? id_qk : id_half, lead);
        kt_commit(bar(XB_SF + slot * PT_MAXST + kr.st), lead);
        kr.next(step, SK);
      };
      while (!dead && px_next(w, walk, s)) {
        const int n = uni(s.n), j0 = uni(s.j);
        const bool idle = uni(nt == 2 && s.rb * 2 * PT_ROWS + slot * PT_ROWS >= (shared ? w.rows : w.R));
        const int i0 = nt == 2 ? 0 : (slot - gc) & 1;    // this slot's first chunk
        len = uni(clamp_len(c, c.len[shared ? 0 : s.b]));
        pc = (len + PX_KEYS - 1) / PX_KEYS;
        const int qb = QB == 1 ? 0 : qn & 1;
        if (!kt_warp_wait(bar(XB_QF + qb), (QB == 1 ? qn : qn >> 1) & 1)) { dead = true; break; }
        fence_proxy_async();
        tc_fence_after();
        q = dq + qb * (CHUNK >> 4);
        if (idle) {                                      // no rows: only let the stages go
          for (int i = 0; i < n; ++i) {
            if (!wait_k(j0 + i) || !wait_v(j0 + i)) { dead = true; break; }
            kt_commit(bar(XB_SF + slot * PT_MAXST + kr.st), lead);
            kt_commit(bar(XB_OF + slot * PT_MAXST + vr.st), lead);
            kr.next(1, SK);
            vr.next(1, SV);
          }
        } else if (i0 < n) {
          if (!wait_k(j0 + i0)) { dead = true; break; }
          scores(j0 + i0);
          if (i0 + step >= n) kt_commit(bar(XB_QE + qb), lead);
#pragma unroll 1
          for (int i = i0; i < n && !dead; i += step) {
            const int j = j0 + i;
            const uint64_t v = dv + vr.st * (CHUNK >> 4);
            // one tile: slot 1's O may be overwritten only after the first warpgroup has merged it into the
            // previous block's partial
            if (nt == 1 && slot == 1 && i == i0 && mc > 0 && !kt_warp_wait(bar(XB_MFR), (mc - 1) & 1)) { dead = true; break; }
            if (!wait_v(j)) { dead = true; break; }
            const bool both = two(j), more = i + step < n;
            if (both) {
              if (!kt_warp_wait(bar(XB_P1 + slot), halves & 1)) { dead = true; break; }
              ++halves;
              tc_fence_after();
              kt_pv(od, sp, v, id_pv, i != i0, lead);
              kt_commit(bar(XB_O1 + slot), lead);
            }
            if (!kt_warp_wait(bar(XB_P2 + slot), done & 1)) { dead = true; break; }
            ++done;
            tc_fence_after();
            if (both) kt_pv(od, sp + 32, v + 512, id_pv, 1, lead);
            else kt_pv(od, sp, v, id_pv, i != i0, lead);
            kt_commit(bar(XB_OF + slot * PT_MAXST + vr.st), lead);
            vr.next(step, SV);
            if (more) {
              if (!wait_k(j + step)) { dead = true; break; }
              scores(j + step);
              if (i + 2 * step >= n) kt_commit(bar(XB_QE + qb), lead);
            }
          }
        }
        if (idle || i0 >= n) kt_commit(bar(XB_QE + qb), lead);
        ++qn;
        mc += nt == 1 && n > 1;
        gc += n;
        if (aborted()) break;
      }
      timed_out = dead;
      kt_commit(bar(XB_END), lead);                      // arrives once this warp's MMAs are done
    } else {
      // ---------------------------------------------------------- copies of queries
      constexpr int UPR = DH / 8, RPI = 32 / UPR;        // 16-byte units of a row, rows a step of the warp
      const int unit = lane % UPR, sub = lane / UPR;
      const bf16* src = static_cast<const bf16*>(a.q);
      for (int qn = 0; px_next(w, walk, s); ++qn) {
        const int qb = QB == 1 ? 0 : qn & 1, turn = QB == 1 ? qn : qn >> 1;
        const uint32_t to = qs + qb * CHUNK + (unit >> 3) * TILE;
        for (int r0 = 32 * (warp - PT_QUERY_WARP); r0 < nt * PT_ROWS; r0 += 64) {
          const PxRow row = px_row(w, shared, s, r0 + lane);
          const long at = row.ok ? row.node_row * a.q_row + row.head * a.q_head : -1;
          if (r0 < 64 && !kt_warp_wait(bar(XB_QE + qb), (turn & 1) ^ 1)) { timed_out = true; break; }
#pragma unroll 4
          for (int y = 0; y < UPR; ++y) {
            const long o = __shfl_sync(0xffffffffu, at, y * RPI + sub);
            const int r = r0 + y * RPI + sub;
            cp_async16(to + (r >> 7) * CHUNK + (r & 127) * 128 + (((unit & 7) ^ (r & 7)) << 4), o >= 0 ? src + o + unit * 8 : src, o >= 0 ? 16 : 0);
          }
        }
        if (timed_out) break;
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(XB_QF + qb)) : "memory");
        if (aborted()) break;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    reg_more<PT_REG_SOFTMAX>();
    const int slot = warp >> 2, wl = warp & 3;
    const int r = wl * 32 + lane;                    // row within the tile = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(wl * 32) << 16);
    const uint32_t scol = lane_base + slot * PT_SLOT_COLS;      // this slot's S / P
    const uint32_t ocol = scol + PX_KEYS;                       // this slot's O
    const float sl2 = a.scale2;
    const int rbrows = shared ? w.rbs : w.rbo;
    float* part_o = shared ? w.o_s : w.o_o;
    float2* part_ml = shared ? w.ml_s : w.ml_o;
    int mc = 0, trees = 0, gc = 0;
    // places of this slot's next chunk in the rings, of its last one (values), and of slot 1's (merging warpgroup)
    PtRing kr = {nt == 2 ? 0 : slot, 0}, vr = kr, last = kr, other = {1, 0}, last1 = other;
    const int step = nt == 2 ? 1 : 2;
    int parts = 0;                                   // this slot's chunks of more than 64 keys so far
    while (px_next(w, walk, s)) {
      const int n = s.n, b = shared ? 0 : s.b, len = clamp_len(c, c.len[b]), pc = (len + PX_KEYS - 1) / PX_KEYS;
      const int tile = nt == 2 ? slot : 0;
      const int br = tile * PT_ROWS + r;             // row of the block
      const PxRow row = px_row(w, shared, s, br);
      const bool live = __any_sync(0xffffffffu, row.ok);
      const bool idle = nt == 2 && s.rb * 2 * PT_ROWS + slot * PT_ROWS >= (shared ? w.rows : w.R);
      const int i0 = nt == 2 ? 0 : (slot - gc) & 1;
      const int njobs = idle ? 0 : nt == 2 ? n : (n + 1 - i0) / 2;
      float m_use = -INFINITY, l_acc = 0.f;
      for (int i = 0; idle && i < n && !timed_out; ++i) {            // (phases have to be seen one by one)
        timed_out = !kt_warp_wait(bar(XB_SF + slot * PT_MAXST + kr.st), kr.ph);
        kr.next(1, SK);
        vr.next(1, SV);
      }
      for (int jj = 0; jj < njobs; ++jj) {
        const int j = s.j + i0 + (nt == 2 ? jj : 2 * jj);
        const bool tree = j >= pc;
        const int keys = pt_keys(a, j, pc, len);
        if (!kt_warp_wait(bar(XB_SF + slot * PT_MAXST + kr.st), kr.ph)) { timed_out = true; break; }
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < (keys > PX_KEYS / 2 ? 4 : 2); ++q) {
          if (live) {
            float v[32];
            kt_ld32(scol + 32 * q, v);
            const int valid = keys - 32 * q;
            const uint32_t see = tree ? (row.ok ? px_sees(a, row.n, (j - pc) * 4 + q) : 0u)
                                      : valid >= 32 ? 0xffffffffu : valid <= 0 ? 0u : (1u << valid) - 1u;
            if (__any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see >> e) & 1u)) v[e] = -INFINITY;
            }
            // Against the reference as it is, the largest score found on the way; where it passes the reference
            // by PT_LAZY (a row's first keys, and hardly ever later) the reference is raised and all is done again.
            uint32_t pk[16];
            float sum;
#pragma unroll 1
            for (;;) {
              const float nm = m_use == -INFINITY ? 0.f : -m_use;   // (nothing seen yet: every score is -infinity)
              F2 l0 = f2(0.f, 0.f), l1 = l0;
              float x0 = v[0], x1 = v[1];
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float p0, p1, p2, p3;
                unf2(fma2(f2(v[e], v[e + 1]), f2(sl2, sl2), f2(nm, nm)), p0, p1);
                unf2(fma2(f2(v[e + 2], v[e + 3]), f2(sl2, sl2), f2(nm, nm)), p2, p3);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                p2 = ex2_approx(p2);
                p3 = ex2_approx(p3);
                l0 = add2(l0, f2(p0, p1));
                l1 = add2(l1, f2(p2, p3));
                pk[e / 2] = pack2(p0, p1);
                pk[e / 2 + 1] = pack2(p2, p3);
                x0 = max3(x0, v[e], v[e + 1]);
                x1 = max3(x1, v[e + 2], v[e + 3]);
              }
              float a0, a1;
              unf2(add2(l0, l1), a0, a1);
              sum = a0 + a1;
              const float mx = fmaxf(x0, x1) * sl2;
              const bool raise = mx > m_use + PT_LAZY;   // (from -infinity: any score)
              if (!__any_sync(0xffffffffu, raise)) break;
              const float f = !raise ? 1.f : m_use == -INFINITY ? 0.f : ex2_approx(m_use - mx);
              // O may be rescaled: the products of the chunks before are done (this S came after them), those of
              // this chunk's first half are waited for
              const bool mixed = q > 1;
              if (mixed && !kt_warp_wait(bar(XB_O1 + slot), (parts - 1) & 1)) { timed_out = true; break; }
              tc_fence_after();
              if (jj > 0 || mixed) {
#pragma unroll 1
                for (int e = 0; e < DH; e += 16) {
                  float u[16];
                  kt_ld16(ocol + e, u);
#pragma unroll
                  for (int y = 0; y < 16; ++y) u[y] *= f;
                  tmem_st16(ocol + e, u);
                }
              }
              kt_st_wait();
#pragma unroll 1
              for (int e = q & 2; e < q; ++e) {          // and so is P that has not been multiplied
                float u[16];
                uint32_t scaled[16];
                kt_ld16(scol + 16 * e, u);
#pragma unroll
                for (int y = 0; y < 16; ++y)
                  scaled[y] = pack2(__uint_as_float(__float_as_uint(u[y]) << 16) * f,
                                     __uint_as_float(__float_as_uint(u[y]) & 0xffff0000u) * f);
                kt_st16(scol + 16 * e, scaled);
              }
              l_acc *= f;
              if (raise) m_use = mx;
            }
            if (timed_out) break;
            l_acc += sum;
            kt_st16(scol + 16 * q, pk);
          }
          if (q == 1 && keys > PX_KEYS / 2) {
            kt_st_wait();
            tc_fence_before();
            mbar_arrive(bar(XB_P1 + slot));
            ++parts;
          }
        }
        if (timed_out) break;
        kt_st_wait();
        tc_fence_before();
        mbar_arrive(bar(XB_P2 + slot));
        last = vr;
        kr.next(step, SK);
        vr.next(step, SV);
      }
      if (timed_out) break;
      // ---- the block's partial
      const long prow = s.slot * rbrows + br;
      float* dst = part_o + prow * DH;
      // a row that sees a value which is not finite has a NaN sum (the copies' notes are in shared memory once
      // the last P V is done)
      const int first_tree = max(s.j, pc), n_trees = max(s.j + n - first_tree, 0);
      auto noted = [&]() {
        bool bad = false;
#pragma unroll 1
        for (int q = 0; q < n_trees; ++q)
#pragma unroll 1
          for (int u = 0; u < 4; ++u)
            bad |= row.ok && (px_sees(a, row.n, (first_tree - pc + q) * 4 + u) & *(volatile uint32_t*)&s_bad[(trees + q) & 7][u]) != 0u;
        return bad;
      };
      if (nt == 2 || n == 1) {
        if (nt == 1 && njobs == 0) other.next(2, SV);     // (the merging warpgroup follows the other's chunks)
        if (njobs > 0 && live) {
          if (!kt_warp_wait(bar(XB_OF + slot * PT_MAXST + last.st), last.ph)) { timed_out = true; break; }
          tc_fence_after();
          if (n_trees > 0 && noted()) l_acc = NAN;
          if (l_acc != l_acc && m_use == -INFINITY) m_use = 0.f;
#pragma unroll 2
          for (int e = 0; e < DH; e += 16) {
            float v[16];
            kt_ld16(ocol + e, v);
            const int quad = br - (lane & 3);
            store_quads<DH>(dst - (lane & 3) * DH + e, min(rbrows - quad, (shared ? w.rows : w.R) - s.rb * rbrows - quad), lane, v);
          }
          if (row.ok) part_ml[prow] = make_float2(m_use, l_acc);
        }
        tc_fence_before();
      } else if (slot == 1) {
        // hand (reference, sum) to the first warpgroup once it has consumed the previous ones
        if (mc > 0 && !kt_warp_wait(bar(XB_MFR), (mc - 1) & 1)) { timed_out = true; break; }
        s_ml[r] = make_float2(m_use, l_acc);
        mbar_arrive(bar(XB_MRG));
        ++mc;
      } else {
        const int nj1 = n - njobs;                   // slot 1's chunks in this block (either may have none)
        for (int i = 0; i < nj1; ++i) {
          last1 = other;
          other.next(2, SV);
        }
        bool ok = njobs == 0 || kt_warp_wait(bar(XB_OF + last.st), last.ph);
        // the second slot's softmax first: it ends once all of its products but the last are done
        if (ok) ok = kt_warp_wait(bar(XB_MRG), mc & 1);
        if (ok && nj1 > 0) ok = kt_warp_wait(bar(XB_OF + PT_MAXST + last1.st), last1.ph);
        if (!ok) { timed_out = true; break; }
        tc_fence_after();
        const float2 ml1 = s_ml[r];
        const float m = fmaxf(m_use, ml1.x);
        const float f0 = m_use == -INFINITY ? 0.f : ex2_approx(m_use - m);
        const float f1 = ml1.x == -INFINITY ? 0.f : ex2_approx(ml1.x - m);
        // (a sum that is NaN with nothing else seen keeps its NaN)
        float l = (l_acc != l_acc ? l_acc : l_acc * f0) + (ml1.y != ml1.y ? ml1.y : ml1.y * f1);
        if (n_trees > 0 && noted()) l = NAN;
        const uint32_t ocol1 = lane_base + PT_SLOT_COLS + PX_KEYS;
        if (live) {
#pragma unroll 2
          for (int e = 0; e < DH; e += 16) {
            float v0[16], v1[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v0[q] = v1[q] = 0.f;
            if (njobs > 0) kt_ld16(ocol + e, v0);
            if (nj1 > 0) kt_ld16(ocol1 + e, v1); // written by this block's P V of slot 1
            if (row.ok) {
#pragma unroll
              for (int q = 0; q < 16; q += 4)
                *reinterpret_cast<float4*>(dst + e + q) =
                    make_float4(v0[q] * f0 + v1[q] * f1, v0[q + 1] * f0 + v1[q + 1] * f1,
                                v0[q + 2] * f0 + v1[q + 2] * f1, v0[q + 3] * f0 + v1[q + 3] * f1);
            }
          }
          if (row.ok) part_ml[prow] = make_float2(l != l && m == -INFINITY ? 0.f : m, l);
        }
        tc_fence_before();
        mbar_arrive(bar(XB_MFR));
        ++mc;
      }
      trees += n_trees;
      gc += n;
    }
  }
  if (timed_out) {
    kt_st_wait();                                    // (a softmax warp may have left in the middle of a chunk)
    set_flag(a.status, MEDUSA_FLAG_TIMEOUT);
    *(volatile int*)&s_abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    mbar_wait(bar(XB_END), 0, TC_TIMEOUT_NS);        // every MMA done
    // and, where the block gave up, each ring's last copies: a stage that a consumer did not come to may still be written
    // (without all arrivals its phase does not end, and the limit is far beyond the time of a copy)
    if (aborted())
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        const int n = part ? SV : SK;
#pragma unroll 1
        for (int y = max(0, s_copied - n); y < s_copied; ++y)
          mbar_wait(bar((part ? XB_VF : XB_KF) + y % n), (y / n) & 1, TC_TIMEOUT_NS / 16);
      }
  }
  __syncthreads();
  if (warp == PT_MMA_WARP) tmem_dealloc(tmem, 2 * PT_SLOT_COLS);
}

// ------------------------------------------------------------------ host side
// (The CUDA cores' kernel in place of this one: 16 x 43 nodes of 4 x 8 heads of 128 over 8192 slots 3.66 ms for 115 us, 32 single
// rows over 16384 687 us for 49.  Float rows it takes alone, and heads of 32, for which this one has not been built: the
// same nodes take 1.25 ms with heads of 32 and 99 us with heads of 64.)
bool prefix_tc_takes(int dtype, int dh) { return dtype == MEDUSA_BF16 && (dh == 64 || dh == 128); }

static bool make_map(CUtensorMap* map, const void* p, const CacheView& c) {
  auto fn = tma_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)c.dh, (cuuint64_t)c.Hkv, (cuuint64_t)c.B * c.capacity};
  const cuuint64_t strides[2] = {(cuuint64_t)c.dh * 2, (cuuint64_t)c.dh * c.Hkv * 2};
  const cuuint32_t box[3] = {64, 1, PX_KEYS}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH> static cudaError_t tc_go(PtArgs& g, cudaStream_t st) {
  constexpr size_t CHUNK = DH / 64 * 128 * 128, limit = 225 * 1024;
  static unsigned long long done = 0;
  for (int kind = 0; kind < 2; ++kind) {
    // with one tile a block's queries are copied a block ahead where blocks are short, of a few chunks (8 x 65 nodes
    // 78.0 -> 76.5 us; with long ones, the shared kind's, it is the same either way)
    g.qb[kind] = g.nt[kind] == 1 && kind == 1 ? 2 : 1;
    const int stages = (int)((limit - 1024) / CHUNK) - g.nt[kind] * g.qb[kind];
    if (g.nt[kind] == 1) {                           // even depths: see above
      g.sk[kind] = stages >= 6 ? 4 : 2;
      g.sv[kind] = stages - g.sk[kind] >= 4 ? 4 : 2;
    } else {
      g.sv[kind] = std::min(PT_MAXST, stages / 2);
      g.sk[kind] = std::min(PT_MAXST, stages - g.sv[kind]);
    }
  }
  const cudaError_t e = allow_smem(prefix_tc_kernel<DH>, limit, &done);
  if (e != cudaSuccess) return e;
  return launch_kernel(prefix_tc_kernel<DH>, dim3(g.w.ctas), dim3(PT_THREADS), limit, st, 1, g);
}

cudaError_t launch_prefix_tc(const PxWork& w, cudaStream_t st) {
  PtArgs g{};
  g.w = w;
  g.nt[0] = w.rbs > PT_ROWS ? 2 : 1;
  g.nt[1] = w.rbo > PT_ROWS ? 2 : 1;
  const CacheView* caches[2] = {&w.a.shared, &w.a.own};
  for (int kind = 0; kind < 2; ++kind) {
    const CacheView& c = *caches[kind];
    // coordinates are 32 bits wide; paged caches have no chunk in one piece
    if (c.page_table || (double)c.B * c.capacity >= 2147483648.0) continue;
    g.tma[kind] = 1;
    if (!make_map(&g.tk[kind], c.k, c) || !make_map(&g.tv[kind], c.v, c)) return cudaErrorInvalidValue;
  }
  return w.a.own.dh == 128 ? tc_go<128>(g, st) : tc_go<64>(g, st);
}

}  // namespace medusa
