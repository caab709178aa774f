// Attention over a shared prefix on the tcgen05 tensor cores: bf16, dh 64 or 128 ("Medusa: Simple LLM
// Inference Acceleration Framework with Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5; how the
// work is dealt out is in prefix.cuh).
//
// For each row r, with s_j = scale q_r . k_j over the keys j it sees: o_r = sum_j 2^(s'_j - m_r) v_j and
// l_r = sum_j 2^(s'_j - m_r), s' in base-2 units, m_r a running reference that is raised (and o rescaled)
// only once a score passes it by PT_LAZY, o and l in float, probabilities rounded to bf16 for the product.
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
//                then O += P V with P read from tensor memory and V from shared memory (MN-major), in
//                halves of 64 keys: while the softmax has one half, the other half's P is multiplied with
//                V and the next chunk's scores take its place
//   warps 0-3,   two softmax warpgroups, one per slot, one query row per thread: they load the block's
//   4-7          queries, read a half of S, exponentiate and write P over it
//
// With two tiles the slots are the tiles and share every chunk; with one both slots work on it and take
// alternate chunks, and the first warpgroup merges the second's (O, reference, sum) before it writes the
// partial.
//
// A wait names a phase by its parity: a waiter has to have seen the phase before.  With one tile a slot
// sees every other chunk of the CTA, odd or even ones over all its items, and the rings are of two or four
// stages, so that a stage is always the same slot's.
// Every wait is bounded; on expiry MEDUSA_FLAG_TIMEOUT is set, the CTA stops taking work, lets its MMAs and
// copies end and frees its tensor memory.
#include <algorithm>

#include "attn_mma.cuh"
#include "launch.cuh"
#include "prefix.cuh"
#include "tma_host.h"

namespace medusa {

constexpr int PT_ROWS = 128, PT_MAXST = 4, PT_MMA_WARP = 8, PT_COPY_WARP = 12, PT_THREADS = 512;
// Registers a thread: 128 at launch (512 x 128 = 65536), then 2 x 176 + 2 x 80 = 4 x 128.
constexpr int PT_REG_SOFTMAX = 176, PT_REG_REST = 80;
static_assert(2 * PT_REG_SOFTMAX + 2 * PT_REG_REST == 4 * 128, "what the launch holds");
constexpr uint32_t PT_SLOT_COLS = 256;              // per slot: S / P [0, 128), O [128, 128 + dh)
constexpr float PT_LAZY = 8.f;

struct PtArgs {
  CUtensorMap tk[2], tv[2];                         // shared, own: dims {dh, Hkv, slots}, box {64, 1, 128}
  int tma[2];                                       // whole chunks come by them
  PxWork w;
  int nt[2], sk[2], sv[2];                          // shared, own: tiles of a block, stages of the rings
};

// QF / QE: query tiles written / no longer read.  KF / KE and VF / VE: stages full / free.  Per slot and half:
// SF (S written), PR (P written), OF (P V done).  MRG / MFR: the second slot's (reference, sum) are in shared
// memory / consumed.  END: every MMA issued has completed.
enum {
  XB_QF = 0, XB_QE = 1, XB_KF = 2, XB_KE = XB_KF + PT_MAXST, XB_VF = XB_KE + PT_MAXST, XB_VE = XB_VF + PT_MAXST,
  XB_SF = XB_VE + PT_MAXST, XB_PR = XB_SF + 4, XB_OF = XB_PR + 4, XB_MRG = XB_OF + 4, XB_MFR = XB_MRG + 1,
  XB_END = XB_MFR + 1, XB_COUNT = XB_END + 1
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

template <int DH>
__global__ void __launch_bounds__(PT_THREADS, 1) prefix_tc_kernel(const __grid_constant__ PtArgs g) {
  constexpr int H = DH / 64;                         // 64-element halves of a head
  constexpr uint32_t TILE = 128 * 128;               // one half of a tile: 128 rows of 128 bytes
  constexpr uint32_t CHUNK = H * TILE;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[XB_COUNT];
  __shared__ uint32_t tmem_slot, s_bad[8][4];        // keys of the call's own rows whose values are not finite
  __shared__ int s_abort;
  __shared__ float2 s_ml[PT_ROWS];                   // second slot's (reference, sum) per row
  const PxWork& w = g.w;
  const PrefixArgs& a = w.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const PxPlan plan = px_plan(w, blockIdx.x == 0 && warp == PT_MMA_WARP + 2);
  if ((int)blockIdx.x >= plan.cs + plan.co) {
    pdl_trigger();
    return;
  }
  PxWalk walk = px_start(w, plan, blockIdx.x);
  const bool shared = walk.shared;
  const int kind = shared ? 0 : 1, nt = g.nt[kind], SK = g.sk[kind], SV = g.sv[kind];
  const CacheView& c = shared ? a.shared : a.own;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t qs = base, k0s = base + nt * CHUNK, v0s = k0s + SK * CHUNK;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    mbar_init(bar(XB_QF), nt * PT_ROWS);
    mbar_init(bar(XB_QE), 2);
    for (int i = 0; i < PT_MAXST; ++i) {
      mbar_init(bar(XB_KF + i), 128);
      mbar_init(bar(XB_KE + i), nt);
      mbar_init(bar(XB_VF + i), 128);
      mbar_init(bar(XB_VE + i), nt);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(XB_SF + s), 1);
      mbar_init(bar(XB_PR + s), PT_ROWS);
      mbar_init(bar(XB_OF + s), 1);
    }
    mbar_init(bar(XB_MRG), PT_ROWS);
    mbar_init(bar(XB_MFR), PT_ROWS);
    mbar_init(bar(XB_END), 2);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == PT_MMA_WARP) tmem_alloc(smem_u32(&tmem_slot), 2 * PT_SLOT_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();                          // only once this CTA holds its TMEM
  const uint32_t tmem = tmem_slot;
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
    auto abandon = [&](bool got) { timed_out = !got; return !got; };
    while (!timed_out && px_next(w, walk, s)) {
      const int b = shared ? 0 : s.b, len = clamp_len(c, c.len[b]), pc = (len + PX_KEYS - 1) / PX_KEYS;
      // first element of the warp's row `lane` of chunk j (< 0: none)
      auto offset = [&](int j) -> long {
        const int t = (j < pc ? j : j - pc) * PX_KEYS + 32 * pw + lane;
        if (j >= pc) return t < a.n1 ? (((long)b * a.n1 + t) * c.Hkv + s.g) * DH : -1;
        if (t >= len) return -1;
        long u;
        int in;
        if (!unit_of(c, b, t, u, in)) {
          set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
          u = 0;
        }
        return plain_offset(c, u, in, s.g);
      };
      long next = offset(s.j);
      for (int i = 0; i < s.n; ++i, ++x) {
        const int j = s.j + i;
        const bool tree = j >= pc, engine = !tree && g.tma[kind] && (j + 1) * PX_KEYS <= len;
        const long at = next;
        if (i + 1 < s.n) next = offset(j + 1);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const int n = part ? SV : SK, st = x % n;
          const uint32_t full = bar((part ? XB_VF : XB_KF) + st), dst = (part ? v0s : k0s) + st * CHUNK;
          if (abandon(kt_warp_wait(bar((part ? XB_VE : XB_KE) + st), ((x / n) & 1) ^ 1))) break;
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
#pragma unroll 4
            for (int y = 0; y < UPR; ++y) {
              const int row = y * RPI + sub;
              const long o = __shfl_sync(0xffffffffu, at, row);
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (o >= 0) v = *reinterpret_cast<const uint4*>(src + o + unit * 8);
              const uint32_t words[4] = {v.x, v.y, v.z, v.w};
              bool no = false;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                no |= (words[e] & 0x7f80u) == 0x7f80u || (words[e] & 0x7f800000u) == 0x7f800000u;
              if (no) v = make_uint4(0u, 0u, 0u, 0u);
              const uint32_t hit = __ballot_sync(0xffffffffu, no);
#pragma unroll
              for (int e = 0; e < RPI; ++e)
                if ((hit >> (e * UPR)) & ((1u << UPR) - 1u)) bad |= 1u << (y * RPI + e);
              const int r = 32 * pw + row;
              st_shared16(to + r * 128 + (((unit & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
            }
            if (lane == 0) s_bad[trees & 7][pw] = bad;
            fence_proxy_async();
            mbar_arrive(full);
          } else {
#pragma unroll 4
            for (int y = 0; y < UPR; ++y) {
              const int row = y * RPI + sub, r = 32 * pw + row;
              const long o = __shfl_sync(0xffffffffu, at, row);
              cp_async16(to + r * 128 + (((unit & 7) ^ (r & 7)) << 4), o >= 0 ? src + o + unit * 8 : src, o >= 0 ? 16 : 0);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
          }
        }
        if (timed_out) break;
        trees += tree;
      }
      if (aborted()) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the last copies of each ring: if the block gives up nobody else waits for them (bounded)
    if (boss && (timed_out || aborted()))
      for (int part = 0; part < 2; ++part) {
        const int n = part ? SV : SK;
        for (int y = max(0, x - n); y < x; ++y) mbar_wait(bar((part ? XB_VF : XB_KF) + y % n), (y / n) & 1, TC_TIMEOUT_NS / 16);
      }
  } else if (warp >= PT_MMA_WARP) {
    // ------------------------------------------------------------ MMAs of one slot
    reg_fewer<PT_REG_REST>();
    if (warp < PT_MMA_WARP + 2) {
      const int slot = warp - PT_MMA_WARP;
      const uint32_t lead = lane == 0;
      const uint32_t id_qk = idesc_bf16(PT_ROWS, PX_KEYS / 2);
      const uint32_t id_pv = idesc_bf16(PT_ROWS, DH) | IDESC_B_MN_MAJOR;
      // descriptors hold addresses in 16-byte units: an offset is added to them
      const uint64_t dq = sw128_desc(qs + (nt == 2 ? slot : 0) * CHUNK), dk = sw128_desc(k0s), dv = sw128_desc_mn(v0s, TILE);
      const uint32_t sp = tmem + slot * PT_SLOT_COLS, od = sp + PX_KEYS;
      const int step = nt == 2 ? 1 : 2;                  // two tiles: every chunk; one: alternate ones
      int gc = 0, qn = 0, js = 0;         // chunks, blocks and this slot's jobs so far
      bool dead = false;
      // stages may have been written by 16-byte copies (the generic proxy): make them visible to the MMAs
      auto wait_k = [&](int x) {
        const bool got = kt_warp_wait(bar(XB_KF + x % SK), (x / SK) & 1);
        fence_proxy_async();
        return got;
      };
      auto wait_v = [&](int x) {
        const bool got = kt_warp_wait(bar(XB_VF + x % SV), (x / SV) & 1);
        fence_proxy_async();
        return got;
      };
      auto scores = [&](int x, int hf) {
        kt_qk<H>(sp + 64 * hf, dq, dk + (x % SK) * (CHUNK >> 4) + 512 * hf, id_qk, lead);
        kt_commit(bar(XB_SF + 2 * slot + hf), lead);
      };
      while (!dead && px_next(w, walk, s)) {
        const int n = s.n;
        const bool idle = nt == 2 && s.rb * 2 * PT_ROWS + slot * PT_ROWS >= (shared ? w.rows : w.R);
        const int i0 = nt == 2 ? 0 : (slot - gc) & 1;    // this slot's first chunk
        if (!kt_warp_wait(bar(XB_QF), qn & 1)) { dead = true; break; }
        tc_fence_after();
        if (idle) {                                      // no rows: only let the stages go
          for (int i = 0; i < n; ++i) {
            if (!wait_k(gc + i) || !wait_v(gc + i)) { dead = true; break; }
            kt_commit(bar(XB_KE + (gc + i) % SK), lead);
            kt_commit(bar(XB_VE + (gc + i) % SV), lead);
          }
        } else if (i0 < n) {
          if (!wait_k(gc + i0)) { dead = true; break; }
          scores(gc + i0, 0);
          scores(gc + i0, 1);
          kt_commit(bar(XB_KE + (gc + i0) % SK), lead);
          if (i0 + step >= n) kt_commit(bar(XB_QE), lead);
#pragma unroll 1
          for (int i = i0; i < n && !dead; i += step) {
            const int x = gc + i, xn = x + step;
            // one tile: slot 1's O may be overwritten only after the first warpgroup has merged it into the
            // previous block's partial
            if (nt == 1 && slot == 1 && i == i0 && qn > 0 && !kt_warp_wait(bar(XB_MFR), (qn - 1) & 1)) { dead = true; break; }
            if (!wait_v(x)) { dead = true; break; }
            // each half of P as it comes, and in its place the next chunk's scores
            int next = i + step < n ? 0 : 2;             // halves of the next chunk's scores issued
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
              if (!kt_warp_wait(bar(XB_PR + 2 * slot + hf), js & 1)) { dead = true; break; }
              tc_fence_after();
              kt_pv(od, sp + 64 * hf, dv + (x % SV) * (CHUNK >> 4) + 512 * hf, id_pv, i != i0 || hf, lead);
              kt_commit(bar(XB_OF + 2 * slot + hf), lead);
              if (hf == 1) kt_commit(bar(XB_VE + x % SV), lead);
              if (next == 0) {
                // the first half's scores wait for P's second half where their keys are not there yet
                const bool now = hf == 1 ? wait_k(xn) : __all_sync(0xffffffffu, mbar_test(bar(XB_KF + xn % SK), (xn / SK) & 1));
                if (hf == 1 && !now) { dead = true; break; }
                if (now) {
                  fence_proxy_async();
                  scores(xn, 0);
                  next = 1;
                }
              }
              if (hf == 1 && next == 1) {
                scores(xn, 1);
                kt_commit(bar(XB_KE + xn % SK), lead);
                if (i + 2 * step >= n) kt_commit(bar(XB_QE), lead);
              }
            }
            ++js;
          }
        }
        if (idle || i0 >= n) kt_commit(bar(XB_QE), lead);
        ++qn;
        gc += n;
        if (aborted()) break;
      }
      timed_out = dead;
      kt_commit(bar(XB_END), lead);                      // arrives once this warp's MMAs are done
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
    int js = 0, mc = 0, qn = 0, trees = 0, gc = 0;
    int js1 = 0;                                     // slot 1's jobs (merging warpgroup)
    while (px_next(w, walk, s)) {
      const int n = s.n, b = shared ? 0 : s.b, len = clamp_len(c, c.len[b]), pc = (len + PX_KEYS - 1) / PX_KEYS;
      const int tile = nt == 2 ? slot : 0;
      const int br = tile * PT_ROWS + r;             // row of the block
      const PxRow row = px_row(w, shared, s, br);
      const bool live = __any_sync(0xffffffffu, row.ok);
      // ---- the block's queries.  Two tiles: each slot its own; one: the second slot, which is done with the
      // block before sooner, while the first one writes that block's partial
      if (nt == 2 || slot == 1) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.q) + row.node_row * a.q_row + row.head * a.q_head);
        uint4 raw[DH / 8];
#pragma unroll
        for (int u = 0; u < DH / 8; ++u) raw[u] = row.ok ? src[u] : make_uint4(0u, 0u, 0u, 0u);
        if (qn > 0 && !kt_warp_wait(bar(XB_QE), (qn - 1) & 1)) { timed_out = true; break; }
        const uint32_t to = qs + tile * CHUNK + r * 128;
#pragma unroll
        for (int u = 0; u < DH / 8; ++u)
          st_shared16(to + (u >> 3) * TILE + (((u & 7) ^ (r & 7)) << 4), raw[u].x, raw[u].y, raw[u].z, raw[u].w);
        fence_proxy_async();
        mbar_arrive(bar(XB_QF));
      }
      const bool idle = nt == 2 && s.rb * 2 * PT_ROWS + slot * PT_ROWS >= (shared ? w.rows : w.R);
      const int i0 = nt == 2 ? 0 : (slot - gc) & 1;
      const int njobs = idle ? 0 : nt == 2 ? n : (n + 1 - i0) / 2;
      float m_use = -INFINITY, l_acc = 0.f;
      for (int jj = 0; jj < njobs; ++jj) {
        const int j = s.j + i0 + (nt == 2 ? jj : 2 * jj);
        const bool tree = j >= pc;
        const int t0 = (tree ? j - pc : j) * PX_KEYS;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          if (!kt_warp_wait(bar(XB_SF + 2 * slot + hf), js & 1)) { timed_out = true; break; }
          tc_fence_after();
          if (live) {
            float v[64];
            tmem_ld64(scol + 64 * hf, v);
            const int valid = len - t0 - 64 * hf;    // cached keys of this half there are
            if (tree) {
              const uint32_t see[2] = {row.ok ? px_sees(a, row.n, (t0 >> 5) + 2 * hf) : 0u,
                                       row.ok ? px_sees(a, row.n, (t0 >> 5) + 2 * hf + 1) : 0u};
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (!((see[e >> 5] >> (e & 31)) & 1u)) v[e] = -INFINITY;
            } else if (valid < 64) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (e >= valid) v[e] = -INFINITY;
            }
            float x0 = fmaxf(v[0], v[1]), x1 = fmaxf(v[2], v[3]);
#pragma unroll
            for (int e = 4; e < 64; e += 4) {
              x0 = max3(x0, v[e], v[e + 1]);
              x1 = max3(x1, v[e + 2], v[e + 3]);
            }
            const float mx = fmaxf(x0, x1) * sl2;
            const bool raise = mx > m_use + PT_LAZY;     // (from -infinity: any score)
            if (__any_sync(0xffffffffu, raise)) {
              const float f = !raise ? 1.f : m_use == -INFINITY ? 0.f : ex2_approx(m_use - mx);
              // O is rescaled once the half before has been added to it; a block's first half finds none
              if (jj > 0 || hf == 1) {
                if (!kt_warp_wait(bar(XB_OF + 2 * slot + (hf ^ 1)), (hf ? js : js - 1) & 1)) { timed_out = true; break; }
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < DH; e += 16) {
                  float u[16];
                  kt_ld16(ocol + e, u);
#pragma unroll
                  for (int q = 0; q < 16; ++q) u[q] *= f;
                  tmem_st16(ocol + e, u);
                }
              }
              l_acc *= f;
              if (raise) m_use = mx;
            }
            F2 ls = f2(0.f, 0.f);
            uint32_t pk[32];
            const float nm = m_use == -INFINITY ? 0.f : -m_use;     // (nothing seen yet: every score is -infinity)
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float p0, p1;
              unf2(fma2(f2(v[e], v[e + 1]), f2(sl2, sl2), f2(nm, nm)), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              ls = add2(ls, f2(p0, p1));
              pk[e / 2] = bf16x2(p0, p1);
            }
            kt_st32(scol + 64 * hf, pk);
            kt_st_wait();
            float l0, l1;
            unf2(ls, l0, l1);
            l_acc += l0 + l1;
          }
          tc_fence_before();
          mbar_arrive(bar(XB_PR + 2 * slot + hf));
        }
        if (timed_out) break;
        ++js;
      }
      if (timed_out) break;
      ++qn;
      // ---- the block's partial
      const long prow = s.slot * rbrows + br;
      float* dst = part_o + prow * DH;
      // a row that sees a value which is not finite has a NaN sum (the copies' notes are in shared memory once
      // the last P V is done)
      const int first_tree = max(s.j, pc), n_trees = max(s.j + n - first_tree, 0);
      auto noted = [&]() {
        bool bad = false;
        for (int q = 0; q < n_trees; ++q)
          for (int u = 0; u < 4; ++u)
            bad |= row.ok && (px_sees(a, row.n, (first_tree - pc + q) * 4 + u) & *(volatile uint32_t*)&s_bad[(trees + q) & 7][u]) != 0u;
        return bad;
      };
      if (nt == 2) {
        if (njobs > 0 && live) {
          if (!kt_warp_wait(bar(XB_OF + 2 * slot + 1), (js - 1) & 1)) { timed_out = true; break; }
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
        js1 += nj1;
        bool ok = njobs == 0 || kt_warp_wait(bar(XB_OF + 1), (js - 1) & 1);
        // the second slot's softmax first: it ends once all of its products but the last are done
        if (ok) ok = kt_warp_wait(bar(XB_MRG), mc & 1);
        if (ok && nj1 > 0) ok = kt_warp_wait(bar(XB_OF + 3), (js1 - 1) & 1);
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
    set_flag(a.status, MEDUSA_FLAG_TIMEOUT);
    *(volatile int*)&s_abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) mbar_wait(bar(XB_END), 0, TC_TIMEOUT_NS);      // every MMA done
  __syncthreads();
  if (warp == PT_MMA_WARP) tmem_dealloc(tmem, 2 * PT_SLOT_COLS);
}

// ------------------------------------------------------------------ host side
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
    const int stages = (int)((limit - 1024) / CHUNK) - g.nt[kind];
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

cudaError_t launch_prefix_tc(const PxWork& w, int num_sms, cudaStream_t st) {
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
