// Attention over a 4-bit KV cache for many query rows a key/value head (trees and chunks of
// bf16 rows, dh 64 or 128) on the tcgen05 tensor cores ("Medusa: Simple LLM Inference
// Acceleration Framework with Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5, over
// the format of include/medusa.h).
//
// The work is dealt out as in k_kv4_attn.cu: one CTA per SM takes an even share of the chunks of
// 128 cached slots, a (sequence, head, row block) at a time, and writes a partial for each it
// leaves.  A row block is one 128-row tile, or two when a head has more rows.  In the CTA
//
//   warps 8-15   decode: a thread takes 64 elements of one slot (32 bytes of codes, 4 scales),
//                loaded a chunk ahead into registers, and writes them as halves (exact) into a
//                128-byte-swizzled tile: K and V chunks in rings of two or three stages
//   warp 16      (one lane) MMAs for two "slots", each with S (128 columns) and O (dh columns) in
//                tensor memory: S = Q K^T, then O += P V with P read from tensor memory (the A
//                operand) and V from shared memory (MN-major)
//   warps 0-3,   two softmax warpgroups, one per slot, one query row per thread: they load the
//   4-7          block's queries (scaled by a power of two into a half's range), read S 64 columns
//                at a time, exponentiate and write P over S as pairs of halves
//
// With two tiles the slots are the tiles and share every chunk; with one both slots work on it
// and take alternate chunks, and the first warpgroup merges the second's (O, reference, sum)
// before it writes the partial.  The call's own tree rows are added by the joining kernel.
// Every wait is bounded; on expiry MEDUSA_FLAG_TIMEOUT is set, the CTA stops taking work, lets
// its MMAs end and frees its tensor memory.
#include <cuda.h>

#include "kv4_attn.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace medusa {

constexpr int KT_ROWS = 128, KT_KEYS = KD_CHUNK, KT_MAXST = 3;
constexpr int KT_MMA_WARP = 16, KT_THREADS = 5 * 128;   // five warpgroups; of the last one warp works
// Registers a thread: 96 at launch (5 x 128 x 96 = 61440), then 136 for softmax, 80 for decode and
// 48 for the MMA warpgroup: 2 x 136 + 2 x 80 + 48 = 5 x 96.
constexpr int KT_REG_SOFTMAX = 136, KT_REG_DECODE = 80, KT_REG_MMA = 48;
static_assert(2 * KT_REG_SOFTMAX + 2 * KT_REG_DECODE + KT_REG_MMA == 5 * 96, "what the launch holds");
constexpr uint32_t KT_SLOT_COLS = 256;               // per slot: S / P [0, 128), O [128, 128 + dh)
constexpr int KT_MIN_ROWS = 17;                      // rows a head from which this kernel is taken

bool kv4_tree_takes(int dtype, int dh, int R) { return dtype == MEDUSA_BF16 && dh >= 64 && R >= KT_MIN_ROWS; }
void kv4_tree_blocks(int R, int* rb, int* nrb) {
  const int most = R > KT_ROWS ? 2 * KT_ROWS : KT_ROWS;
  *rb = R < most ? R : most;
  *nrb = (R + most - 1) / most;
}

// Barriers.  QF / QE: query tiles written / no longer read.  KF / KE and VF / VE: K and V stages
// full / free.  Per slot: SF (S written), PR (P written), OF (P V done).  MRG / MFR: the second
// slot's (reference, sum) are in shared memory / consumed.  END: every MMA issued has completed.
enum {
  TB_QF = 0, TB_QE = 1, TB_KF = 2, TB_KE = TB_KF + KT_MAXST, TB_VF = TB_KE + KT_MAXST, TB_VE = TB_VF + KT_MAXST,
  TB_SF = TB_VE + KT_MAXST, TB_PR = TB_SF + 2, TB_OF = TB_PR + 2, TB_MRG = TB_OF + 2, TB_MFR = TB_MRG + 1,
  TB_END = TB_MFR + 1, TB_COUNT = TB_END + 1
};

struct Kv4TreeArgs {
  Kv4Work w;
  int nt, kst, vst;                   // query tiles of a block, stages of the K and V rings
};

// Instruction descriptor, kind::f16: fp32 D, half A and B, both K-major, M x N.
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }
// D[tmem] (+)= A(smem) B(smem)^T and A(tmem) B(smem), kind::f16.
__device__ __forceinline__ void kt_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  umma_bf16(d, a, b, idesc, acc);     // the descriptor says which 16-bit type the operands are
}
__device__ __forceinline__ void kt_mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 columns of 32 bits of this thread's TMEM lane, without and with the wait.
__device__ __forceinline__ void kt_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void kt_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ bool kt_warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, TC_TIMEOUT_NS));
}
template <int N> __device__ __forceinline__ void reg_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int DH>
__global__ void __launch_bounds__(KT_THREADS, 1) kv4_tree_kernel(const __grid_constant__ Kv4TreeArgs ta) {
  constexpr int H = DH / 64;                         // 64-element halves of a head
  constexpr int BLK = kv4_block(DH);
  constexpr uint32_t TILE = 128 * 128;               // one half of a tile: 128 rows of 128 bytes
  constexpr uint32_t CHUNK = H * TILE;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[TB_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  __shared__ float2 s_ml[KT_ROWS];                   // second slot's (reference, sum) per row
  const Kv4Work& w = ta.w;
  const CacheView& c = w.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nt = ta.nt, SK = ta.kst, SV = ta.vst;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t qs = base, k0s = base + nt * CHUNK, v0s = k0s + SK * CHUNK;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int per = c.Hkv * w.nrb;
  const long W = kd_total(c, per);
  const long ctas = W < (long)gridDim.x ? W : (long)gridDim.x;
  if (blockIdx.x >= ctas) {
    pdl_trigger();
    return;
  }
  const long w0 = W * blockIdx.x / ctas, w1 = W * (blockIdx.x + 1) / ctas;

  if (tid == 0) {
    mbar_init(bar(TB_QF), 2 * KT_ROWS);
    mbar_init(bar(TB_QE), 1);
    for (int i = 0; i < KT_MAXST; ++i) {
      mbar_init(bar(TB_KF + i), 128 * H);
      mbar_init(bar(TB_KE + i), 1);
      mbar_init(bar(TB_VF + i), 128 * H);
      mbar_init(bar(TB_VE + i), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(TB_SF + s), 1);
      mbar_init(bar(TB_PR + s), KT_ROWS);
      mbar_init(bar(TB_OF + s), 1);
    }
    mbar_init(bar(TB_MRG), KT_ROWS);
    mbar_init(bar(TB_MFR), KT_ROWS);
    mbar_init(bar(TB_END), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == KT_MMA_WARP) tmem_alloc(smem_u32(&tmem_slot), 2 * KT_SLOT_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();                          // only once this CTA holds its TMEM
  const uint32_t tmem = tmem_slot;
  bool timed_out = false;
  auto aborted = [&]() { return *(volatile int*)&s_abort != 0; };

  if (warp >= 8 && warp < KT_MMA_WARP) {
    // ------------------------------------------------------------ decode
    reg_fewer<KT_REG_DECODE>();
    // dh 128: 256 threads take the two halves of 128 slots, keys then values; dh 64: one half
    // of the threads takes the keys, the other the values
    const int slot = (warp & 3) * 32 + lane, half = (warp - 8) >> 2;
    const int eh = H == 2 ? half : 0;                 // 64-element half of the head
    const bool do_k = H == 2 || half == 0, do_v = H == 2 || half == 1;
    const int upp = (c.page_table ? c.page_size : c.capacity) / KV4_SLOTS;
    struct Piece {
      uint4 a, b;
      uint32_t sc;
    };
    Piece kp, vp;
    // two walks: one chunk ahead the codes are loaded, two chunks ahead the page is looked up
    KdCursor lk = kd_seek(c, per, w0);
    long lw = w0;
    int len_b = -1, len = 0;
    long blk = 0;                                     // this slot's block for lk (head 0)
    auto look = [&]() {                               // of chunk lw, if there is one
      if (lw >= w1) return;
      if (lk.b != len_b) {
        len_b = lk.b;
        len = clamp_len(c, c.len[lk.b]);
      }
      const int t = lk.j * KT_KEYS + slot;
      blk = -1;
      if (t < len) {
        long unit;
        int in;
        if (!unit_of(c, lk.b, t, unit, in)) {
          set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
          unit = 0;
        }
        blk = (unit * c.Hkv + lk.q / w.nrb) * upp + in / KV4_SLOTS;
      }
    };
    auto step = [&]() {
      if (++lw < w1) kd_next(c, per, lk);
    };
    const int in16 = slot % KV4_SLOTS;                // chunks start on a block's first slot
    auto load = [&](Piece& p, const void* pool, long b) {
      if (b < 0) {                                    // past the length: zeros, whatever lies there
        p.a = p.b = make_uint4(0u, 0u, 0u, 0u);
        p.sc = 0u;
        return;
      }
      const uint8_t* s = static_cast<const uint8_t*>(pool) + b * BLK;
      const uint4* q = reinterpret_cast<const uint4*>(s + in16 * (DH / 2) + eh * 32);
      p.a = __ldg(q);
      p.b = __ldg(q + 1);
      p.sc = __ldg(reinterpret_cast<const uint32_t*>(s + 8 * DH + in16 * (DH / 16) + eh * 4));
    };
    auto store = [&](const Piece& p, uint32_t tile) {
      const uint32_t wd[8] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w};
      const __half2 s01 = kv4_scales((uint16_t)(p.sc & 0xffffu)), s23 = kv4_scales((uint16_t)(p.sc >> 16));
      const uint32_t row = tile + eh * TILE + slot * 128;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2 s = i < 2 ? __low2half2(s01) : i < 4 ? __high2half2(s01) : i < 6 ? __low2half2(s23) : __high2half2(s23);
        __half2 y[4];
        kv4_pairs(wd[i], y);
        st_shared16(row + ((i ^ (slot & 7)) << 4), h2u(__hmul2(y[0], s)), h2u(__hmul2(y[1], s)), h2u(__hmul2(y[2], s)),
                    h2u(__hmul2(y[3], s)));
      }
      fence_proxy_async();
    };
    look();
    long cur = blk;
    step();
    look();                                           // blk: chunk w0 + 1
    if (do_k) load(kp, c.k, cur);
    if (do_v) load(vp, c.v, cur);
    for (long x = w0; x < w1; ++x) {
      const int i = (int)(x - w0);
      const long next = blk;
      const bool more = x + 1 < w1;
      step();
      look();                                         // chunk x + 2
      if (do_k) {
        if (!kt_warp_wait(bar(TB_KE + i % SK), ((i / SK) & 1) ^ 1)) { timed_out = true; break; }
        store(kp, k0s + (i % SK) * CHUNK);
        mbar_arrive(bar(TB_KF + i % SK));
        if (more) load(kp, c.k, next);
      }
      if (do_v) {
        if (!kt_warp_wait(bar(TB_VE + i % SV), ((i / SV) & 1) ^ 1)) { timed_out = true; break; }
        store(vp, v0s + (i % SV) * CHUNK);
        mbar_arrive(bar(TB_VF + i % SV));
        if (more) load(vp, c.v, next);
      }
      if (aborted()) break;
    }
  } else if (warp >= KT_MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    reg_fewer<KT_REG_MMA>();
    KdCursor k = kd_seek(c, per, w0);
    if (warp == KT_MMA_WARP && lane == 0) {
      const uint32_t id_qk = idesc_f16(KT_ROWS, KT_KEYS);
      const uint32_t id_pv = idesc_f16(KT_ROWS, DH) | IDESC_B_MN_MAJOR;
      int gc = 0, qn = 0, mc = 0;
      int js0 = 0, js1 = 0;               // jobs (chunk x slot) issued per slot
      auto wait_k = [&](int x) -> bool {
        if (!mbar_wait(bar(TB_KF + x % SK), (x / SK) & 1, TC_TIMEOUT_NS)) return false;
        tc_fence_after();
        return true;
      };
      auto wait_v = [&](int x) -> bool {
        if (!mbar_wait(bar(TB_VF + x % SV), (x / SV) & 1, TC_TIMEOUT_NS)) return false;
        tc_fence_after();
        return true;
      };
      auto issue_qk = [&](int slot, int tile, int x) {
        const uint32_t ks = k0s + (x % SK) * CHUNK, d = tmem + slot * KT_SLOT_COLS;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            kt_mma(d, sw128_desc(qs + tile * CHUNK + h * TILE) + 2 * kk, sw128_desc(ks + h * TILE) + 2 * kk, id_qk,
                   (h | kk) != 0);
        umma_commit(bar(TB_SF + slot));
      };
      auto wait_p = [&](int slot) -> bool {
        if (!mbar_wait(bar(TB_PR + slot), (slot ? js1 : js0) & 1, TC_TIMEOUT_NS)) return false;
        tc_fence_after();
        return true;
      };
      auto issue_pv = [&](int slot, int x, bool acc) {
        const uint32_t vs = v0s + (x % SV) * CHUNK, pa = tmem + slot * KT_SLOT_COLS, d = pa + KT_KEYS;
#pragma unroll
        for (int kk = 0; kk < KT_KEYS / 16; ++kk)      // 16 keys per MMA: 8 columns of P
          kt_mma_tmem_a(d, pa + 8 * kk, sw128_desc_mn(vs + kk * 2048, TILE), id_pv, acc || kk > 0);
        umma_commit(bar(TB_OF + slot));
        if (slot) ++js1;
        else ++js0;
      };
      bool dead = false;
      for (long wi = w0; wi < w1 && !dead;) {
        const int n = (int)min((long)(k.nb - k.j), w1 - wi);
        const int row0 = (k.q % w.nrb) * KT_ROWS * nt;
        const int nta = nt == 2 ? (row0 + KT_ROWS < w.R ? 2 : 1) : 1;
        if (!mbar_wait(bar(TB_QF), qn & 1, TC_TIMEOUT_NS)) { dead = true; break; }
        ++qn;
        tc_fence_after();
        if (nt == 2) {
          // every chunk goes to each active tile's slot
          if (!wait_k(gc)) { dead = true; break; }
          for (int s = 0; s < nta; ++s) issue_qk(s, s, gc);
          umma_commit(bar(TB_KE + gc % SK));
          if (n == 1) umma_commit(bar(TB_QE));
          for (int i = 0; i < n && !dead; ++i) {
            const int x = gc + i;
            if (!wait_v(x)) { dead = true; break; }
            for (int s = 0; s < nta; ++s) {
              if (!wait_p(s)) { dead = true; break; }
              issue_pv(s, x, i > 0);
              if (i + 1 < n) {
                if (s == 0 && !wait_k(x + 1)) { dead = true; break; }
                issue_qk(s, s, x + 1);
                if (s == nta - 1) {
                  umma_commit(bar(TB_KE + (x + 1) % SK));   // both tiles' S of chunk x + 1
                  if (i + 2 == n) umma_commit(bar(TB_QE));
                }
              }
            }
            if (!dead) umma_commit(bar(TB_VE + x % SV));     // both tiles' P V of chunk x
          }
        } else {
          // one tile: chunk i goes to slot i & 1; slot 1's O may be overwritten only after the
          // first warpgroup has merged it into the previous block's partial
          if (!wait_k(gc)) { dead = true; break; }
          issue_qk(0, 0, gc);
          umma_commit(bar(TB_KE + gc % SK));
          if (n > 1) {
            if (!wait_k(gc + 1)) { dead = true; break; }
            issue_qk(1, 0, gc + 1);
            umma_commit(bar(TB_KE + (gc + 1) % SK));
          }
          if (n <= 2) umma_commit(bar(TB_QE));
          for (int i = 0; i < n; ++i) {
            const int s = i & 1, x = gc + i;
            if (!wait_v(x) || !wait_p(s)) { dead = true; break; }
            if (i == 1 && mc > 0 && !mbar_wait(bar(TB_MFR), (mc - 1) & 1, TC_TIMEOUT_NS)) { dead = true; break; }
            issue_pv(s, x, i > 1);
            umma_commit(bar(TB_VE + x % SV));
            if (i + 2 < n) {
              if (!wait_k(x + 2)) { dead = true; break; }
              issue_qk(s, 0, x + 2);
              umma_commit(bar(TB_KE + (x + 2) % SK));
              if (i + 3 == n) umma_commit(bar(TB_QE));
            }
          }
          ++mc;
        }
        gc += n;
        wi += n;
        k.j += n - 1;
        if (wi < w1) kd_next(c, per, k);
        if (aborted()) break;
      }
      timed_out = dead;
      umma_commit(bar(TB_END));           // arrives once every MMA issued above is done
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    reg_more<KT_REG_SOFTMAX>();
    const int slot = warp >> 2, wl = warp & 3;
    const int r = wl * 32 + lane;                    // row within the tile = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(wl * 32) << 16);
    const uint32_t scol = lane_base + slot * KT_SLOT_COLS;      // this slot's S / P
    const uint32_t ocol = scol + KT_KEYS;                       // this slot's O
    KdCursor k = kd_seek(c, per, w0);
    int js = 0, mc = 0, qn = 0;
    int js1 = 0;                                     // slot 1's jobs (merging warpgroup)
    for (long wi = w0; wi < w1;) {
      const int n = (int)min((long)(k.nb - k.j), w1 - wi);
      const int g = k.q / w.nrb, rblk = k.q - g * w.nrb, len = clamp_len(c, c.len[k.b]);
      const int row0 = rblk * KT_ROWS * nt, tile = nt == 2 ? slot : 0;
      const int gr = row0 + tile * KT_ROWS + r;
      const bool row_ok = gr < w.R;
      const bool live = row0 + tile * KT_ROWS + wl * 32 < w.R;     // the warp has rows
      // ---- the block's queries: scaled into [1, 2) by a power of two, as halves.  One tile:
      // the warpgroups write a 64-element half each (dh 64: the first all of it)
      float rs;
      {
        const int node = row_ok ? gr / w.a.G : 0, hq = g * w.a.G + (row_ok ? gr - node * w.a.G : 0);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const bf16*>(w.a.q) +
                                                          ((long)k.b * w.a.n1 + node) * w.a.q_row + hq * w.a.q_head);
        float top = 0.f;
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < DH / 8; ++i) {
            float f[8];
            unpack16(src[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
          }
        }
        float down, up;
        row_scale(top, down, up);
        rs = up * (w.a.scale * c.gk) * 1.4426950408889634f;
        if (qn > 0 && !kt_warp_wait(bar(TB_QE), (qn - 1) & 1)) { timed_out = true; break; }
        ++qn;
        if (nt == 2 || H == 2 || slot == 0) {
          const int h0 = nt == 2 ? 0 : slot, h1 = nt == 2 || H == 1 ? H : slot + 1;
          for (int h = h0; h < h1; ++h) {
            const uint32_t row = qs + tile * CHUNK + h * TILE + r * 128;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              float f[8];
              unpack16(row_ok ? src[h * 8 + u] : make_uint4(0u, 0u, 0u, 0u), f);
              st_shared16(row + ((u ^ (r & 7)) << 4), half_pair(f[0] * down, f[1] * down), half_pair(f[2] * down, f[3] * down),
                          half_pair(f[4] * down, f[5] * down), half_pair(f[6] * down, f[7] * down));
            }
          }
        }
        fence_proxy_async();
        mbar_arrive(bar(TB_QF));
      }
      const bool idle = nt == 2 && row0 + tile * KT_ROWS >= w.R;   // this tile has no rows
      const int njobs = idle ? 0 : nt == 2 ? n : (n + 1 - slot) / 2;
      float m_use = -INFINITY, l_acc = 0.f;
      for (int jj = 0; jj < njobs; ++jj) {
        const int i = nt == 2 ? jj : 2 * jj + slot;
        if (!kt_warp_wait(bar(TB_SF + slot), js & 1)) { timed_out = true; break; }
        tc_fence_after();
        if (live) {
          const int t0 = (k.j + i) * KT_KEYS;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float s[64];
            tmem_ld64(scol + 64 * hf, s);
            const int valid = len - t0 - 64 * hf;    // keys of this half there are
            if (valid < 64) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (j >= valid) s[j] = -INFINITY;
            }
            float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]);
#pragma unroll
            for (int j = 4; j < 64; j += 4) {
              x0 = fmaxf(x0, fmaxf(s[j], s[j + 1]));
              x1 = fmaxf(x1, fmaxf(s[j + 2], s[j + 3]));
            }
            const float mx = fmaxf(x0, x1) * rs;     // the row's factor is positive
            const bool raise = mx > m_use + KD_TOP;
            if (__any_sync(0xffffffffu, raise)) {
              const float mn = raise ? mx - KD_BACK<false> : m_use;
              const float f = !raise ? 1.f : m_use == -INFINITY ? 0.f : ex2_approx(m_use - mn);
              // The P V of this slot's previous chunk has completed (this S comes from a later
              // MMA of the same issuer), so O may be rescaled here; in a block's first chunk
              // there is no O yet.
              if (jj > 0) {
#pragma unroll
                for (int x = 0; x < DH; x += 16) {
                  float v[16];
                  tmem_ld16(ocol + x, v);
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[e] *= f;
                  tmem_st16(ocol + x, v);
                }
              }
              if (hf == 1) {                         // and the first half's P, already written
                const __half2 fh = __float2half2_rn(f);
#pragma unroll
                for (int x = 0; x < 32; x += 16) {
                  float v[16];
                  tmem_ld16(scol + x, v);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    uint32_t u = __float_as_uint(v[e]);
                    u = h2u(__hmul2(*reinterpret_cast<__half2*>(&u), fh));
                    v[e] = __uint_as_float(u);
                  }
                  tmem_st16(scol + x, v);
                }
              }
              l_acc *= f;
              m_use = mn;
            }
            float l0 = 0.f, l1 = 0.f;
            uint32_t pk[32];
            const float nm = -m_use;
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const float p0 = ex2_approx(fmaf(s[j], rs, nm)), p1 = ex2_approx(fmaf(s[j + 1], rs, nm));
              l0 += p0;
              l1 += p1;
              pk[j / 2] = half_pair(p0, p1);
            }
            kt_st32(scol + 32 * hf, pk);
            kt_st_wait();
            l_acc += l0 + l1;
          }
        }
        tc_fence_before();
        mbar_arrive(bar(TB_PR + slot));
        ++js;
      }
      if (timed_out) break;
      // ---- the block's partial
      const long pair = (long)k.b * per + k.q, part = pair + blockIdx.x;
      const long prow = part * w.rb + tile * KT_ROWS + r;
      float* dst = w.part_o + prow * DH;
      if (tid == 0) {
        if (k.j == 0) w.span[pair].x = (int)part;
        if (k.j + n == k.nb) w.span[pair].y = (int)part + 1;
      }
      if (nt == 2) {
        if (njobs > 0 && live) {
          if (!kt_warp_wait(bar(TB_OF + slot), (js - 1) & 1)) { timed_out = true; break; }
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < DH; x += 16) {
            float v[16];
            tmem_ld16(ocol + x, v);
            if (row_ok) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(dst + x + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
          }
          if (row_ok) w.part_ml[prow] = make_float2(m_use, l_acc);
        }
        tc_fence_before();
      } else if (slot == 1) {
        // hand (reference, sum) to the first warpgroup once it has consumed the previous ones
        if (mc > 0 && !kt_warp_wait(bar(TB_MFR), (mc - 1) & 1)) { timed_out = true; break; }
        s_ml[r] = make_float2(m_use, l_acc);
        mbar_arrive(bar(TB_MRG));
        ++mc;
      } else {
        const int nj1 = n / 2;                       // slot 1's chunks in this block
        js1 += nj1;
        bool ok = kt_warp_wait(bar(TB_OF), (js - 1) & 1);
        if (ok && nj1 > 0) ok = kt_warp_wait(bar(TB_OF + 1), (js1 - 1) & 1);
        if (ok) ok = kt_warp_wait(bar(TB_MRG), mc & 1);
        if (!ok) { timed_out = true; break; }
        tc_fence_after();
        const float2 ml1 = s_ml[r];
        const float m = fmaxf(m_use, ml1.x);
        const float f0 = m_use == -INFINITY ? 0.f : ex2_approx(m_use - m);
        const float f1 = ml1.x == -INFINITY ? 0.f : ex2_approx(ml1.x - m);
        const uint32_t ocol1 = lane_base + KT_SLOT_COLS + KT_KEYS;
        if (live) {
#pragma unroll
          for (int x = 0; x < DH; x += 16) {
            float v0[16], v1[16];
            tmem_ld16(ocol + x, v0);
            if (nj1 > 0) {
              tmem_ld16(ocol1 + x, v1);            // written by this block's P V of slot 1
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) v1[e] = 0.f;
            }
            if (row_ok) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(dst + x + e) =
                    make_float4(v0[e] * f0 + v1[e] * f1, v0[e + 1] * f0 + v1[e + 1] * f1,
                                v0[e + 2] * f0 + v1[e + 2] * f1, v0[e + 3] * f0 + v1[e + 3] * f1);
            }
          }
          if (row_ok) w.part_ml[prow] = make_float2(m, l_acc * f0 + ml1.y * f1);
        }
        tc_fence_before();
        mbar_arrive(bar(TB_MFR));
        ++mc;
      }
      wi += n;
      k.j += n - 1;
      if (wi < w1) kd_next(c, per, k);
    }
  }
  if (timed_out) {
    set_flag(c.status, MEDUSA_FLAG_TIMEOUT);
    *(volatile int*)&s_abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) mbar_wait(bar(TB_END), 0, TC_TIMEOUT_NS);      // every MMA done
  __syncthreads();
  if (warp == KT_MMA_WARP) tmem_dealloc(tmem, 2 * KT_SLOT_COLS);
}

cudaError_t launch_kv4_tree(const Kv4Work& w, int num_sms, cudaStream_t st) {
  Kv4TreeArgs a;
  a.w = w;
  a.nt = w.R > KT_ROWS ? 2 : 1;
  a.kst = a.nt == 2 ? 2 : 3;
  a.vst = 2;
  const size_t chunk = (size_t)w.a.c.dh / 64 * 128 * 128, most = 1024 + 6 * chunk;   // both forms hold six tiles
  static unsigned long long done128 = 0, done64 = 0;
  auto kern = w.a.c.dh == 128 ? kv4_tree_kernel<128> : kv4_tree_kernel<64>;
  const cudaError_t e = allow_smem(kern, most, w.a.c.dh == 128 ? &done128 : &done64);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(num_sms), dim3(KT_THREADS), most, st, 1, a);
}

}  // namespace medusa
