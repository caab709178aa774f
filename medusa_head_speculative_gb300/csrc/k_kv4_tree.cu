// Attention over a 4-bit KV cache for many query rows a key/value head (trees and chunks of
// bf16 rows, dh 64 or 128) on the tcgen05 tensor cores ("Medusa: Simple LLM Inference
// Acceleration Framework with Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5, over
// the format of include/medusa.h).
//
// For each row r of a head, with s_j = scale q_r . k_j over the cached slots j:
// o_r = sum_j 2^(s'_j - m_r) v_j and l_r = sum_j 2^(s'_j - m_r), s' in base-2 units, m_r a running
// reference at or below the maximum (kv4_attn.cuh), o and l in float; the joining kernel of
// k_kv4_attn.cu adds the partials and the call's own rows up and divides.
//
// The work is dealt out as in k_kv4_attn.cu: one CTA per SM takes an even share of the chunks of
// 128 cached slots, a (sequence, head, row block) at a time, and writes a partial for each it
// leaves.  A row block is one 128-row tile, or two when a head has more rows.  In the CTA
//
//   warp 19      writes down where each triple's partials lie, before and without any wait: the joining
//                kernel reads by it, also after a wait of this one expired
//   warp 18      copies: the blocks of a chunk's keys, then of its values, by the copy engine into
//                rings of staging slots, one copy for each page (eight 1152-byte copies cost its
//                issue half as much again as one; copies issued by the decode warps, a ring each,
//                were slower: 112 us for 98)
//   warps 8-11,  decode keys and values: a thread takes 32 elements of one slot at a time (16 bytes
//   12-15        of codes, 2 scales) and writes them as halves (exact) into a 128-byte-swizzled tile;
//                K and V have two tiles each.  Warps of their own, because in one order a value
//                tile still in use held up the next keys (long 65-node trees 134 -> 121 us)
//   warps 16, 17 MMAs, a warp for each of two "slots" with S (128 columns) and O (dh columns) in
//                tensor memory: S = Q K^T, then O += P V with P read from tensor memory (the A
//                operand) and V from shared memory (MN-major), in halves of 64 slots: while the
//                softmax has one half, the other half's P is multiplied with V and the next
//                chunk's scores take its place (43 x 4 rows: 154 us with whole chunks, 146 so)
//   warps 0-3,   two softmax warpgroups, one per slot, one query row per thread: they load the
//   4-7          block's queries (scaled by a power of two into a half's range), read a half of S,
//                exponentiate and write P over it as pairs of halves
//
// With two tiles the slots are the tiles and share every chunk; with one both slots work on it
// and take alternate chunks, and the first warpgroup merges the second's (O, reference, sum)
// before it writes the partial.
//
// Measured: 8 sequences x 40 heads x 65 nodes over 2048-4096 slots each (161 MB, 24 us at copy
// bandwidth) 96 us; 16 x 8 heads x 172 rows over 8192 slots (165 MB; 92 GFLOP, 73 us of tensor time
// on whole tiles) 139.5 us; 17 us of either for joining.  No single part bounds it: a chunk takes
// 2000 cycles (two tiles: 3900), with copies and signals alone 1250 (2500), and besides these
// with only the softmax 1500 (2700), the decoding 1650 (2700) or the MMAs 1650 (3300): the parts
// wait for one another.
//
// Every wait is bounded; on expiry MEDUSA_FLAG_TIMEOUT is set, the CTA stops taking work, lets
// its MMAs end and frees its tensor memory.
#include <cuda.h>

#include "kv4_attn.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace medusa {

constexpr int KT_ROWS = 128, KT_KEYS = KD_CHUNK, KT_ST = 2, KT_MAXLD = 6;
constexpr int KT_DECODERS = 4, KT_MMA_WARP = 16, KT_LOAD_WARP = 18;
constexpr int KT_THREADS = 5 * 128;                 // five warpgroups; of the last one three warps work
// Registers a thread: 96 at launch (5 x 128 x 96 = 61440), then 152 for softmax, 56 for decode and
// 64 for the MMA and copy warps: 2 x 152 + 2 x 56 + 64 = 5 x 96.
constexpr int KT_REG_SOFTMAX = 152, KT_REG_DECODE = 56, KT_REG_MMA = 64;
static_assert(2 * KT_REG_SOFTMAX + 2 * KT_REG_DECODE + KT_REG_MMA == 5 * 96, "what the launch holds");
constexpr uint32_t KT_SLOT_COLS = 256;               // per slot: S / P [0, 128), O [128, 128 + dh)
// Rows a head from which this kernel is taken; k_kv4_attn.cu, in blocks of 16 rows, against this
// one (us): 8 x 40 heads of 128, 3100 slots: 17 rows 85 / 78, 32 rows 87 / 82, 64 rows 162 / 88 (16 rows
// there: 50); 16 x 8 heads of 128, 6000 slots: 24 rows 65 / 57, 64 rows 121 / 61; 4 x 8 heads of 64, 2000
// slots: 17 rows 14.5 / 14.1, 64 rows 17.2 / 14.9.
constexpr int KT_MIN_ROWS = 17;

bool kv4_tree_takes(int dtype, int dh, int R) { return dtype == MEDUSA_BF16 && dh >= 64 && R >= KT_MIN_ROWS; }
void kv4_tree_blocks(int R, int* rb, int* nrb) {
  const int most = R > KT_ROWS ? 2 * KT_ROWS : KT_ROWS;
  *rb = R < most ? R : most;
  *nrb = (R + most - 1) / most;
}

// A wait names a phase by its parity, which tells it from its neighbours only: a waiter has to have
// seen the phase before, or something that implies it.  So keys and values are staged in rings of
// their own (in one ring of three a slot's next user skipped a phase), and where the slots of one
// tile share a barrier the order of the waits matters (see the comments there).
// Barriers.  LF / LE: a staging slot has landed / been read.  QF / QE: query tiles written / no
// longer read.  KF / KE and VF / VE: K and V stages
// full / free.  Per slot: SF (S written), PR (P written), OF (P V done).  MRG / MFR: the second
// slot's (reference, sum) are in shared memory / consumed.  END: every MMA issued has completed.
// NEVER: for failure-path tests, nothing arrives there.
enum {
  TB_QF = 0, TB_QE = 1, TB_KF = 2, TB_KE = TB_KF + KT_ST, TB_VF = TB_KE + KT_ST, TB_VE = TB_VF + KT_ST,
  TB_SF = TB_VE + KT_ST, TB_PR = TB_SF + 4, TB_OF = TB_PR + 4, TB_MRG = TB_OF + 4, TB_MFR = TB_MRG + 1,
  TB_END = TB_MFR + 1, TB_NEVER = TB_END + 1, TB_LF = TB_NEVER + 1, TB_LE = TB_LF + KT_MAXLD, TB_COUNT = TB_LE + KT_MAXLD
};

// Instruction descriptor, kind::f16: fp32 D, half A and B, both K-major, M x N.
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }
// The MMAs of one S = Q K^T (4 a 64-element half) and of one O += P V (8 x 16 keys), kind::f16
// (the descriptor says which 16-bit type the operands are), and their commits.  The whole warp
// comes here and lane 0 issues, by predicate and not in a branch, so that the operands stay in
// uniform registers.
#define KT_QK(OFF, ACC)                                  \
  "add.s64 x, %1, " OFF ";\n\tadd.s64 y, %2, " OFF ";\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, " ACC ";\n\t"
template <int H>
__device__ __forceinline__ void kt_qk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t lead) {
  if constexpr (H == 2)
    asm volatile("{\n\t.reg .pred e, no, yes;\n\t.reg .b64 x, y;\n\t"
                 "setp.ne.b32 e, %4, 0;\n\tsetp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
                 KT_QK("0", "no") KT_QK("2", "yes") KT_QK("4", "yes") KT_QK("6", "yes")
                 KT_QK("1024", "yes") KT_QK("1026", "yes") KT_QK("1028", "yes") KT_QK("1030", "yes") "}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(lead) : "memory");
  else
    asm volatile("{\n\t.reg .pred e, no, yes;\n\t.reg .b64 x, y;\n\t"
                 "setp.ne.b32 e, %4, 0;\n\tsetp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
                 KT_QK("0", "no") KT_QK("2", "yes") KT_QK("4", "yes") KT_QK("6", "yes") "}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(lead) : "memory");
}
#define KT_PV(AOFF, BOFF, ACC)                             \
  "add.u32 x, %1, " AOFF ";\n\tadd.s64 y, %2, " BOFF ";\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, " ACC ";\n\t"
__device__ __forceinline__ void kt_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile("{\n\t.reg .pred e, first, yes;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
               "setp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 first, %4, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
               KT_PV("0", "0", "first") KT_PV("8", "128", "yes") KT_PV("16", "256", "yes") KT_PV("24", "384", "yes") "}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void kt_commit(uint32_t bar, uint32_t lead) {
  asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
               ::"r"(bar), "r"(lead) : "memory");
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
// 16 columns of this thread's TMEM lane.  Load and wait are one statement: nothing else keeps the compiler from
// using a register between them.
__device__ __forceinline__ void kt_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void kt_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool kt_warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, TC_TIMEOUT_NS));
}
template <int N> __device__ __forceinline__ void reg_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int DH, int NT>
__global__ void __launch_bounds__(KT_THREADS, 1) kv4_tree_kernel(const __grid_constant__ Kv4Work w) {
  constexpr int H = DH / 64;                         // 64-element halves of a head
  constexpr int BLK = kv4_block(DH);
  constexpr uint32_t TILE = 128 * 128;               // one half of a tile: 128 rows of 128 bytes
  constexpr uint32_t CHUNK = H * TILE;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[TB_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  __shared__ int s_valid[KT_MAXLD];                  // slots of the chunk there are
  __shared__ float2 s_ml[KT_ROWS];                   // second slot's (reference, sum) per row
  __shared__ float s_rs[2][KT_ROWS];                 // one tile: the rows' score factors, two blocks
  const CacheView& c = w.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int nt = NT, SK = KT_ST, SV = KT_ST, SLK = NT == 2 ? 2 : 3, SLV = NT == 2 ? 1 : 3;   // tiles, stages of the rings: K, V, staged K and V
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t qs = base, k0s = base + nt * CHUNK, v0s = k0s + SK * CHUNK, l0s = v0s + SV * CHUNK;
  constexpr uint32_t STAGE = 8 * BLK;                // the blocks of 128 slots
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int per = c.Hkv * w.nrb;
  const long W = kd_total(c, per);
  const long ctas = W < (long)gridDim.x ? W : (long)gridDim.x;
  if (blockIdx.x >= ctas) {
    pdl_trigger();
    return;
  }
  const long w0 = W * blockIdx.x / ctas;
  const int total = (int)(W * (blockIdx.x + 1) / ctas - w0);   // this CTA's chunks

  if (tid == 0) {
    mbar_init(bar(TB_QF), nt * KT_ROWS);
    mbar_init(bar(TB_QE), 2);
    for (int i = 0; i < KT_ST; ++i) {
      mbar_init(bar(TB_KF + i), KT_DECODERS);
      mbar_init(bar(TB_KE + i), nt);
      mbar_init(bar(TB_VF + i), KT_DECODERS);
      mbar_init(bar(TB_VE + i), nt);
    }
    for (int i = 0; i < KT_MAXLD; ++i) {
      mbar_init(bar(TB_LF + i), 1);
      mbar_init(bar(TB_LE + i), KT_DECODERS);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(TB_SF + s), 1);
      mbar_init(bar(TB_PR + s), KT_ROWS);
      mbar_init(bar(TB_OF + s), 1);
    }
    mbar_init(bar(TB_MRG), KT_ROWS);
    mbar_init(bar(TB_MFR), KT_ROWS);
    mbar_init(bar(TB_END), 2);
    mbar_init(bar(TB_NEVER), 1);
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
    // 16 bytes of codes a lane: neighbouring lanes the quarters (dh 64: halves) of a slot, so that
    // reading a staging slot takes every bank once; and so does writing the tile, with the upper
    // half of a head (16 KB further on: the same banks) written two 16-byte units out of step.
    // A warp has one block (16 slots) of each chunk; all its addresses are fixed but for the stage.
    constexpr int Q = DH / 32, PIECES = Q / 2;        // lanes a slot, pieces (8 slots on) a lane
    const int quarter = lane % Q, eh = quarter >> 1, part = (warp - 8) >> 2, dw = 2 * ((warp - 8) & 3), key0 = dw * KV4_SLOTS + lane / Q;
    const uint32_t codes_at = l0s + dw * BLK + lane / Q * (DH / 2) + quarter * 16;
    const uint32_t scales_at = l0s + dw * BLK + 8 * DH + lane / Q * (DH / 16) + quarter * 2;
    uint32_t out_at[4];                               // of words 0..3 in the order they are written
#pragma unroll
    for (int z = 0; z < 4; ++z)
      out_at[z] = eh * TILE + key0 * 128 + ((((quarter & 1) * 4 + (z ^ (eh << 1))) ^ (key0 & 7)) << 4);
    const uint32_t first = eh ? 8 : 0, swap = eh ? 0x4401u : 0x4410u;   // an upper half's lane: words 2, 3 first
    const int slots = part ? SLV : SLK, slot0 = part ? SLK : 0;
    bool dead = false;
    for (int i = 0; i < total && !dead; ++i) {
        const int st = slot0 + i % slots;
        if (!kt_warp_wait(bar(TB_LF + st), (i / slots) & 1)) { dead = true; break; }
        const int valid = s_valid[st];
        constexpr int PP = 2 * PIECES;
        uint32_t cw[PP][4], sc[PP];
#pragma unroll
        for (int y = 0; y < PP; ++y) {
          const int bo = y / PIECES * BLK + y % PIECES * 8 * (DH / 2), so = y / PIECES * BLK + y % PIECES * 8 * (DH / 16);
          const uint32_t at = codes_at + st * STAGE + bo;
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(cw[y][0]), "=r"(cw[y][1]) : "r"(at + first));
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(cw[y][2]), "=r"(cw[y][3]) : "r"(at + (first ^ 8)));
          uint16_t two;
          asm volatile("ld.shared.b16 %0, [%1];" : "=h"(two) : "r"(scales_at + st * STAGE + so));
          sc[y] = __byte_perm(two, 0, swap);
        }
        if (valid < KT_KEYS) {                        // past the length: zeros, whatever lies there
#pragma unroll
          for (int y = 0; y < PP; ++y)
            if (key0 + (DH == 128 ? 8 * y : 16 * y) >= valid) cw[y][0] = cw[y][1] = cw[y][2] = cw[y][3] = sc[y] = 0u;
        }
        // the reads above come before the copy engine's next write there: an arrival alone does not order
        // the two proxies, and now and then a late read found the next chunk's codes
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(TB_LE + st));
        const int NS = part ? SV : SK, stage = i % NS, turn = i / NS;
        if (!kt_warp_wait(bar((part ? TB_VE : TB_KE) + stage), (turn & 1) ^ 1)) { dead = true; break; }
        const uint32_t tile = (part ? v0s : k0s) + stage * CHUNK;
#pragma unroll
        for (int y = 0; y < PP; ++y) {
          const __half2 s2 = kv4_scales((uint16_t)sc[y]);
          const __half2 s0 = __low2half2(s2), s1 = __high2half2(s2);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const __half2 s = z < 2 ? s0 : s1;
            __half2 h[4];
            kv4_pairs(cw[y][z], h);
            st_shared16(tile + out_at[z] + (DH == 128 ? y * 1024 : y * 2048), h2u(__hmul2(h[0], s)), h2u(__hmul2(h[1], s)), h2u(__hmul2(h[2], s)),
                        h2u(__hmul2(h[3], s)));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((part ? TB_VF : TB_KF) + stage));
      if (aborted()) break;
    }
    timed_out = dead;
  } else if (warp >= KT_MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    reg_fewer<KT_REG_MMA>();
    KdCursor k = kd_seek(c, per, w0);
    if (warp < KT_LOAD_WARP) {
      // ---------------------------------------------------------- MMAs of one slot
      const int slot = warp - KT_MMA_WARP;
      const uint32_t lead = lane == 0;
      const uint32_t id_qk = idesc_f16(KT_ROWS, KT_KEYS / 2);
      const uint32_t id_pv = idesc_f16(KT_ROWS, DH) | IDESC_B_MN_MAJOR;
      // descriptors hold addresses in 16-byte units: an offset is added to them
      const uint64_t dq = sw128_desc(qs + (nt == 2 ? slot : 0) * CHUNK), dk = sw128_desc(k0s), dv = sw128_desc_mn(v0s, TILE);
      const uint32_t sp = tmem + slot * KT_SLOT_COLS, od = sp + KT_KEYS;
      int gc = 0, qn = 0, js = 0;         // chunks, blocks and this slot's jobs so far
      bool dead = false;
      auto wait_k = [&](int x) { return kt_warp_wait(bar(TB_KF + x % SK), (x / SK) & 1); };
      auto wait_v = [&](int x) { return kt_warp_wait(bar(TB_VF + x % SV), (x / SV) & 1); };
      auto scores = [&](int x, int hf) {
        kt_qk<H>(sp + 64 * hf, dq, dk + (x % SK) * (CHUNK >> 4) + 512 * hf, id_qk, lead);
        kt_commit(bar(TB_SF + 2 * slot + hf), lead);
      };
      for (int wi = 0; wi < total && !dead;) {
        const int n = min(k.nb - k.j, total - wi);
        const bool idle = nt == 2 && (k.q % w.nrb) * KT_ROWS * nt + slot * KT_ROWS >= w.R;
        constexpr int STEP = nt == 2 ? 1 : 2;            // two tiles: every chunk; one: alternate ones
        const int i0 = nt == 2 ? 0 : slot;
        if (!kt_warp_wait(bar(TB_QF), qn & 1)) { dead = true; break; }
        tc_fence_after();
        if (idle) {                                      // no rows: only let the stages go
          for (int i = 0; i < n; ++i) {
            if (!wait_k(gc + i) || !wait_v(gc + i)) { dead = true; break; }
            kt_commit(bar(TB_KE + (gc + i) % SK), lead);
            kt_commit(bar(TB_VE + (gc + i) % SV), lead);
          }
        } else if (i0 < n) {
          if (!wait_k(gc + i0)) { dead = true; break; }
          scores(gc + i0, 0);
          scores(gc + i0, 1);
          kt_commit(bar(TB_KE + (gc + i0) % SK), lead);
          if (i0 + STEP >= n) kt_commit(bar(TB_QE), lead);
#pragma unroll 1
          for (int i = i0; i < n && !dead; i += STEP) {
            const int x = gc + i, xn = x + STEP;
            // one tile: slot 1's O may be overwritten only after the first warpgroup has merged it
            // into the previous block's partial (which also means that chunk x - 2's values, perhaps the
            // other slot's, have been there: without that the wait for this chunk's could end early)
            if (nt == 1 && i == 1 && qn > 0 && !kt_warp_wait(bar(TB_MFR), (qn - 1) & 1)) { dead = true; break; }
            if (!wait_v(x)) { dead = true; break; }
            // each half of P as it comes, and in its place the next chunk's scores
            int next = i + STEP < n ? 0 : 2;             // halves of the next chunk's scores issued
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
              if (!kt_warp_wait(bar(TB_PR + 2 * slot + hf), js & 1)) { dead = true; break; }
              tc_fence_after();
              kt_pv(od, sp + 64 * hf, dv + (x % SV) * (CHUNK >> 4) + 512 * hf, id_pv, i != i0 || hf, lead);
              kt_commit(bar(TB_OF + 2 * slot + hf), lead);
              if (hf == 1) kt_commit(bar(TB_VE + x % SV), lead);
              if (next == 0) {
                // the first half's scores wait for P's second half where their keys are not there yet
                const bool now = hf == 1 ? wait_k(xn) : __all_sync(0xffffffffu, mbar_test(bar(TB_KF + xn % SK), (xn / SK) & 1));
                if (hf == 1 && !now) { dead = true; break; }
                if (now) {
                  scores(xn, 0);
                  next = 1;
                }
              }
              if (hf == 1 && next == 1) {
                scores(xn, 1);
                kt_commit(bar(TB_KE + xn % SK), lead);
                if (i + 2 * STEP >= n) kt_commit(bar(TB_QE), lead);
              }
            }
            ++js;
          }
        }
        if (idle || i0 >= n) kt_commit(bar(TB_QE), lead);
        ++qn;
        gc += n;
        wi += n;
        k.j += n - 1;
        if (wi < total) kd_next(c, per, k);
        if (aborted()) break;
      }
      timed_out = dead;
      kt_commit(bar(TB_END), lead);                      // arrives once this warp's MMAs are done
    }
    else if (warp == KT_LOAD_WARP) {
      // ---------------------------------------------------------- copies: lane l < 8 block l
      // Blocks of one page lie side by side, so a page's (a contiguous cache's: the chunk's) go in
      // one copy, by the lane of the first.  The next chunk's pages are looked up a chunk ahead.
      const int upp = (c.page_table ? c.page_size : c.capacity) / KV4_SLOTS;
      const uint64_t pol = policy_evict_first();
      int issued[2] = {0, 0}, len_b = k.b, len = clamp_len(c, c.len[k.b]);
      auto page_of = [&]() {
        const int t = k.j * KT_KEYS + lane * KV4_SLOTS;
        return c.page_table && lane < 8 && t < len ? c.page_table[(long)k.b * c.pages_per_seq + t / c.page_size] : 0;
      };
      int page = page_of();
      for (int x = 0; x < total; ++x) {
        const int j = k.j, t = j * KT_KEYS + lane * KV4_SLOTS, valid = min(len - j * KT_KEYS, KT_KEYS);
        const int blocks = (valid + KV4_SLOTS - 1) / KV4_SLOTS;
        const int in = (c.page_table ? t % c.page_size : t) / KV4_SLOTS;
        const bool lead = lane < blocks && (lane == 0 || in == 0);
        const uint32_t bytes = lead ? min(upp - in, blocks - lane) * BLK : 0;
        long unit = c.page_table ? page : k.b;
        if (lead && c.page_table && (page < 0 || page >= c.num_pages)) {
          set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
          unit = 0;
        }
        const long off = ((unit * c.Hkv + k.q / w.nrb) * upp + in) * BLK;
        if (x + 1 < total) {
          kd_next(c, per, k);
          if (k.b != len_b) {
            len_b = k.b;
            len = clamp_len(c, c.len[k.b]);
          }
          page = page_of();
        }
        bool ok = true;
        for (int part = 0; part < 2 && ok; ++part) {
          const int slots = part ? SLV : SLK, st = (part ? SLK : 0) + x % slots;
          ok = kt_warp_wait(bar(TB_LE + st), ((x / slots) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            s_valid[st] = valid;
            mbar_expect_tx(bar(TB_LF + st), blocks * BLK);
          }
          __syncwarp();
          if (lead)
            bulk_load(l0s + st * STAGE + lane * BLK, static_cast<const uint8_t*>(part ? c.v : c.k) + off, bytes,
                      bar(TB_LF + st), pol);
          ++issued[part];
        }
        if (!ok) { timed_out = true; break; }
        if (aborted()) break;
      }
      // the last copies of each ring: if the block gives up nobody else waits for them (bounded)
      for (int part = 0; part < 2; ++part) {
        const int slots = part ? SLV : SLK;
        for (int x = max(0, issued[part] - slots); x < issued[part]; ++x)
          mbar_wait(bar(TB_LF + (part ? SLK : 0) + x % slots), (x / slots) & 1, TC_TIMEOUT_NS / 16);
      }
    } else {
      // ---------------------------------------------------------- slots of the partials
      for (int wi = 0; wi < total;) {
        const int n = min(k.nb - k.j, total - wi);
        const long pair = (long)k.b * per + k.q;
        if (lane == 0) {
          if (k.j == 0) w.span[pair].x = (int)(pair + blockIdx.x);
          if (k.j + n == k.nb) w.span[pair].y = (int)(pair + blockIdx.x) + 1;
        }
        wi += n;
        k.j += n - 1;
        if (wi < total) kd_next(c, per, k);
      }
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
    // 16 columns of the warp's 32 rows to global memory: the four lanes of a quad trade 16-byte
    // pieces so that each store writes 64 bytes of a row (a row a lane: 16, four times the lines).
    // dst: the quad's first row; rows: how many there are from it on.  Two tiles: 143 -> 139.5 us (43 x 4
    // rows); with one, where one warpgroup alone writes and the other goes on, 98 -> 102, so not there.
    auto store_rows = [&](float* dst, int rows, const float (&v)[16]) {
      const bool up2 = lane & 2, up1 = lane & 1;
      float lo[2][4], hi[2][4];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = v[4 * y + e], a1 = v[4 * y + 8 + e];
          const float got = __shfl_xor_sync(0xffffffffu, up2 ? a0 : a1, 2);
          lo[y][e] = up2 ? got : a0;
          hi[y][e] = up2 ? a1 : got;
        }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float r0[4], r1[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = z ? hi[0][e] : lo[0][e], a1 = z ? hi[1][e] : lo[1][e];
          const float got = __shfl_xor_sync(0xffffffffu, up1 ? a0 : a1, 1);
          r0[e] = up1 ? got : a0;
          r1[e] = up1 ? a1 : got;
        }
        float* at = dst + 2 * z * DH + (lane & 3) * 4;
        if (2 * z < rows) *reinterpret_cast<float4*>(at) = make_float4(r0[0], r0[1], r0[2], r0[3]);
        if (2 * z + 1 < rows) *reinterpret_cast<float4*>(at + DH) = make_float4(r1[0], r1[1], r1[2], r1[3]);
      }
    };
    if (w.a.test_wait_ns && slot == 0)
      timed_out = !__all_sync(0xffffffffu, mbar_wait(bar(TB_NEVER), 0, w.a.test_wait_ns));
    for (int wi = timed_out ? total : 0; wi < total;) {
      const int n = min(k.nb - k.j, total - wi);
      const int g = k.q / w.nrb, rblk = k.q - g * w.nrb, len = clamp_len(c, c.len[k.b]);
      const int row0 = rblk * KT_ROWS * nt, tile = nt == 2 ? slot : 0;
      const int gr = row0 + tile * KT_ROWS + r;
      const bool row_ok = gr < w.R;
      const bool live = row0 + tile * KT_ROWS + wl * 32 < w.R;     // the warp has rows
      // ---- the block's queries: scaled into [1, 2) by a power of two, as halves.  Two tiles: each
      // slot its own; one: the second slot, which is done with the block before sooner, while the
      // first one writes that block's partial (and finds the rows' factors in shared memory)
      float rs = 0.f;
      if (nt == 2 || slot == 1) {
        const int node = row_ok ? gr / w.a.G : 0, hq = g * w.a.G + (row_ok ? gr - node * w.a.G : 0);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const bf16*>(w.a.q) +
                                                          ((long)k.b * w.a.n1 + node) * w.a.q_row + hq * w.a.q_head);
        uint4 raw[DH / 8];
#pragma unroll
        for (int u = 0; u < DH / 8; ++u) raw[u] = row_ok ? src[u] : make_uint4(0u, 0u, 0u, 0u);
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < DH / 8; ++u) {
          float f[8];
          unpack16(raw[u], f);
#pragma unroll
          for (int e = 0; e < 8; e += 2) top = max3(top, fabsf(f[e]), fabsf(f[e + 1]));
        }
        float down;
        rs = row_scale(w.a, top, down);
        if (nt == 1) s_rs[qn & 1][r] = rs;
        if (qn > 0 && !kt_warp_wait(bar(TB_QE), (qn - 1) & 1)) { timed_out = true; break; }
        const uint32_t row = qs + tile * CHUNK + r * 128;
#pragma unroll
        for (int u = 0; u < DH / 8; ++u) {
          float f[8];
          unpack16(raw[u], f);
          st_shared16(row + (u >> 3) * TILE + (((u & 7) ^ (r & 7)) << 4), half_pair(f[0] * down, f[1] * down),
                      half_pair(f[2] * down, f[3] * down), half_pair(f[4] * down, f[5] * down),
                      half_pair(f[6] * down, f[7] * down));
        }
        fence_proxy_async();
        mbar_arrive(bar(TB_QF));
      }
      const bool idle = nt == 2 && row0 + tile * KT_ROWS >= w.R;   // this tile has no rows
      const int njobs = idle ? 0 : nt == 2 ? n : (n + 1 - slot) / 2;
      float m_use = -INFINITY, l_acc = 0.f;
      for (int jj = 0; jj < njobs; ++jj) {
        const int i = nt == 2 ? jj : 2 * jj + slot;
        const int t0 = (k.j + i) * KT_KEYS;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          if (!kt_warp_wait(bar(TB_SF + 2 * slot + hf), js & 1)) { timed_out = true; break; }
          tc_fence_after();
          if (nt == 1 && slot == 0 && jj == 0 && hf == 0) rs = s_rs[qn & 1][r];
          if (live) {
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
              x0 = max3(x0, s[j], s[j + 1]);
              x1 = max3(x1, s[j + 2], s[j + 3]);
            }
            const float mx = fmaxf(x0, x1) * rs;     // the row's factor is positive
            const bool raise = !(mx <= m_use + KD_TOP);
            if (__any_sync(0xffffffffu, raise)) {
              const float mn = raise ? mx - KD_BACK<false> : m_use;
              const float f = !raise ? 1.f : m_use == -INFINITY ? 0.f : ex2_approx(m_use - mn);
              // O is rescaled once the half before has been added to it; a block's first half finds none
              if (jj > 0 || hf == 1) {
                if (!kt_warp_wait(bar(TB_OF + 2 * slot + (hf ^ 1)), (hf ? js : js - 1) & 1)) { timed_out = true; break; }
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < DH; x += 16) {
                  float v[16];
                  kt_ld16(ocol + x, v);
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[e] *= f;
                  tmem_st16(ocol + x, v);
                }
              }
              l_acc *= f;
              m_use = mn;
            }
            F2 ls = f2(0.f, 0.f);
            uint32_t pk[32];
            const float nm = -m_use;
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              float p0, p1;
              unf2(fma2(f2(s[j], s[j + 1]), f2(rs, rs), f2(nm, nm)), p0, p1);
              p0 = ex2_approx(p0); p1 = ex2_approx(p1);
              ls = add2(ls, f2(p0, p1));
              pk[j / 2] = half_pair(p0, p1);
            }
            kt_st32(scol + 64 * hf, pk);
            kt_st_wait();
            float l0, l1; unf2(ls, l0, l1); l_acc += l0 + l1;
          }
          tc_fence_before();
          mbar_arrive(bar(TB_PR + 2 * slot + hf));
        }
        if (timed_out) break;
        ++js;
      }
      if (timed_out) break;
      ++qn;
      // ---- the block's partial
      const long pair = (long)k.b * per + k.q, part = pair + blockIdx.x;
      const long prow = part * w.rb + tile * KT_ROWS + r;
      float* dst = w.part_o + prow * DH;
      if (nt == 2) {
        if (njobs > 0 && live) {
          if (!kt_warp_wait(bar(TB_OF + 2 * slot + 1), (js - 1) & 1)) { timed_out = true; break; }
          tc_fence_after();
#pragma unroll 2
          for (int x = 0; x < DH; x += 16) {
            float v[16];
            kt_ld16(ocol + x, v);
            store_rows(dst - (lane & 3) * DH + x, w.R - (gr - (lane & 3)), v);
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
        bool ok = kt_warp_wait(bar(TB_OF + 1), (js - 1) & 1);
        // the second slot's softmax first: it ends once all of its products but the last are done
        if (ok) ok = kt_warp_wait(bar(TB_MRG), mc & 1);
        if (ok && nj1 > 0) ok = kt_warp_wait(bar(TB_OF + 3), (js1 - 1) & 1);
        if (!ok) { timed_out = true; break; }
        tc_fence_after();
        const float2 ml1 = s_ml[r];
        const float m = fmaxf(m_use, ml1.x);
        const float f0 = m_use == -INFINITY ? 0.f : ex2_approx(m_use - m);
        const float f1 = ml1.x == -INFINITY ? 0.f : ex2_approx(ml1.x - m);
        const uint32_t ocol1 = lane_base + KT_SLOT_COLS + KT_KEYS;
        if (live) {
#pragma unroll 2
          for (int x = 0; x < DH; x += 16) {
            float v0[16], v1[16];
            kt_ld16(ocol + x, v0);
            if (nj1 > 0) {
              kt_ld16(ocol1 + x, v1);            // written by this block's P V of slot 1
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
      if (wi < total) kd_next(c, per, k);
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

template <int DH, int NT> static cudaError_t tree_go(const Kv4Work& w, int num_sms, cudaStream_t st) {
  constexpr size_t CHUNK = DH / 64 * 128 * 128, STAGE = 8 * kv4_block(DH);
  constexpr size_t smem = 1024 + (NT + 2 * KT_ST) * CHUNK + (NT == 2 ? 3 : 6) * STAGE;
  static unsigned long long done = 0;
  const cudaError_t e = allow_smem(kv4_tree_kernel<DH, NT>, smem, &done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv4_tree_kernel<DH, NT>, dim3(num_sms), dim3(KT_THREADS), smem, st, 1, w);
}

cudaError_t launch_kv4_tree(const Kv4Work& w, int num_sms, cudaStream_t st) {
  const bool two = w.R > KT_ROWS;
  if (w.a.c.dh == 128) return two ? tree_go<128, 2>(w, num_sms, st) : tree_go<128, 1>(w, num_sms, st);
  return two ? tree_go<64, 2>(w, num_sms, st) : tree_go<64, 1>(w, num_sms, st);
}

}  // namespace medusa
