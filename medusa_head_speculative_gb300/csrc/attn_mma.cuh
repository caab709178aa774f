// Pieces of the attention kernels whose two slots have a warp of MMAs and a warpgroup of softmax each
// (k_kv4_tree.cu, k_prefix_tc.cu): the MMAs of half a chunk (64 keys), loads and stores of tensor memory.
#pragma once
#include "common.cuh"
#include "tc_ptx.cuh"

namespace medusa {

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
// 16 columns of 32 bits of this thread's TMEM lane, without the wait.
__device__ __forceinline__ void kt_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 32 columns of this thread's TMEM lane, load and wait in one statement.
__device__ __forceinline__ void kt_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
      "%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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

// 16 columns of the warp's 32 rows to global memory ([row][DH], row r the lane's): the four lanes of a quad
// trade 16-byte pieces so that each store writes 64 bytes of a row (a row a lane: 16, four times the lines).
// dst: the quad's first row; rows: how many there are from it on.
template <int DH> __device__ __forceinline__ void store_quads(float* dst, int rows, int lane, const float (&v)[16]) {
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
}

}  // namespace medusa
