// Attention of a batch whose sequences share a prefix ("Medusa: Simple LLM Inference Acceleration Framework
// with Multiple Decoding Heads" §3.4 Tree Attention, Steps 3 and 5, with the common part of the prefixes
// held once): the kernel for float rows and small heads, on the CUDA cores, and the joining kernel.
//
// A CTA has 64 query rows; of a chunk of 128 keys it takes two halves of 64 through shared memory in float.
// A thread has 4 rows x 4 keys of the scores and 4 rows x dh/16 columns of o; a row's 64 scores lie in 16
// lanes, which share its running maximum m and sum l: o = sum 2^(s - m) v, l = sum 2^(s - m), s in base-2
// units.  Products run two at a time (packed), and a half's keys and values are all asked for before the first is
// used: 3 x 31 x 4 float rows over 777 + 0-100 slots of 64 elements 32 -> 20 us, 13 of them one chunk's products.
//
// Measured (one GB300), large calls: 16 x 43 nodes of 4 x 8 heads over 8192 + 64-512 slots, float, heads of 128 3.1 ms (31
// TFLOP/s), of 64 1.83 ms (26); bf16 heads of 32 1.25 ms (19); 32 single rows over 16384, float heads of 128 555 us (0.55
// TB/s).  What bounds them: 8 warps an SM with nothing in flight while they multiply, and shared memory, from which 4 x 4
// scores read eight 16-byte words for 32 packed products.
#include <algorithm>

#include "launch.cuh"
#include "prefix.cuh"
#include "units.cuh"
#include "tc_ptx.cuh"

namespace medusa {

constexpr int PS_ROWS = 64, PS_KEYS = 64;

__device__ __forceinline__ bool nonfinite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

template <typename T, int DH>
__global__ void __launch_bounds__(256) prefix_simt_kernel(PxWork w) {
  constexpr int P = DH + 4, C = DH / 16, UNITS = PS_KEYS * DH / 4 / 256;
  static_assert(PS_ROWS == PS_KEYS, "queries and keys are loaded alike");
  extern __shared__ float sm[];
  float* Qs = sm;                                 // [64][DH + 4]
  float* Ks = Qs + PS_ROWS * P;                   // [64][DH + 4]
  float* Vs = Ks + PS_KEYS * P;                   // [64][DH]
  float* Ps = Vs + PS_KEYS * DH;                  // [64][64 + 4]
  __shared__ uint32_t s_bad[2];                   // keys whose value holds an infinity or a NaN
  pdl_trigger();
  pdl_wait();
  const PrefixArgs& a = w.a;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const PxPlan plan = px_plan(w, blockIdx.x == 0 && tid < 32);
  PxWalk walk = px_start(w, plan, blockIdx.x);
  const bool shared = walk.shared;
  const CacheView& c = shared ? a.shared : a.own;
  PxSeg s;
  while (px_next(w, walk, s)) {
    const int b = shared ? 0 : s.b, len = clamp_len(c, c.len[b]), prefix_chunks = (len + PX_KEYS - 1) / PX_KEYS;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {             // four elements a thread at a time
      const int e = tid + u * 256, r = e / (DH / 4), i = e % (DH / 4) * 4;
      const PxRow x = px_row(w, shared, s, r);
      float v[4] = {};
      if (x.ok) load4(static_cast<const T*>(a.q) + x.node_row * a.q_row + x.head * a.q_head + i, true, v);
      *reinterpret_cast<float4*>(Qs + r * P + i) = make_float4(v[0], v[1], v[2], v[3]);
    }
    F2 o[4][C / 2];
    float m[4], l[4] = {};
    PxRow row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
#pragma unroll
      for (int e = 0; e < C / 2; ++e) o[i][e] = f2(0.f, 0.f);
      row[i] = px_row(w, shared, s, ty + 16 * i);
    }
    for (int jj = 2 * s.j; jj < 2 * (s.j + s.n); ++jj) {
      const bool tree = jj / 2 >= prefix_chunks;
      const int t0 = tree ? jj * PS_KEYS - prefix_chunks * PX_KEYS : jj * PS_KEYS, end = tree ? a.n1 : len;
      if (t0 >= end) continue;
      __syncthreads();
      if (tid < 2) s_bad[tid] = 0;
      __syncthreads();
      float kx[UNITS][4], vx[UNITS][4];           // all asked for before the first is used
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int e = tid + u * 256, t = t0 + e / (DH / 4), i = e % (DH / 4) * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) kx[u][q] = vx[u][q] = 0.f;
        if (t >= end) continue;
        const T *ks, *vs;
        if (tree) {
          const long at = (((long)b * a.n1 + t) * c.Hkv + s.g) * DH + i;
          ks = static_cast<const T*>(a.tk) + at;
          vs = static_cast<const T*>(a.tv) + at;
        } else {
          long unit;
          int in;
          if (!unit_of(c, b, t, unit, in)) {
            set_flag(c.status, MEDUSA_FLAG_PAGE_RANGE);
            unit = 0;
          }
          const long at = plain_offset(c, unit, in, s.g) + i;
          ks = static_cast<const T*>(c.k) + at;
          vs = static_cast<const T*>(c.v) + at;
        }
        load4(ks, true, kx[u]);
        load4(vs, true, vx[u]);
      }
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int e = tid + u * 256, j = e / (DH / 4), i = e % (DH / 4) * 4;
        if (tree && (nonfinite(vx[u][0]) || nonfinite(vx[u][1]) || nonfinite(vx[u][2]) || nonfinite(vx[u][3]))) {
          // not every row sees it: 0, and a NaN sum for those that do
#pragma unroll
          for (int q = 0; q < 4; ++q) vx[u][q] = 0.f;
          atomicOr(&s_bad[j >> 5], 1u << (j & 31));
        }
        *reinterpret_cast<float4*>(Ks + j * P + i) = make_float4(kx[u][0], kx[u][1], kx[u][2], kx[u][3]);
        *reinterpret_cast<float4*>(Vs + j * DH + i) = make_float4(vx[u][0], vx[u][1], vx[u][2], vx[u][3]);
      }
      __syncthreads();
      F2 p2[4][4];                                // even and odd elements' sums
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) p2[u][v] = f2(0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < DH; i += 4) {
        ulonglong2 q[4], k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          q[u] = *reinterpret_cast<const ulonglong2*>(Qs + (ty + 16 * u) * P + i);
          k[u] = *reinterpret_cast<const ulonglong2*>(Ks + (tx + 16 * u) * P + i);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            p2[u][v] = fma2(F2{q[u].y}, F2{k[v].y}, fma2(F2{q[u].x}, F2{k[v].x}, p2[u][v]));
      }
      float p[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float a0, a1;
          unf2(p2[u][v], a0, a1);
          p[u][v] = a0 + a1;
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t see[2] = {0xffffffffu, 0xffffffffu};
        if (tree && row[u].ok)
          for (int i = 0; i < 2; ++i) see[i] = px_sees(a, row[u].n, (t0 >> 5) + i);
        float mx = -INFINITY;
        bool bad = false;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int j = tx + 16 * v;
          const bool seen = row[u].ok && t0 + j < end && ((see[j >> 5] >> (j & 31)) & 1u);
          p[u][v] = seen ? p[u][v] * a.scale2 : -INFINITY;
          bad |= seen && ((s_bad[j >> 5] >> (j & 31)) & 1u);
          mx = fmaxf(mx, p[u][v]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float top = fmaxf(m[u], mx), ref = top == -INFINITY ? 0.f : top;
        const float f = m[u] == -INFINITY ? 0.f : exp2f(m[u] - ref);
        float sum = bad ? NAN : 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float x = exp2f(p[u][v] - ref);
          sum += x;
          Ps[(ty + 16 * u) * 68 + tx + 16 * v] = x;
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[u] = l[u] * f + sum;
        m[u] = top;
#pragma unroll
        for (int i = 0; i < C / 2; ++i) o[u][i] = mul2(o[u][i], f2(f, f));
      }
      __syncwarp();                               // a row's probabilities are read by its own 16 lanes
      for (int j = 0; j < PS_KEYS; j += 4) {
        float pr[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 x = *reinterpret_cast<const float4*>(Ps + (ty + 16 * u) * 68 + j);
          pr[u][0] = x.x;
          pr[u][1] = x.y;
          pr[u][2] = x.z;
          pr[u][3] = x.w;
        }
#pragma unroll
        for (int jj2 = 0; jj2 < 4; ++jj2) {
          F2 v[C / 2];
#pragma unroll
          for (int i = 0; i < C / 2; ++i)
            v[i].v = *reinterpret_cast<const unsigned long long*>(Vs + (j + jj2) * DH + tx * 2 + 32 * i);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < C / 2; ++i) o[u][i] = fma2(f2(pr[u][jj2], pr[u][jj2]), v[i], o[u][i]);
        }
      }
    }
    const int rb = shared ? w.rbs : w.rbo;
    float* po = shared ? w.o_s : w.o_o;
    float2* pml = shared ? w.ml_s : w.ml_o;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = ty + 16 * u;
      if (!row[u].ok) continue;
      const long at = s.slot * rb + r;
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        *reinterpret_cast<unsigned long long*>(po + at * DH + tx * 2 + 32 * i) = o[u][i].v;
      if (tx == 0) pml[at] = make_float2(l[u] != l[u] && m[u] == -INFINITY ? 0.f : m[u], l[u]);
    }
  }
}

// o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over a row's partials, M the largest m_s.  Eight lanes have
// a row (dh/8 columns each), so that four rows' loads are in flight a warp: a row's time is a chain of loads (its
// length, its references, its sums).  A row's partials are those of the CTAs that its item's chunks lie in:
// with W units over C CTAs unit x is CTA ceil((x + 1) C / W) - 1's.
constexpr int PJ_THREADS = 64;                    // few: small calls have a block an SM, and each round of loads counts
template <typename T, int DH>
__global__ void __launch_bounds__(PJ_THREADS) prefix_join_kernel(PxWork w) {
  constexpr int SB = 4, U = DH / 32;              // partials a round, 16-byte units a lane
  pdl_trigger();
  pdl_wait();
  const PrefixArgs& a = w.a;
  const long i = (long)blockIdx.x * (PJ_THREADS / 8) + (threadIdx.x >> 3);
  if (i >= (long)w.rows * a.own.Hkv) return;
  const int lane = threadIdx.x & 7;
  const int g = (int)(i / w.rows), gr = (int)(i - (long)g * w.rows);       // row of head g over all sequences
  const int b = gr / w.R, r = gr - b * w.R, node = gr / a.G, head = g * a.G + gr - node * a.G;
  const PxPlan p = *w.plan;
  const int nb = px_chunks(w, b);
  const long first = w.first[b];
  auto cta = [](long x, long n, long total) { return (((x + 1) * n + total - 1) / total) - 1; };
  // the row's first partial, how far the next one is and how many there are: of the shared item, of the own one
  long at[2] = {0, 0};
  int n[2] = {0, 0};
  if (p.ns > 0) {
    const int rbi = gr / w.rbs, item = g * w.nrbs + rbi;
    const long x = (long)item * px_units(w, p.ns) + w.item, c0 = cta(x, p.cs, p.ws);
    n[0] = (int)(cta(x + p.ns - 1, p.cs, p.ws) - c0) + 1;
    at[0] = (c0 + item) * w.rbs + gr - rbi * w.rbs;
  }
  if (nb > 0) {
    const int rbi = r / w.rbo, per = a.own.Hkv * w.nrbo, item = g * w.nrbo + rbi;
    const long x = first * per + (long)item * px_units(w, nb) + w.item, c0 = cta(x, p.co, p.wo);
    n[1] = (int)(cta(x + nb - 1, p.co, p.wo) - c0) + 1;
    at[1] = (c0 + (long)b * per + item) * w.rbo + r - rbi * w.rbo;
  }
  float M = -INFINITY, L = 0.f, acc[U][4] = {};
#pragma unroll 1
  for (int s0 = 0; s0 < n[0] + n[1]; s0 += SB) {
    float2 ml[SB];
    float4 v[SB][U];
#pragma unroll
    for (int u = 0; u < SB; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < U; ++e) v[u][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int i = s0 + u, own = i - n[0];
      if (own >= n[1]) continue;
      const long row = own < 0 ? at[0] + (long)i * w.rbs : at[1] + (long)own * w.rbo;
      ml[u] = (own < 0 ? w.ml_s : w.ml_o)[row];
      const float* po = (own < 0 ? w.o_s : w.o_o) + row * DH + lane * 4;
#pragma unroll
      for (int e = 0; e < U; ++e) v[u][e] = *reinterpret_cast<const float4*>(po + e * 32);
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < SB; ++u) top = fmaxf(top, ml[u].x);
    if (top == -INFINITY) continue;               // nothing seen so far
    const float f = M == -INFINITY ? 0.f : exp2f(M - top);
    L *= f;
#pragma unroll
    for (int e = 0; e < U; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[e][q] *= f;
    M = top;
#pragma unroll
    for (int u = 0; u < SB; ++u) {
      if (ml[u].x == -INFINITY) continue;
      const float x = exp2f(ml[u].x - M);
      L += x * ml[u].y;
#pragma unroll
      for (int e = 0; e < U; ++e) {
        acc[e][0] += x * v[u][e].x;
        acc[e][1] += x * v[u][e].y;
        acc[e][2] += x * v[u][e].z;
        acc[e][3] += x * v[u][e].w;
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;     // (a NaN sum stays one)
  T* dst = static_cast<T*>(a.o) + (long)node * a.o_row + (long)head * a.o_head + lane * 4;
#pragma unroll
  for (int e = 0; e < U; ++e) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[e][q] = L == 0.f ? 0.f : acc[e][q] * inv;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(dst + e * 32) = make_float4(acc[e][0], acc[e][1], acc[e][2], acc[e][3]);
    } else {
      *reinterpret_cast<uint2*>(dst + e * 32) = make_uint2(pack2(acc[e][0], acc[e][1]), pack2(acc[e][2], acc[e][3]));
    }
  }
}

// ------------------------------------------------------------------ host side
// Rows of a block: 64 here, on the tensor cores a tile of 128 rows or two.
static void row_blocks(bool tc, int R, int* rb, int* nrb) {
  const int most = !tc ? PS_ROWS : R > 128 ? 256 : 128;
  *rb = std::min(R, most);
  *nrb = (R + most - 1) / most;
}
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static int max_ctas(int num_sms) { return std::max(2, num_sms); }

size_t prefix_workspace(int B, int Hq, int Hkv, int dh, int max_nodes, int num_sms) {
  // slots of a kind: its items and a CTA's each; items' blocks together: their rows, and a block over
  const size_t G = Hq / Hkv, R = (size_t)max_nodes * G, C = max_ctas(num_sms);
  const size_t rbo = std::min<size_t>(R, 256), rbs = std::min<size_t>((size_t)B * R, 256);
  const size_t own = (size_t)B * Hkv * (R + rbo) + C * rbo, shared = Hkv * ((size_t)B * R + rbs) + C * rbs;
  return up256(sizeof(PxPlan)) + up256(B * sizeof(long)) + up256(own * dh * 4) + up256(own * 8) +
         up256(shared * dh * 4) + up256(shared * 8);
}

template <typename T, int DH> static cudaError_t simt_go(const PxWork& w, cudaStream_t st) {
  const size_t smem = (size_t)(2 * PS_ROWS * (DH + 4) + PS_KEYS * DH + PS_ROWS * 68) * sizeof(float);
  static unsigned long long done = 0;
  const cudaError_t e = allow_smem(prefix_simt_kernel<T, DH>, smem, &done);
  if (e != cudaSuccess) return e;
  return launch_kernel(prefix_simt_kernel<T, DH>, dim3(w.ctas), dim3(256), smem, st, 1, w);
}
template <typename T> static cudaError_t prefix_go(const PxWork& w, bool tc, cudaStream_t st) {
  cudaError_t e;
  const int dh = w.a.own.dh;
  if (tc) e = launch_prefix_tc(w, st);
  else if (dh == 32) e = simt_go<T, 32>(w, st);
  else if (dh == 64) e = simt_go<T, 64>(w, st);
  else e = simt_go<T, 128>(w, st);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(((long)w.rows * w.a.own.Hkv + PJ_THREADS / 8 - 1) / (PJ_THREADS / 8)));
  if (dh == 32) return launch_kernel(prefix_join_kernel<T, 32>, grid, dim3(PJ_THREADS), 0, st, 1, w);
  if (dh == 64) return launch_kernel(prefix_join_kernel<T, 64>, grid, dim3(PJ_THREADS), 0, st, 1, w);
  return launch_kernel(prefix_join_kernel<T, 128>, grid, dim3(PJ_THREADS), 0, st, 1, w);
}

cudaError_t launch_prefix_attention(const PrefixArgs& a, int dtype, void* ws, int num_sms, cudaStream_t st) {
  const bool tc = prefix_tc_takes(dtype, a.own.dh);
  PxWork w{};
  w.a = a;
  w.R = a.n1 * a.G;
  w.rows = a.own.B * w.R;
  row_blocks(tc, w.rows, &w.rbs, &w.nrbs);
  row_blocks(tc, w.R, &w.rbo, &w.nrbo);
  // In units of half a chunk against one tile.  A chunk against two tiles takes 3 (2: 8 x 65 nodes 84 us for 77), and an item
  // besides as long as 3 chunks (1: 102; 2 and 4: 32 single rows 52 and 53 us for 50).  On the CUDA cores calls are small, and
  // a share without chunks would be an idle CTA (3: 3 x 31 nodes 30 us for 20).
  w.item = tc ? 3 : 0;
  w.cost_s = tc && w.rbs > 128 ? 3 : 2;
  w.cost_o = tc && w.rbo > 128 ? 3 : 2;
  w.tree = a.tk ? (a.n1 + PX_KEYS - 1) / PX_KEYS : 0;
  w.ctas = max_ctas(num_sms);
  char* p = static_cast<char*>(ws);
  auto take = [&](size_t bytes) {
    char* at = p;
    p += up256(bytes);
    return at;
  };
  w.plan = reinterpret_cast<PxPlan*>(take(sizeof(PxPlan)));
  w.first = reinterpret_cast<long*>(take(a.own.B * sizeof(long)));
  const size_t so = ((size_t)a.own.B * a.own.Hkv * w.nrbo + w.ctas) * w.rbo;
  const size_t ss = ((size_t)a.own.Hkv * w.nrbs + w.ctas) * w.rbs;
  w.o_o = reinterpret_cast<float*>(take(so * a.own.dh * 4));
  w.ml_o = reinterpret_cast<float2*>(take(so * 8));
  w.o_s = reinterpret_cast<float*>(take(ss * a.own.dh * 4));
  w.ml_s = reinterpret_cast<float2*>(take(ss * 8));
  return dtype == MEDUSA_F32 ? prefix_go<float>(w, tc, st) : prefix_go<bf16>(w, tc, st);
}

}  // namespace medusa
