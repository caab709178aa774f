// C ABI of the rotary positions and the KV caches: handles, checks and launches.  The rules
// every call keeps to are in include/medusa.h.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <new>

#include "cache.h"
#include "common.cuh"
#include "launch.cuh"

using namespace medusa;

struct medusa_rope {
  medusa_rope_desc d;
  float* cs = nullptr;
  uint32_t* status = nullptr;
  int device = 0;
};

struct medusa_cache {
  medusa_cache_dims d;
  uint32_t* status = nullptr;
  int device = 0, num_sms = 152;
  size_t pool_bytes = 0, ws_bytes = 0;
  mutable std::atomic<unsigned long long> test_wait_ns{0};
};

namespace {

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
size_t elem(int dtype) { return dtype == MEDUSA_F32 ? 4 : 2; }
bool is_dtype(int t) { return t == MEDUSA_F32 || t == MEDUSA_BF16; }
// A handle's memory lives on the device that was current when it was made.
bool here(int device) {
  int d = -1;
  return cudaGetDevice(&d) == cudaSuccess && d == device;
}
// Whether no two of rows x heads pieces of dh elements, row and head elements apart, share an element: results
// that lie on one another would be written in any order.
bool lie_apart(long long rows, long long row, long long heads, long long head, int dh) {
  if ((rows > 1 && row < dh) || (heads > 1 && head < dh)) return false;
  if (rows <= 1 || heads <= 1) return true;
  if (row >= (__int128)(heads - 1) * head + dh || head >= (__int128)(rows - 1) * row + dh) return true;
  for (long long i = 1; i < heads; ++i) {          // neither within the other's gaps: piece by piece
    const __int128 at = (__int128)i * head, j = at / row;
    if ((j < rows && at - j * row < dh) || (j + 1 < rows && (j + 1) * row - at < dh)) return false;
  }
  return true;
}
medusa_status done(cudaError_t e) { return e == cudaSuccess ? MEDUSA_OK : MEDUSA_ERR_CUDA; }

medusa_status read_status(uint32_t* word, void* stream, uint32_t* flags) {
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, S(stream)) != cudaSuccess ||
      cudaMemsetAsync(word, 0, sizeof(v), S(stream)) != cudaSuccess || cudaStreamSynchronize(S(stream)) != cudaSuccess)
    return MEDUSA_ERR_CUDA;
  *flags = v;
  return v ? MEDUSA_ERR_DEVICE : MEDUSA_OK;
}

bool finite_pos(double x) { return x > 0 && std::isfinite(x); }

medusa_status check_rope(const medusa_rope_desc* d) {
  if (!d || d->rot < 2 || d->rot % 2 != 0 || d->max_pos < 1) return MEDUSA_ERR_INVALID;
  if (d->layout != MEDUSA_ROPE_HALF && d->layout != MEDUSA_ROPE_INTERLEAVED) return MEDUSA_ERR_INVALID;
  if (d->scaling < MEDUSA_ROPE_PLAIN || d->scaling > MEDUSA_ROPE_RAMP) return MEDUSA_ERR_INVALID;
  if (!(d->base > 1.0) || !std::isfinite(d->base) || !std::isfinite(d->attn) || d->attn < 0)
    return MEDUSA_ERR_INVALID;
  if (d->scaling != MEDUSA_ROPE_PLAIN && !finite_pos(d->factor)) return MEDUSA_ERR_INVALID;
  if (d->scaling >= MEDUSA_ROPE_BANDED &&
      (!finite_pos(d->orig_pos) || !finite_pos(d->low) || !finite_pos(d->high) || !(d->low < d->high)))
    return MEDUSA_ERR_INVALID;
  if (d->rot > 1024) return MEDUSA_ERR_UNSUPPORTED;
  return MEDUSA_OK;
}

void rope_frequencies(const medusa_rope_desc& d, double* f) {
  const int h = d.rot / 2;
  const double two_pi = 6.283185307179586476925286766559;
  auto index_of = [&](double turns) {
    return d.rot * std::log(d.orig_pos / (two_pi * turns)) / (2.0 * std::log(d.base));
  };
  double a = 0, b = 0;
  if (d.scaling == MEDUSA_ROPE_RAMP) {
    a = std::fmax(0.0, std::floor(index_of(d.high)));
    b = std::fmin(d.rot - 1.0, std::ceil(index_of(d.low)));
  }
  for (int i = 0; i < h; ++i) {
    const double t = std::pow(d.base, -2.0 * i / d.rot);
    double w = 1.0;                                  // share of the plain frequency
    if (d.scaling == MEDUSA_ROPE_LINEAR) w = 0.0;
    if (d.scaling == MEDUSA_ROPE_BANDED) w = (d.orig_pos * t / two_pi - d.low) / (d.high - d.low);
    if (d.scaling == MEDUSA_ROPE_RAMP) w = 1.0 - (i - a) / std::fmax(b - a, 0.001);
    w = std::fmin(1.0, std::fmax(0.0, w));
    f[i] = d.scaling == MEDUSA_ROPE_PLAIN ? t : d.scaling == MEDUSA_ROPE_LINEAR ? t / d.factor
                                                                                 : w * t + (1.0 - w) * t / d.factor;
  }
}

RopeTable table_of(const medusa_rope* r) { return {r->cs, r->d.rot, r->d.max_pos, r->d.layout, r->status}; }

medusa_status check_cache(const medusa_cache_dims* d) {
  if (!d || d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->dh < 1 || d->Hq % d->Hkv != 0) return MEDUSA_ERR_INVALID;
  if (d->format != MEDUSA_F32 && d->format != MEDUSA_BF16 && d->format != MEDUSA_KV4) return MEDUSA_ERR_INVALID;
  if (d->capacity < 1 || d->page_size < 0 || d->max_nodes < 1) return MEDUSA_ERR_INVALID;
  if (d->page_size > 0 && (d->capacity % d->page_size != 0 || d->num_pages < 1)) return MEDUSA_ERR_INVALID;
  if (d->dh != 32 && d->dh != 64 && d->dh != 128) return MEDUSA_ERR_UNSUPPORTED;
  if (d->Hq > 65535 || d->B > (1 << 22)) return MEDUSA_ERR_UNSUPPORTED;         // launch grids
  if (d->max_nodes > MEDUSA_MAX_NODES || d->capacity > MEDUSA_MAX_CAPACITY) return MEDUSA_ERR_UNSUPPORTED;
  // far beyond any memory: sizes in bytes stay below 2^63
  const double slots = d->page_size > 0 ? (double)d->num_pages * d->page_size : (double)d->B * d->capacity;
  const double most = 1125899906842624.0;                                      // 2^50 elements
  if (slots * d->Hkv * d->dh > most || (double)d->B * d->Hq * d->max_nodes * d->dh > most)
    return MEDUSA_ERR_UNSUPPORTED;
  if (d->format == MEDUSA_KV4 && (d->page_size > 0 ? d->page_size : d->capacity) % 16 != 0)
    return MEDUSA_ERR_UNSUPPORTED;
  return MEDUSA_OK;
}

medusa_status check_kv(const medusa_cache* c, const medusa_kv* kv, bool out) {
  if (!kv || !kv->k || !kv->v || !kv->len) return MEDUSA_ERR_INVALID;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return MEDUSA_ERR_INVALID;
  if (c->d.page_size > 0 && !kv->page_table) return MEDUSA_ERR_INVALID;
  if (out && !kv->len_out) return MEDUSA_ERR_INVALID;
  return MEDUSA_OK;
}

medusa_status check_scales(const medusa_cache* c, float gk, float gv) {
  auto ok = [](float g) { return g >= 1e-20f && g <= 1e20f; };
  if (c->d.format == MEDUSA_KV4 && (!ok(gk) || !ok(gv))) return MEDUSA_ERR_INVALID;
  return MEDUSA_OK;
}

CacheView view_of(const medusa_cache* c, const medusa_kv* kv, float gk, float gv) {
  const medusa_cache_dims& d = c->d;
  CacheView v{};
  v.k = kv->k;
  v.v = kv->v;
  v.page_table = d.page_size > 0 ? kv->page_table : nullptr;
  v.len = kv->len;
  v.len_out = kv->len_out;
  v.B = d.B;
  v.Hkv = d.Hkv;
  v.dh = d.dh;
  v.capacity = d.capacity;
  v.page_size = d.page_size;
  v.pages_per_seq = d.page_size > 0 ? d.capacity / d.page_size : 0;
  v.num_pages = d.num_pages;
  v.gk = gk;
  v.gv = gv;
  v.status = c->status;
  return v;
}

// rows, start, per_seq, count of medusa_kv_rows and medusa_kv_places
template <typename T> medusa_status check_items(const medusa_cache* c, const T* r, ItemMap* m) {
  if (!r || !is_dtype(r->dtype) || r->rows < 0 || (r->rows > 0 && (!r->k || !r->v))) return MEDUSA_ERR_INVALID;
  if (!aligned(r->k, elem(r->dtype)) || !aligned(r->v, elem(r->dtype))) return MEDUSA_ERR_INVALID;
  if (r->k_row < 0 || r->k_head < 0 || r->v_row < 0 || r->v_head < 0) return MEDUSA_ERR_INVALID;
  constexpr long long kApart = 1ll << 31;                  // heads lie less than this many bytes apart
  if (r->k_head * (long long)elem(r->dtype) >= kApart || r->v_head * (long long)elem(r->dtype) >= kApart)
    return MEDUSA_ERR_UNSUPPORTED;
  if (!r->start && (r->per_seq < 1 || (long long)r->per_seq * c->d.B != r->rows)) return MEDUSA_ERR_INVALID;
  m->rows = r->rows;
  m->per_seq = r->start ? 0 : r->per_seq;
  m->start = r->start;
  m->count = r->start ? nullptr : r->count;
  return MEDUSA_OK;
}
template <typename T> bool vector_rows(const T* r) {
  const long long n = 16 / (long long)elem(r->dtype);
  return aligned(r->k, 16) && aligned(r->v, 16) && r->k_row % n == 0 && r->k_head % n == 0 && r->v_row % n == 0 &&
         r->v_head % n == 0;
}

}  // namespace

extern "C" {

medusa_status medusa_rope_create(const medusa_rope_desc* desc, medusa_rope** out) {
  if (!out) return MEDUSA_ERR_INVALID;
  *out = nullptr;
  const medusa_status s = check_rope(desc);
  if (s != MEDUSA_OK) return s;
  medusa_rope* r = new (std::nothrow) medusa_rope();
  if (!r) return MEDUSA_ERR_CUDA;
  r->d = *desc;
  double freq[512];
  rope_frequencies(r->d, freq);
  double* d_freq = nullptr;
  cudaStream_t st = nullptr;
  const size_t n = (size_t)desc->rot / 2 * sizeof(double);
  bool ok = cudaGetDevice(&r->device) == cudaSuccess &&
            cudaMalloc(&r->cs, (size_t)desc->max_pos * desc->rot * sizeof(float)) == cudaSuccess &&
            cudaMalloc(&r->status, sizeof(uint32_t)) == cudaSuccess && cudaMalloc(&d_freq, n) == cudaSuccess &&
            cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) == cudaSuccess;
  if (ok) {
    pdl_reset();
    ok = cudaMemcpyAsync(d_freq, freq, n, cudaMemcpyHostToDevice, st) == cudaSuccess &&
         cudaMemsetAsync(r->status, 0, sizeof(uint32_t), st) == cudaSuccess &&
         launch_rope_fill(r->cs, d_freq, desc->rot, desc->max_pos, desc->attn > 0 ? desc->attn : 1.0, st) ==
             cudaSuccess &&
         cudaStreamSynchronize(st) == cudaSuccess;
  }
  if (st) cudaStreamDestroy(st);
  if (d_freq) cudaFree(d_freq);
  if (!ok) {
    cudaGetLastError();                    // an allocation that failed leaves no error behind
    medusa_rope_destroy(r);
    return MEDUSA_ERR_CUDA;
  }
  *out = r;
  return MEDUSA_OK;
}

void medusa_rope_destroy(medusa_rope* r) {
  if (!r) return;
  if (r->cs) cudaFree(r->cs);
  if (r->status) cudaFree(r->status);
  delete r;
}

medusa_status medusa_rope_get_status(const medusa_rope* r, void* stream, uint32_t* flags) {
  if (!r || !flags || !here(r->device)) return MEDUSA_ERR_INVALID;
  return read_status(r->status, stream, flags);
}

medusa_status medusa_rope_apply(const medusa_rope* r, int dtype, int dh, int rows, const int32_t* pos,
                                const medusa_rope_rows* parts, int n_parts, int inverse, void* stream) {
  EntryScope scope("medusa_rope_apply");
  if (!r || !is_dtype(dtype) || rows < 0 || (rows > 0 && !pos) || !parts || n_parts < 1 || n_parts > kRopeParts)
    return MEDUSA_ERR_INVALID;
  if (dh < r->d.rot || !here(r->device)) return MEDUSA_ERR_INVALID;
  if (dh > 1024) return MEDUSA_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.t = table_of(r);
  a.pos = pos;
  a.rows = rows;
  a.dh = dh;
  a.n_parts = n_parts;
  a.inverse = inverse != 0;
  for (int i = 0; i < n_parts; ++i) {
    const medusa_rope_rows& p = parts[i];
    if ((rows > 0 && (!p.x || !p.y)) || p.heads < 1 || p.x_row < 0 || p.x_head < 0 || p.y_row < 0 || p.y_head < 0)
      return MEDUSA_ERR_INVALID;
    if (!aligned(p.x, elem(dtype)) || !aligned(p.y, elem(dtype))) return MEDUSA_ERR_INVALID;
    if (rows > 0 && p.x == p.y && (p.x_row != p.y_row || p.x_head != p.y_head)) return MEDUSA_ERR_INVALID;
    if (rows > 0 && !lie_apart(rows, p.y_row, p.heads, p.y_head, dh)) return MEDUSA_ERR_INVALID;
    if (p.heads > 65535 || a.heads + p.heads > 65535) return MEDUSA_ERR_UNSUPPORTED;
    a.part[i] = p;
    a.heads += p.heads;
  }
  if (rows == 0) return MEDUSA_OK;
  return done(launch_rope(a, dtype, S(stream)));
}

medusa_status medusa_cache_create(const medusa_cache_dims* dims, medusa_cache** out) {
  if (!out) return MEDUSA_ERR_INVALID;
  *out = nullptr;
  const medusa_status s = check_cache(dims);
  if (s != MEDUSA_OK) return s;
  medusa_cache* c = new (std::nothrow) medusa_cache();
  if (!c) return MEDUSA_ERR_CUDA;
  c->d = *dims;
  const size_t slots = dims->page_size > 0 ? (size_t)dims->num_pages * dims->page_size
                                           : (size_t)dims->B * dims->capacity;
  const size_t n = slots * dims->Hkv * dims->dh;
  c->pool_bytes = dims->format == MEDUSA_KV4 ? n / 16 * 9 : n * elem(dims->format);
  int sms = 0;
  bool ok = cudaGetDevice(&c->device) == cudaSuccess &&
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device) == cudaSuccess &&
            cudaMalloc(&c->status, sizeof(uint32_t)) == cudaSuccess &&
            cudaMemset(c->status, 0, sizeof(uint32_t)) == cudaSuccess &&
            cudaStreamSynchronize(nullptr) == cudaSuccess;   // before a call on any other stream
  if (!ok) {
    cudaGetLastError();
    medusa_cache_destroy(c);
    return MEDUSA_ERR_CUDA;
  }
  c->num_sms = sms;
  if (dims->format == MEDUSA_KV4)
    c->ws_bytes = kv4_workspace(dims->B, dims->Hq, dims->Hkv, dims->dh, dims->max_nodes, sms);
  *out = c;
  return MEDUSA_OK;
}

void medusa_cache_destroy(medusa_cache* c) {
  if (!c) return;
  if (c->status) cudaFree(c->status);
  delete c;
}

size_t medusa_cache_pool_bytes(const medusa_cache* c) { return c ? c->pool_bytes : 0; }
size_t medusa_cache_workspace_size(const medusa_cache* c) { return c ? c->ws_bytes : 0; }

medusa_status medusa_cache_get_status(const medusa_cache* c, void* stream, uint32_t* flags) {
  if (!c || !flags || !here(c->device)) return MEDUSA_ERR_INVALID;
  return read_status(c->status, stream, flags);
}

medusa_status medusa_cache_expire_wait_once(medusa_cache* c, unsigned long long ns) {
  if (!c || ns == 0 || ns > 10000000000ull) return MEDUSA_ERR_INVALID;
  if (c->d.format != MEDUSA_KV4) return MEDUSA_ERR_UNSUPPORTED;
  c->test_wait_ns.store(ns);
  return MEDUSA_OK;
}

medusa_status medusa_kv_append(const medusa_cache* c, const medusa_kv* kv, const medusa_kv_rows* rows,
                               const medusa_rope* rope, float k_scale, float v_scale, void* stream) {
  EntryScope scope("medusa_kv_append");
  if (!c || !here(c->device)) return MEDUSA_ERR_INVALID;
  AppendArgs a{};
  medusa_status s = check_kv(c, kv, true);
  if (s != MEDUSA_OK) return s;
  if ((s = check_scales(c, k_scale, v_scale)) != MEDUSA_OK) return s;
  if ((s = check_items(c, rows, &a.m)) != MEDUSA_OK) return s;
  if (rows->index && rows->index_rows < 1) return MEDUSA_ERR_INVALID;
  if (rope && (rope->device != c->device || rope->d.rot > c->d.dh)) return MEDUSA_ERR_INVALID;
  a.c = view_of(c, kv, k_scale, v_scale);
  a.k = rows->k;
  a.v = rows->v;
  a.k_row = rows->k_row;
  a.k_head = rows->k_head;
  a.v_row = rows->v_row;
  a.v_head = rows->v_head;
  a.index = rows->index;
  a.index_rows = rows->index_rows;
  a.pos = rope ? rows->pos : nullptr;
  a.turn = rope != nullptr;
  if (rope) a.t = table_of(rope);
  a.vec = vector_rows(rows);
  return done(launch_kv_append(a, rows->dtype, c->d.format, S(stream)));
}

medusa_status medusa_kv_read(const medusa_cache* c, const medusa_kv* kv, const medusa_kv_places* places,
                             float k_scale, float v_scale, void* stream) {
  EntryScope scope("medusa_kv_read");
  if (!c || !here(c->device)) return MEDUSA_ERR_INVALID;
  ReadArgs a{};
  medusa_status s = check_kv(c, kv, false);
  if (s != MEDUSA_OK) return s;
  if ((s = check_scales(c, k_scale, v_scale)) != MEDUSA_OK) return s;
  if ((s = check_items(c, places, &a.m)) != MEDUSA_OK) return s;
  if (!lie_apart(places->rows, places->k_row, c->d.Hkv, places->k_head, c->d.dh) ||
      !lie_apart(places->rows, places->v_row, c->d.Hkv, places->v_head, c->d.dh))
    return MEDUSA_ERR_INVALID;
  a.c = view_of(c, kv, k_scale, v_scale);
  a.k = places->k;
  a.v = places->v;
  a.k_row = places->k_row;
  a.k_head = places->k_head;
  a.v_row = places->v_row;
  a.v_head = places->v_head;
  a.first = places->first;
  a.vec = vector_rows(places);
  if (places->rows == 0) return MEDUSA_OK;
  return done(launch_kv_read(a, places->dtype, c->d.format, S(stream)));
}

medusa_status medusa_kv4_attention(const medusa_cache* c, const medusa_kv* kv, const medusa_kv4_query* q,
                                   void* ws, size_t ws_bytes, void* stream) {
  EntryScope scope("medusa_kv4_attention");
  if (!c || !q || !here(c->device)) return MEDUSA_ERR_INVALID;
  if (c->d.format != MEDUSA_KV4) return MEDUSA_ERR_UNSUPPORTED;
  medusa_status s = check_kv(c, kv, false);
  if (s != MEDUSA_OK) return s;
  if ((s = check_scales(c, q->k_scale, q->v_scale)) != MEDUSA_OK) return s;
  if (!q->q || !q->o || !is_dtype(q->dtype) || q->n1 < 1 || q->n1 > c->d.max_nodes) return MEDUSA_ERR_INVALID;
  if (!q->tree_k != !q->tree_v || (q->mask && !q->tree_k)) return MEDUSA_ERR_INVALID;
  if (!(q->scale >= 0 && q->scale <= 1e38f)) return MEDUSA_ERR_INVALID;        // times log2(e) it stays a float
  const long long n = 16 / (long long)elem(q->dtype);
  if (!aligned(q->q, 16) || !aligned(q->o, 16) || !aligned(q->tree_k, 16) || !aligned(q->tree_v, 16))
    return MEDUSA_ERR_INVALID;
  if (q->q_row < 0 || q->q_head < 0 || q->o_row < 0 || q->o_head < 0 || q->q_row % n || q->q_head % n ||
      q->o_row % n || q->o_head % n)
    return MEDUSA_ERR_INVALID;
  if (!lie_apart((long long)c->d.B * q->n1, q->o_row, c->d.Hq, q->o_head, c->d.dh)) return MEDUSA_ERR_INVALID;
  if (!ws || ws_bytes < c->ws_bytes || !aligned(ws, 256)) return MEDUSA_ERR_WORKSPACE;
  Kv4AttnArgs a{};
  a.c = view_of(c, kv, q->k_scale, q->v_scale);
  a.q = q->q;
  a.o = q->o;
  a.q_row = q->q_row;
  a.q_head = q->q_head;
  a.o_row = q->o_row;
  a.o_head = q->o_head;
  a.tk = q->tree_k;
  a.tv = q->tree_v;
  a.mask = q->mask;
  a.n1 = q->n1;
  a.Hq = c->d.Hq;
  a.G = c->d.Hq / c->d.Hkv;
  a.scale = q->scale > 0 ? q->scale : 1.0f / std::sqrt((float)c->d.dh);
  a.factor_m = (float)(2.0 * std::frexp((double)a.scale * q->k_scale * 1.4426950408889634, &a.factor_e));
  --a.factor_e;
  if (a.factor_m >= 2.0f) {                       // rounded up
    a.factor_m = 1.0f;
    ++a.factor_e;
  }
  if (c->test_wait_ns.load(std::memory_order_relaxed)) a.test_wait_ns = c->test_wait_ns.exchange(0);
  return done(launch_kv4_attention(a, q->dtype, ws, c->num_sms, S(stream)));
}

}  // extern "C"
