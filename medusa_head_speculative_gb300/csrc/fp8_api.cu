// C ABI of the 8-bit projections: handles, checks and launches.  The rules every call keeps to are in
// include/medusa.h.
#include <cuda_runtime.h>

#include <atomic>
#include <new>

#include "api.h"
#include "common.cuh"
#include "fp8.h"
#include "launch.cuh"

using namespace medusa;

struct medusa_fp8 {
  medusa_fp8_dims d;
  uint32_t* status = nullptr;
  int device = 0, num_sms = 152, kb = 0;
  size_t codes_bytes = 0, scales_bytes = 0, ws_bytes = 0;
  mutable std::atomic<unsigned long long> test_wait_ns{0};
};

namespace {

size_t round_up(size_t x, size_t n) { return (x + n - 1) / n * n; }

medusa_status check_dims(const medusa_fp8_dims* d) {
  if (!d || d->n < 1 || d->k < 16 || d->k % 16 != 0 || d->max_rows < 1 || (d->gated != 0 && d->gated != 1))
    return MEDUSA_ERR_INVALID;
  const double most = 274877906944.0;                       // 2^38 elements
  if (d->n > (1 << 24) || d->k > (1 << 20) || d->max_rows > (1 << 24) || (double)d->n * d->k > most ||
      (double)d->max_rows * d->k > most || (double)d->max_rows * d->n > most)
    return MEDUSA_ERR_UNSUPPORTED;
  return MEDUSA_OK;
}

// rows of a call that rounds or reads
bool rows_fit(const medusa_fp8* h, int rows, int block) {
  return block == 1 ? rows >= 0 && rows <= h->d.max_rows : block == kFp8Group && rows == h->d.n;
}

}  // namespace

extern "C" {

medusa_status medusa_fp8_create(const medusa_fp8_dims* dims, medusa_fp8** out) {
  if (!out) return MEDUSA_ERR_INVALID;
  *out = nullptr;
  const medusa_status s = check_dims(dims);
  if (s != MEDUSA_OK) return s;
  medusa_fp8* h = new (std::nothrow) medusa_fp8();
  if (!h) return MEDUSA_ERR_CUDA;
  h->d = *dims;
  h->kb = (dims->k + kFp8Group - 1) / kFp8Group;
  bool ok = cudaGetDevice(&h->device) == cudaSuccess &&
            cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) == cudaSuccess &&
            cudaMalloc(&h->status, sizeof(uint32_t)) == cudaSuccess &&
            cudaMemset(h->status, 0, sizeof(uint32_t)) == cudaSuccess &&
            cudaStreamSynchronize(nullptr) == cudaSuccess;   // before a call on any other stream
  if (!ok) {
    cudaGetLastError();
    medusa_fp8_destroy(h);
    return MEDUSA_ERR_CUDA;
  }
  h->codes_bytes = round_up((size_t)dims->max_rows * dims->k, 256);
  h->scales_bytes = round_up((size_t)dims->max_rows * h->kb * sizeof(float), 256);
  h->ws_bytes = h->codes_bytes + h->scales_bytes +
                fp8_linear_partials(dims->max_rows, dims->n, h->kb, h->num_sms);
  *out = h;
  return MEDUSA_OK;
}

void medusa_fp8_destroy(medusa_fp8* h) {
  if (!h) return;
  if (h->status) cudaFree(h->status);
  delete h;
}

size_t medusa_fp8_workspace_size(const medusa_fp8* h) { return h ? h->ws_bytes : 0; }

medusa_status medusa_fp8_get_status(const medusa_fp8* h, void* stream, uint32_t* flags) {
  if (!h || !flags || !here(h->device)) return MEDUSA_ERR_INVALID;
  return read_status(h->status, stream, flags);
}

medusa_status medusa_fp8_tiles(const medusa_fp8* h, int rows, int gated, int* columns, int* whole, int* shared) {
  if (!h || !columns || !whole || !shared || rows < 1 || rows > h->d.max_rows || (gated != 0 && gated != h->d.gated))
    return MEDUSA_ERR_INVALID;
  const Fp8Tiles t = fp8_linear_tiles(rows, h->d.n, h->kb, gated != 0, h->num_sms);
  *columns = gated ? t.columns / 2 : t.columns;
  *whole = t.whole;
  *shared = t.shared;
  return MEDUSA_OK;
}

medusa_status medusa_fp8_expire_wait_once(medusa_fp8* h, unsigned long long ns) {
  if (!h || ns == 0 || ns > 10000000000ull) return MEDUSA_ERR_INVALID;
  h->test_wait_ns.store(ns);
  return MEDUSA_OK;
}

medusa_status medusa_fp8_round(const medusa_fp8* h, const void* x, int dtype, int rows, long long x_row,
                               void* codes, float* scales, int block, void* stream) {
  EntryScope scope("medusa_fp8_round");
  if (!h || !here(h->device) || !is_dtype(dtype) || !rows_fit(h, rows, block) || x_row < 0) return MEDUSA_ERR_INVALID;
  if (rows == 0) return MEDUSA_OK;
  if (!x || !codes || !scales || !aligned(x, elem(dtype)) || !aligned(codes, 4) || !aligned(scales, 4))
    return MEDUSA_ERR_INVALID;
  Fp8RoundArgs a{};
  a.x = x;
  a.x_row = x_row;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.rows = rows;
  a.k = h->d.k;
  a.kb = h->kb;
  a.vec = aligned(x, 4 * elem(dtype)) && x_row % 4 == 0;
  a.status = h->status;
  return done(launch_fp8_round(a, dtype, block, h->num_sms, S(stream)));
}

medusa_status medusa_fp8_read(const medusa_fp8* h, const void* codes, const float* scales, int rows, int block,
                              void* y, int dtype, long long y_row, void* stream) {
  EntryScope scope("medusa_fp8_read");
  if (!h || !here(h->device) || !is_dtype(dtype) || !rows_fit(h, rows, block)) return MEDUSA_ERR_INVALID;
  if (rows == 0) return MEDUSA_OK;
  if (!y || !codes || !scales || !aligned(y, elem(dtype)) || !aligned(codes, 4) || !aligned(scales, 4))
    return MEDUSA_ERR_INVALID;
  if (y_row < 0 || (rows > 1 && y_row < h->d.k)) return MEDUSA_ERR_INVALID;
  Fp8ReadArgs a{};
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = scales;
  a.y = y;
  a.y_row = y_row;
  a.rows = rows;
  a.k = h->d.k;
  a.kb = h->kb;
  a.block = block;
  a.vec = aligned(y, 4 * elem(dtype)) && y_row % 4 == 0;
  return done(launch_fp8_read(a, dtype, h->num_sms, S(stream)));
}

medusa_status medusa_fp8_linear(const medusa_fp8* h, const medusa_fp8_product* p, void* ws, size_t ws_bytes,
                                void* stream) {
  EntryScope scope("medusa_fp8_linear");
  if (!h || !p || !here(h->device)) return MEDUSA_ERR_INVALID;
  const bool codes = p->x_dtype == MEDUSA_E4M3;
  if ((!codes && !is_dtype(p->x_dtype)) || !is_dtype(p->y_dtype)) return MEDUSA_ERR_INVALID;
  if (p->rows < 0 || p->rows > h->d.max_rows || p->x_row < 0 || p->add_row < 0 || p->y_row < 0)
    return MEDUSA_ERR_INVALID;
  if (!p->w || !p->w_scales || !aligned(p->w, 16) || !aligned(p->w_scales, 4)) return MEDUSA_ERR_INVALID;
  if (!p->up != !p->up_scales || (p->up && (!h->d.gated || p->add)) || !aligned(p->up, 16) || !aligned(p->up_scales, 4))
    return MEDUSA_ERR_INVALID;
  if (!ws || ws_bytes < h->ws_bytes || !aligned(ws, 256)) return MEDUSA_ERR_WORKSPACE;
  if (p->rows == 0) return MEDUSA_OK;
  if (codes != (p->x_scales != nullptr)) return MEDUSA_ERR_INVALID;
  if (!p->x || !p->y || !aligned(p->x, codes ? 16 : elem(p->x_dtype)) || !aligned(p->x_scales, 4) ||
      !aligned(p->y, elem(p->y_dtype)) || !aligned(p->add, elem(p->y_dtype)))
    return MEDUSA_ERR_INVALID;
  if (p->rows > 1 && (p->y_row < h->d.n || (codes && (p->x_row < h->d.k || p->x_row % 16 != 0))))
    return MEDUSA_ERR_INVALID;
  if (p->add == p->y && p->rows > 1 && p->add_row != p->y_row) return MEDUSA_ERR_INVALID;
  uint8_t* base = static_cast<uint8_t*>(ws);
  Fp8LinearArgs a{};
  a.rows = p->rows;
  a.n = h->d.n;
  a.k = h->d.k;
  a.kb = h->kb;
  a.w[0] = static_cast<const uint8_t*>(p->w);
  a.ws[0] = p->w_scales;
  a.w[1] = static_cast<const uint8_t*>(p->up);
  a.ws[1] = p->up_scales;
  a.add = p->add;
  a.add_row = p->add_row;
  a.y = p->y;
  a.y_row = p->y_row;
  a.status = h->status;
  a.x = static_cast<const uint8_t*>(p->x);
  a.xs = p->x_scales;
  a.x_row = p->rows > 1 ? p->x_row : (long)round_up(h->d.k, 16);
  if (!codes) {
    Fp8RoundArgs r{};
    r.x = p->x;
    r.x_row = p->x_row;
    r.codes = base;
    r.scales = reinterpret_cast<float*>(base + h->codes_bytes);
    r.rows = p->rows;
    r.k = h->d.k;
    r.kb = h->kb;
    r.vec = aligned(p->x, 4 * elem(p->x_dtype)) && p->x_row % 4 == 0;
    r.status = h->status;
    const cudaError_t e = launch_fp8_round(r, p->x_dtype, 1, h->num_sms, S(stream));
    if (e != cudaSuccess) return MEDUSA_ERR_CUDA;
    a.x = base;
    a.xs = r.scales;
    a.x_row = h->d.k;
  }
  if (h->test_wait_ns.load(std::memory_order_relaxed)) a.test_wait_ns = h->test_wait_ns.exchange(0);
  return done(launch_fp8_linear(a, p->y_dtype, base + h->codes_bytes + h->scales_bytes, h->num_sms, S(stream)));
}

}  // extern "C"
