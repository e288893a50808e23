// kv_api.cu -- host side of the paged 8-bit cache: argument checks and launches
// on the caller's streams.  The cache's memory is the caller's; a handle holds
// its geometry, the attention's workspace and an error word.
#include <atomic>
#include <new>

#include "device_scope.h"
#include "kv_internal.h"
#include "sgd_internal.h"

using namespace sgd;

struct sgd_kv {
  sgd_kv_config cfg;
  int device = 0;
  int sms = 0;
  uint32_t *d_err = nullptr;
  unsigned char *d_work = nullptr;
  size_t work_bytes = 0;
  std::atomic<uint64_t> launches{0};
};

namespace {

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool valid_type(int t) { return t == SGD_F32 || t == SGD_F16 || t == SGD_BF16; }
int type_size(int t) { return t == SGD_F32 ? 4 : 2; }

int validate(const sgd_kv_config &c) {
  if (c.num_pages < 1 || c.kv_heads < 1 || c.kv_heads > 1024 || c.max_batch < 1) return SGD_EINVAL;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128) return SGD_EINVAL;
  if (c.head_dim != 64 && c.head_dim != 128) return SGD_EINVAL;
  if (c.q_heads < c.kv_heads || c.q_heads % c.kv_heads != 0 || c.q_heads / c.kv_heads > 64) return SGD_EINVAL;
  if (c.max_pages_per_row < 1 || (int64_t)c.max_pages_per_row * c.page_size > (1LL << 30)) return SGD_EINVAL;
  if ((int64_t)c.num_pages * c.kv_heads * c.page_size > 0x7fffffffLL) return SGD_EINVAL;
  return SGD_OK;
}

int view(const sgd_kv *x, const sgd_kv_layer *l, KvView *v) {
  if (!l || !l->k || !l->v || !l->k_scale || !l->v_scale) return SGD_EINVAL;
  if (!aligned(l->k, 16) || !aligned(l->v, 16) || !aligned(l->k_scale, 4) || !aligned(l->v_scale, 4)) return SGD_EINVAL;
  *v = KvView{static_cast<uint8_t *>(l->k), static_cast<uint8_t *>(l->v), l->k_scale, l->v_scale,
              x->cfg.num_pages, x->cfg.kv_heads, x->cfg.page_size, x->cfg.head_dim, 0};
  while (1 << v->page_bits < v->page) ++v->page_bits;
  return SGD_OK;
}

int rows(const sgd_kv *x, const int32_t *table, const int32_t *seq_lens, const int32_t *q_start, int32_t B,
         int32_t N, KvRows *r) {
  if (B < 0 || B > x->cfg.max_batch || N < 0) return SGD_EINVAL;
  if (B > 0 && N > 0 && (!table || !seq_lens || !q_start)) return SGD_EINVAL;
  *r = KvRows{table, q_start, seq_lens, B, N, x->cfg.max_pages_per_row};
  return SGD_OK;
}

int check_cuda(cudaError_t e) { return e == cudaSuccess ? SGD_OK : SGD_ECUDA; }

}  // namespace

extern "C" {

int sgd_kv_create(const sgd_kv_config *cfg, int device, sgd_kv **out) {
  if (!cfg || !out) return SGD_EINVAL;
  *out = nullptr;
  const int v = validate(*cfg);
  if (v != SGD_OK) return v;
  const DeviceScope on(device);
  if (!on.ok()) return SGD_ECUDA;
  sgd_kv *x = new (std::nothrow) sgd_kv;
  if (!x) return SGD_ENOMEM;
  x->cfg = *cfg;
  x->device = device;
  x->work_bytes = kv_attend_workspace();
  cudaError_t e = cudaMalloc((void **)&x->d_err, 4);
  if (e == cudaSuccess) e = cudaMemset(x->d_err, 0, 4);
  if (e == cudaSuccess) e = cudaMalloc((void **)&x->d_work, x->work_bytes);
  if (e == cudaSuccess) e = cudaMemset(x->d_work, 0, x->work_bytes);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&x->sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = kv_attend_set_limits();
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(x->d_err);
    cudaFree(x->d_work);
    delete x;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? SGD_ENOMEM : SGD_ECUDA;
  }
  *out = x;
  return SGD_OK;
}

int sgd_kv_destroy(sgd_kv *x) {
  if (!x) return SGD_EINVAL;
  const DeviceScope on(x->device);
  cudaDeviceSynchronize();
  cudaFree(x->d_err);
  cudaFree(x->d_work);
  delete x;
  return SGD_OK;
}

int sgd_kv_write(sgd_kv *x, const sgd_kv_layer *layer, const void *k, const void *v, int32_t dtype,
                 int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                 int64_t v_head_stride, const int32_t *block_table, const int32_t *seq_lens,
                 const int32_t *q_start, int32_t B, int32_t N, void *stream) {
  if (!x || !valid_type(dtype)) return SGD_EINVAL;
  KvWriteArgs a{};
  int s = rows(x, block_table, seq_lens, q_start, B, N, &a.r);
  if (s != SGD_OK) return s;
  if (B == 0 || N == 0) return SGD_OK;
  s = view(x, layer, &a.c);
  if (s != SGD_OK) return s;
  if (!k || !v || !aligned(k, type_size(dtype)) || !aligned(v, type_size(dtype))) return SGD_EINVAL;
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0) return SGD_EINVAL;
  a.k = k;
  a.v = v;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  const int64_t per = 16 / type_size(dtype);
  a.vec = aligned(k, 16) && aligned(v, 16) && k_token_stride % per == 0 && k_head_stride % per == 0 &&
          v_token_stride % per == 0 && v_head_stride % per == 0;
  a.err = x->d_err;
  const DeviceScope on(x->device);
  if (!on.ok()) return SGD_ECUDA;
  x->launches++;
  return check_cuda(launch_kv_write(a, dtype, (cudaStream_t)stream));
}

int sgd_kv_read(sgd_kv *x, const sgd_kv_layer *layer, const int32_t *block_table, const int32_t *from,
                const int32_t *out_start, int32_t B, int32_t N, void *k, void *v, int32_t dtype,
                void *stream) {
  if (!x || !valid_type(dtype)) return SGD_EINVAL;
  if (B < 0 || B > x->cfg.max_batch || N < 0) return SGD_EINVAL;
  if (B == 0 || N == 0) return SGD_OK;
  KvReadArgs a{};
  const int s = view(x, layer, &a.c);
  if (s != SGD_OK) return s;
  if (!block_table || !from || !out_start || !k || !v || !aligned(k, 16) || !aligned(v, 16)) return SGD_EINVAL;
  a.table = block_table;
  a.from = from;
  a.out_start = out_start;
  a.B = B;
  a.N = N;
  a.max_pages = x->cfg.max_pages_per_row;
  a.k = k;
  a.v = v;
  a.err = x->d_err;
  const DeviceScope on(x->device);
  if (!on.ok()) return SGD_ECUDA;
  x->launches++;
  return check_cuda(launch_kv_read(a, dtype, (cudaStream_t)stream));
}

int sgd_kv_attend(sgd_kv *x, const sgd_kv_layer *layer, const void *q, int32_t dtype,
                  int64_t q_token_stride, int64_t q_head_stride, const int32_t *block_table,
                  const int32_t *seq_lens, const int32_t *q_start, int32_t B, int32_t N, int32_t max_q,
                  float scale, int32_t window, int32_t sinks, void *out, void *stream) {
  if (!x || (dtype != SGD_F16 && dtype != SGD_BF16)) return SGD_EINVAL;
  KvAttendArgs a{};
  int s = rows(x, block_table, seq_lens, q_start, B, N, &a.r);
  if (s != SGD_OK) return s;
  if (window < 0 || sinks < 0 || !(scale == scale)) return SGD_EINVAL;
  if (B == 0 || N == 0) return SGD_OK;
  if (max_q < 1) return SGD_EINVAL;
  s = view(x, layer, &a.c);
  if (s != SGD_OK) return s;
  if (!q || !out || !aligned(q, 2) || !aligned(out, 16)) return SGD_EINVAL;
  if (q_token_stride < 0 || q_head_stride < 0) return SGD_EINVAL;
  a.q = q;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.q_vec = aligned(q, 16) && q_token_stride % 8 == 0 && q_head_stride % 8 == 0;
  a.out = out;
  a.q_heads = x->cfg.q_heads;
  a.group = x->cfg.q_heads / x->cfg.kv_heads;
  a.max_q = max_q < N ? max_q : N;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.sms = x->sms;
  a.work = x->d_work;
  a.err = x->d_err;
  const DeviceScope on(x->device);
  if (!on.ok()) return SGD_ECUDA;
  int launches = 0;
  const cudaError_t e = launch_kv_attend(a, dtype, (cudaStream_t)stream, &launches);
  x->launches += launches;
  return check_cuda(e);
}

int sgd_kv_get_error(sgd_kv *x, uint32_t *flags, int clear) {
  if (!x || !flags) return SGD_EINVAL;
  const DeviceScope on(x->device);
  if (!on.ok()) return SGD_ECUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return SGD_ECUDA;
  if (cudaMemcpy(flags, x->d_err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return SGD_ECUDA;
  if (clear && cudaMemset(x->d_err, 0, 4) != cudaSuccess) return SGD_ECUDA;
  return SGD_OK;
}

int sgd_kv_memory(sgd_kv *x, int64_t *device_bytes) {
  if (!x || !device_bytes) return SGD_EINVAL;
  *device_bytes = (int64_t)x->work_bytes + 4;
  return SGD_OK;
}

int sgd_kv_launch_count(sgd_kv *x, uint64_t *count) {
  if (!x || !count) return SGD_EINVAL;
  *count = x->launches.load();
  return SGD_OK;
}

}  // extern "C"
