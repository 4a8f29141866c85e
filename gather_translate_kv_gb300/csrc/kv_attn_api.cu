// The C ABI of include/kv_attention.h: argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "kv_attn_launch.h"
#include "kv_pool_internal.h"

namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launched(cudaError_t e) {
  if (e == cudaSuccess) return KV_OK;
  cudaGetLastError();  // reported once, here
  return KV_ERR_CUDA;
}

cudaStream_t as_stream(kv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

int type_size(int32_t type) {
  return type == KV_TYPE_BF16 || type == KV_TYPE_F16 ? 2 : type == KV_TYPE_F32 ? 4 : 0;
}

// Pool, layer and batch; fills *b. A batch without rows or sequences is KV_OK with b->n_rows = 0.
int enter(const kv_pool_t* pool, int32_t layer, const kv_batch* in, gtkv::Batch* b) {
  if (pool == nullptr || in == nullptr) return KV_ERR_INVALID;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return KV_ERR_CUDA;
  }
  if (dev != pool->device) return KV_ERR_DEVICE;
  if (pool->desc.latent_only || layer < 0 || layer >= pool->desc.layer_num) return KV_ERR_INVALID;
  if (in->n_seqs < 0 || in->max_pages < 0 || in->n_rows < 0 || in->reserved != 0 ||
      (in->kernel_facing != 0 && in->kernel_facing != 1))
    return KV_ERR_INVALID;
  if (static_cast<int64_t>(in->n_seqs) * in->max_pages >= (int64_t(1) << 31) ||
      static_cast<int64_t>(in->max_pages) * pool->desc.page_size >= (int64_t(1) << 31))
    return KV_ERR_INVALID;
  *b = gtkv::Batch{in->table_dev, in->seq_start_dev, in->seq_len_dev, in->cu_dev,
                   in->n_rows,    in->n_seqs,        in->max_pages,   in->kernel_facing};
  if (in->n_rows == 0 || in->n_seqs == 0) {
    b->n_rows = 0;
    return KV_OK;
  }
  if (in->seq_len_dev == nullptr || in->cu_dev == nullptr || (in->table_dev == nullptr && in->max_pages > 0))
    return KV_ERR_INVALID;
  if (!aligned(in->table_dev, 4) || !aligned(in->seq_start_dev, 4) || !aligned(in->seq_len_dev, 4) ||
      !aligned(in->cu_dev, 8))
    return KV_ERR_ALIGN;
  return KV_OK;
}

gtkv::Kind kind_of(const kv_pool_t* pool) { return gtkv::kind_of(pool->desc); }

// The scale buffer goes with 8-bit pools and with them only.
int check_scales(const kv_pool_t* pool, const float* scales) {
  if ((kind_of(pool) == gtkv::Kind::kE4M3) != (scales != nullptr)) return KV_ERR_INVALID;
  return aligned(scales, 4) ? KV_OK : KV_ERR_ALIGN;
}

int check_rotary(const kv_pool_t* pool, const kv_rotary* r) {
  if (r == nullptr) return KV_OK;
  if (r->reserved != 0 || r->rotary_dim < 0 || r->rotary_dim % 2 != 0 || r->rotary_dim > pool->desc.head_dim ||
      (r->interleaved != 0 && r->interleaved != 1) || r->n_axes < 1 || r->n_axes > 4 || r->n_positions < 0)
    return KV_ERR_INVALID;
  int64_t pairs = 0;
  for (int a = 0; a < r->n_axes; ++a) {
    if (r->axis_pairs[a] < 0) return KV_ERR_INVALID;
    pairs += r->axis_pairs[a];
  }
  if (pairs != r->rotary_dim / 2) return KV_ERR_INVALID;
  if (r->rotary_dim > 0 && r->n_positions > 0 && r->cos_sin_dev == nullptr) return KV_ERR_INVALID;
  return aligned(r->cos_sin_dev, 4) && aligned(r->positions_dev, 4) ? KV_OK : KV_ERR_ALIGN;
}

// What the two attention calls check alike; fills *b and *a. Nothing to do: KV_OK with b->n_rows = 0.
int enter_attend(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, int32_t type, const void* q_dev,
                 int64_t q_stride, int32_t q_heads, void* out_dev, float* lse_dev, float scale, int32_t window,
                 int32_t sinks, const float* scales_dev, const void* workspace_dev, int64_t workspace_bytes,
                 int (*need_of)(const kv_pool_t*, int32_t, int32_t, int64_t, int64_t*), gtkv::Batch* b,
                 gtkv::AttendArgs* a) {
  int rc = enter(pool, layer, batch, b);
  if (rc != KV_OK) return rc;
  const int32_t H = pool->desc.head_num, D = pool->desc.head_dim, it = pool->desc.itemsize;
  if ((type != KV_TYPE_BF16 && type != KV_TYPE_F16) || (it != 1 && it != 2)) return KV_ERR_INVALID;
  if ((rc = check_scales(pool, scales_dev)) != KV_OK) return rc;
  if (q_heads < 1 || q_heads > (1 << 16) || q_heads % H != 0 || D > 256 || !isfinite(scale) || window < 0 || sinks < 0)
    return KV_ERR_INVALID;
  int64_t need = 0;
  if ((rc = need_of(pool, q_heads, batch->n_seqs, batch->n_rows, &need)) != KV_OK) return rc;
  if (b->n_rows == 0) return KV_OK;
  if (q_dev == nullptr || out_dev == nullptr || workspace_dev == nullptr || workspace_bytes < need)
    return KV_ERR_INVALID;
  if (b->n_rows > 1 && q_stride < static_cast<int64_t>(q_heads) * D) return KV_ERR_INVALID;
  if (!aligned(q_dev, 2) || !aligned(out_dev, 2) || !aligned(lse_dev, 4) || !aligned(workspace_dev, 16))
    return KV_ERR_ALIGN;
  *a = gtkv::AttendArgs{q_dev, out_dev, lse_dev, scales_dev, q_stride, scale * 1.4426950408889634f, window, sinks,
                        H,     q_heads, D,       q_heads / H, layer,   type, q_heads / H};
  return KV_OK;
}

// Sets up the kernels for shared prefixes, with the pool's device current, once a pool: kv_pool_create leaves them out,
// since loading them takes a process 1 to 1.5 ms for each kind of pool. It may be called while a stream is captured.
int ready_shared(const kv_pool_t* pool) {
  if (pool->shared_ready.load(std::memory_order_acquire)) return KV_OK;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e == cudaSuccess) {
    e = gtkv::prepare_attend(pool->desc, true);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) e = back;
  }
  if (e == cudaSuccess) pool->shared_ready.store(true, std::memory_order_release);
  return launched(e);
}

}  // namespace

extern "C" {

int kv_scale_bytes(const kv_pool_t* pool, int64_t* bytes) {
  if (pool == nullptr || bytes == nullptr || pool->desc.latent_only || kind_of(pool) != gtkv::Kind::kE4M3)
    return KV_ERR_INVALID;
  *bytes = 4 * pool->desc.num_pages * pool->lay.blocks * pool->desc.head_num;
  return KV_OK;
}

int kv_append_layer(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, int32_t type, const void* k_dev,
                    int64_t k_stride, const void* v_dev, int64_t v_stride, const kv_rotary* rotary, const void* q_dev,
                    int64_t q_stride, int32_t q_heads, void* q_out_dev, float* scales_dev, kv_stream_t stream) {
  Range nvtx("kv_append_layer");
  gtkv::Batch b;
  int rc = enter(pool, layer, batch, &b);
  if (rc != KV_OK) return rc;
  const int size = type_size(type);
  const int32_t H = pool->desc.head_num, D = pool->desc.head_dim, it = pool->desc.itemsize;
  if (size == 0 || (it != 1 && it != size)) return KV_ERR_INVALID;
  if ((rc = check_scales(pool, scales_dev)) != KV_OK) return rc;
  if ((rc = check_rotary(pool, rotary)) != KV_OK) return rc;
  if (q_heads < 0 || q_heads > (1 << 16) || (q_dev == nullptr) != (q_heads == 0) || (q_heads > 0 && q_out_dev == nullptr))
    return KV_ERR_INVALID;
  const int64_t row = static_cast<int64_t>(H) * D, q_row = static_cast<int64_t>(q_heads) * D;
  if (b.n_rows == 0) return KV_OK;
  if (k_dev == nullptr || v_dev == nullptr) return KV_ERR_INVALID;
  if (b.n_rows > 1 && (k_stride < row || v_stride < row || (q_heads > 0 && q_stride < q_row))) return KV_ERR_INVALID;
  if (q_dev != nullptr && q_dev == q_out_dev && b.n_rows > 1 && q_stride != q_row) return KV_ERR_INVALID;
  if (!aligned(k_dev, size) || !aligned(v_dev, size) || !aligned(q_dev, size) || !aligned(q_out_dev, size))
    return KV_ERR_ALIGN;
  return launched(gtkv::launch_append(pool->dev, b, layer, type, kind_of(pool), H, D, k_dev, k_stride, v_dev, v_stride,
                                      rotary, q_dev, q_stride, q_heads, q_out_dev, scales_dev, pool->sm_count,
                                      as_stream(stream)));
}

int kv_attend_workspace_bytes(const kv_pool_t* pool, int32_t q_heads, int32_t n_seqs, int64_t n_rows,
                              int64_t* bytes) {
  if (pool == nullptr || bytes == nullptr || n_seqs < 0 || n_rows < 0 || q_heads < 1 || q_heads > (1 << 16) ||
      pool->desc.latent_only || q_heads % pool->desc.head_num != 0)
    return KV_ERR_INVALID;
  *bytes = gtkv::attend_workspace_bytes(pool->desc.head_num, q_heads, pool->desc.head_dim, n_seqs, n_rows,
                                        pool->sm_count);
  return KV_OK;
}

int kv_attend_layer(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, int32_t type, const void* q_dev,
                    int64_t q_stride, int32_t q_heads, void* out_dev, float* lse_dev, float scale, int32_t window,
                    int32_t sinks, const float* scales_dev, void* workspace_dev, int64_t workspace_bytes,
                    kv_stream_t stream) {
  Range nvtx("kv_attend_layer");
  gtkv::Batch b;
  gtkv::AttendArgs a;
  const int rc = enter_attend(pool, layer, batch, type, q_dev, q_stride, q_heads, out_dev, lse_dev, scale, window, sinks,
                              scales_dev, workspace_dev, workspace_bytes, kv_attend_workspace_bytes, &b, &a);
  if (rc != KV_OK || b.n_rows == 0) return rc;
  return launched(gtkv::launch_attend(pool->dev, b, a, kind_of(pool), {}, workspace_dev, pool->sm_count, as_stream(stream)));
}

int kv_attend_shared_workspace_bytes(const kv_pool_t* pool, int32_t q_heads, int32_t n_seqs, int64_t n_rows,
                                     int64_t* bytes) {
  const int rc = kv_attend_workspace_bytes(pool, q_heads, n_seqs, n_rows, bytes);
  if (rc != KV_OK) return rc;
  if (n_rows > (int64_t(1) << 36)) return KV_ERR_INVALID;  // 4 * n_rows * q_heads * (head_dim + 2) stays below 2^63
  // a program asks before its first call, which then finds its kernels (asked on another device, it sets them up)
  int dev = -1;
  if (!pool->shared_ready.load(std::memory_order_acquire) && cudaGetDevice(&dev) == cudaSuccess && dev == pool->device)
    ready_shared(pool);
  *bytes = gtkv::attend_shared_workspace_bytes(q_heads, pool->desc.head_dim, n_seqs, n_rows, pool->sm_count);
  return KV_OK;
}

int kv_attend_shared_layer(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, const kv_prefix_groups* groups,
                           int32_t type, const void* q_dev, int64_t q_stride, int32_t q_heads, void* out_dev,
                           float* lse_dev, float scale, const float* scales_dev, void* workspace_dev,
                           int64_t workspace_bytes, kv_stream_t stream) {
  Range nvtx("kv_attend_shared_layer");
  gtkv::Batch b;
  gtkv::AttendArgs a;
  if (groups == nullptr || groups->n_groups < 0 || groups->reserved != 0) return KV_ERR_INVALID;
  int rc = enter_attend(pool, layer, batch, type, q_dev, q_stride, q_heads, out_dev, lse_dev, scale, 0, 0, scales_dev,
                        workspace_dev, workspace_bytes, kv_attend_shared_workspace_bytes, &b, &a);
  if (rc != KV_OK || b.n_rows == 0) return rc;
  if (groups->n_groups < 1 || groups->group_dev == nullptr || groups->prefix_len_dev == nullptr) return KV_ERR_INVALID;
  if (!aligned(groups->group_dev, 4) || !aligned(groups->prefix_len_dev, 4)) return KV_ERR_ALIGN;
  if ((rc = ready_shared(pool)) != KV_OK) return rc;
  return launched(gtkv::launch_attend_shared(pool->dev, b, a, kind_of(pool), gtkv::Groups{groups->group_dev, groups->n_groups},
                                             groups->prefix_len_dev, workspace_dev, pool->sm_count, as_stream(stream)));
}

int kv_gather_layer_scaled(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, const float* scales_dev,
                           int32_t type, void* out_k_dev, void* out_v_dev, kv_stream_t stream) {
  Range nvtx("kv_gather_layer_scaled");
  gtkv::Batch b;
  int rc = enter(pool, layer, batch, &b);
  if (rc != KV_OK) return rc;
  const gtkv::Kind kind = kind_of(pool);
  if (type_size(type) == 0 || kind == gtkv::Kind::kElements) return KV_ERR_INVALID;
  if ((rc = check_scales(pool, scales_dev)) != KV_OK) return rc;
  if (b.n_rows == 0) return KV_OK;
  if (out_k_dev == nullptr || out_v_dev == nullptr) return KV_ERR_INVALID;
  if (!aligned(out_k_dev, 16) || !aligned(out_v_dev, 16)) return KV_ERR_ALIGN;
  if (kind == gtkv::Kind::kE2M1)
    return launched(gtkv::launch_gather4(pool->dev, b, layer, pool->desc.head_num, pool->desc.head_dim, type, out_k_dev,
                                         out_v_dev, as_stream(stream)));
  return launched(gtkv::launch_gather_scaled(pool->dev, b, layer, pool->desc.head_num, pool->desc.head_dim, scales_dev,
                                             type, out_k_dev, out_v_dev, as_stream(stream)));
}

}  // extern "C"
