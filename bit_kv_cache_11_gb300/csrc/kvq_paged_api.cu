// kvq_paged_api.cu — the paged caches' part of the C ABI (include/kvq.h):
// validation, tensor maps, workspace layout and launches.  Nothing is kept
// between calls but the driver entry point, each kernel's shared-memory opt-in
// and the wait limit that a test may have set.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <mutex>

#include "kvq.h"
#include "kvq_paged4.cuh"

namespace kvq {
void count_launches(uint64_t n);

cudaError_t allow_smem(const void* fn, int bytes) {
  struct Entry {
    const void* fn;
    int device;
  };
  static std::mutex mu;
  static Entry done[256];
  static int n_done = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_done; ++i)
    if (done[i].fn == fn && done[i].device == dev) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && n_done < 256) done[n_done++] = {fn, dev};
  return e;
}
}  // namespace kvq

using namespace kvq;

namespace {

std::atomic<uint32_t> g_wait_limit{UINT32_MAX};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dev_ptr(const void* p, uintptr_t a) { return p != nullptr && aligned(p, a); }

// Whether two arrays of 32-bit numbers share an element.
bool overlap(const int* a, size_t n_a, const int* b, size_t n_b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * n_b && y < x + 4 * n_a;
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }

kvq_status check_pool(const kvq_paged_pool* c) {
  if (c == nullptr || c->n_pages < 1 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1)
    return KVQ_ERR_INVALID_ARG;
  if (!page_size_ok(c->page_size) || (c->head_dim != 64 && c->head_dim != 128))
    return KVQ_ERR_UNSUPPORTED;
  // rows of a pool are tensor-map coordinates, slots are 32-bit
  if (static_cast<long long>(c->n_pages) * c->n_kv_heads > INT_MAX / c->page_size)
    return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

bool pool_pointers(const kvq_paged_pool* c) {
  return dev_ptr(c->k_pages, 16) && dev_ptr(c->v_pages, 16) && dev_ptr(c->k_scale, 4) &&
         dev_ptr(c->v_scale, 4);
}

// A 4-bit pool's metadata is copied in bulk.
bool meta_pointers(const kvq_paged_pool* c) { return dev_ptr(c->k_scale, 16) && dev_ptr(c->v_scale, 16); }

bool dtype_ok(int dtype) { return dtype == KVQ_DTYPE_FP16 || dtype == KVQ_DTYPE_BF16; }

// Rows of `heads` heads at a stride: the stride holds them and keeps rows
// 16-byte aligned.
bool stride_ok(long long stride, int heads, int D) {
  return stride >= static_cast<long long>(heads) * D && stride % 8 == 0;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// The pool's rows (one token of one page and head, `width` bytes) as a 2-D tensor
// of bytes; a box is `box_rows` whole rows, swizzled over its row's width.
bool row_map(CUtensorMap* m, void* pages, const kvq_paged_pool* c, int width, int box_rows) {
  EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width),
                              static_cast<cuuint64_t>(c->n_pages) * c->n_kv_heads * c->page_size};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pages, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            width == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
            : width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_32B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: ticket counters (zero between calls), then the split's partials.
constexpr size_t kTicketBytes = 1024;
constexpr size_t part_floats(int rg, int D) { return static_cast<size_t>(rg) * (D + 2); }
size_t workspace_bytes(int D) {
  size_t most = 0;  // per CTA: a slot for each warp and two of its own
  for (int nt = 1; nt <= 2; ++nt)
    for (const bool four : {false, true})
      most = std::max(most, (paged_warps(nt, four) + 2) * part_floats(8 * nt, D) * sizeof(float));
  return kTicketBytes + kPagedMaxCtas * most;
}
static_assert(kPagedMaxCtas * sizeof(int) <= kTicketBytes, "a ticket per CTA");

// The attention over either kind of pages; `four`: *pool holds a 4-bit pool's
// buffers (codes as pages, metadata as scales).
kvq_status attention(const kvq_paged_pool* pool, bool four, const void* q, int dtype,
                     long long q_stride, void* out, long long out_stride, int n_tokens,
                     int n_q_heads, const int* block_table, int max_pages, const int* cu_new,
                     const int* seq_len, int batch, int max_new, float softmax_scale, int window,
                     void* workspace, size_t n_workspace, int* device_error, void* stream) {
  kvq_status s = check_pool(pool);
  if (s != KVQ_OK) return s;
  const int H = pool->n_kv_heads, D = pool->head_dim;
  if (!pool_pointers(pool) || (four && !meta_pointers(pool)) || !dtype_ok(dtype) || n_tokens < 0 || batch < 1 || max_pages < 1 ||
      max_new < 1 || window < 0 || n_q_heads < 1 || !std::isfinite(softmax_scale) ||
      !aligned(device_error, 4))
    return KVQ_ERR_INVALID_ARG;
  if (n_q_heads % H != 0) return KVQ_ERR_INVALID_ARG;
  if (!dev_ptr(block_table, 4) || !dev_ptr(cu_new, 4) || !dev_ptr(seq_len, 4) ||
      !dev_ptr(workspace, 16) || n_workspace < workspace_bytes(D))
    return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVQ_OK;
  if (!dev_ptr(q, 16) || !dev_ptr(out, 16) || !stride_ok(q_stride, n_q_heads, D) ||
      !stride_ok(out_stride, n_q_heads, D))
    return KVQ_ERR_INVALID_ARG;
  const int R = n_q_heads / H;
  // (the kernels name positions of up to a batch of tiles behind the last token)
  if (R > 16 || batch > kPagedMaxBatch || max_pages > (INT_MAX - 4096) / pool->page_size)
    return KVQ_ERR_UNSUPPORTED;
  max_new = std::min(max_new, n_tokens);
  // positions minus the window stay inside 32 bits
  if (window >= static_cast<long long>(max_pages) * pool->page_size) window = 0;
  if (window > INT_MAX - (1 << 28)) return KVQ_ERR_UNSUPPORTED;
  const int nt = static_cast<long long>(max_new) * R <= 8 ? 1 : 2;
  // units of the decode kernel's items are counted in 31 bits
  const int ut = paged_unit_tokens(D);
  const long long span = static_cast<long long>(max_pages) * pool->page_size;
  const long long rows_all = static_cast<long long>(n_tokens) * R;
  if (rows_all >= 1 << 28) return KVQ_ERR_UNSUPPORTED;  // row_token's range
  const int turn = decode_rows(static_cast<long long>(batch) * H, D);
  const long long groups = std::min<long long>(static_cast<long long>(batch) * ((turn + 8 * nt - 1) / (8 * nt)),
                                               rows_all / (8 * nt) + batch);
  if (static_cast<double>(H) * groups * (static_cast<double>(span) / ut + 2) >= 2147483647.0)
    return KVQ_ERR_UNSUPPORTED;
  // row-tile pairs of the prompt kernel, at most
  const bool prompts = static_cast<long long>(max_new) * R > turn;
  const long long pairs = rows_all / 256 + std::min<long long>(batch, rows_all / (turn + 1));
  if (prompts && pairs * H > INT_MAX) return KVQ_ERR_UNSUPPORTED;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  PagedAttnParams p;
  p.q = q;
  p.out = out;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.table = block_table;
  p.max_pages = max_pages;
  p.cu_new = cu_new;
  p.seq_len = seq_len;
  p.batch = batch;
  p.n_tokens = n_tokens;
  p.max_new = max_new;
  p.H = H;
  p.R = R;
  p.r_magic = static_cast<uint32_t>(((1ull << 32) + R - 1) / R);
  p.lg_ps = log2_of(pool->page_size);
  p.n_pages = pool->n_pages;
  p.k_scale = four ? nullptr : pool->k_scale;
  p.v_scale = four ? nullptr : pool->v_scale;
  p.meta[0] = four ? reinterpret_cast<const uint32_t*>(pool->k_scale) : nullptr;
  p.meta[1] = four ? reinterpret_cast<const uint32_t*>(pool->v_scale) : nullptr;
  p.qscale = softmax_scale * 1.4426950408889634f;
  p.window = window;
  p.row_min = 1;
  p.row_max = turn;
  p.n_warps = std::min(sms, kPagedMaxCtas) * paged_warps(nt, four);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.tickets = reinterpret_cast<int*>(ws);
  p.warp_part = reinterpret_cast<float*>(ws + kTicketBytes);
  p.cta_part = p.warp_part + static_cast<size_t>(p.n_warps) * part_floats(8 * nt, D);
  p.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  p.err = device_error;
  const bool bf = dtype == KVQ_DTYPE_BF16;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int width = four ? D / 2 : D;
  CUtensorMap km, vm;
  if (prompts && pairs > 0) {
    PagedAttnParams a = p;
    a.row_min = turn + 1;
    a.row_max = INT_MAX;
    a.box_rows = pool->page_size;
    if (!row_map(&km, pool->k_pages, pool, width, a.box_rows) ||
        !row_map(&vm, pool->v_pages, pool, width, a.box_rows))
      return KVQ_ERR_CUDA;
    if ((four ? launch_paged4_prompt : launch_paged_prompt)(a, static_cast<int>(pairs), km, vm, D, bf, st) !=
        cudaSuccess) {
      cudaGetLastError();
      return KVQ_ERR_CUDA;
    }
    count_launches(1);
  }
  p.box_rows = std::min(pool->page_size, ut);
  if (!row_map(&km, pool->k_pages, pool, width, p.box_rows) ||
      !row_map(&vm, pool->v_pages, pool, width, p.box_rows))
    return KVQ_ERR_CUDA;
  const auto decode = four ? (D == 128 ? paged4_decode_d128 : paged4_decode_d64)
                           : (D == 128 ? paged_decode_d128 : paged_decode_d64);
  const cudaError_t e = decode(p, km, vm, bf, nt, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

// A 4-bit pool's buffers and sizes as the calls of both kinds of pages pass them
// on: codes as pages, metadata as scales.
kvq_paged_pool as_pool(const kvq_paged4_pool* p) {
  if (p == nullptr) return {};
  return {p->k_codes, p->v_codes, static_cast<float*>(p->k_meta), static_cast<float*>(p->v_meta),
          p->n_pages, p->n_kv_heads, p->page_size, p->head_dim};
}

kvq_status store_params(PagedStoreParams* p, const kvq_paged_pool* pool, const void* k, const void* v, int dtype,
                        long long k_stride, long long v_stride, const int* slots, int n_tokens, int* device_error) {
  const kvq_status s = check_pool(pool);
  if (s != KVQ_OK) return s;
  if (!pool_pointers(pool) || n_tokens < 0 || !dtype_ok(dtype) || !aligned(device_error, 4))
    return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVQ_OK;
  if (!dev_ptr(k, 16) || !dev_ptr(v, 16) || !dev_ptr(slots, 4) ||
      !stride_ok(k_stride, pool->n_kv_heads, pool->head_dim) ||
      !stride_ok(v_stride, pool->n_kv_heads, pool->head_dim))
    return KVQ_ERR_INVALID_ARG;
  if (pool->n_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;  // grid.y
  p->pages[0] = static_cast<uint8_t*>(pool->k_pages);
  p->pages[1] = static_cast<uint8_t*>(pool->v_pages);
  p->scale[0] = pool->k_scale;
  p->scale[1] = pool->v_scale;
  p->x[0] = k;
  p->x[1] = v;
  p->stride[0] = k_stride;
  p->stride[1] = v_stride;
  p->slots = slots;
  p->n_tokens = n_tokens;
  p->n_pages = pool->n_pages;
  p->H = pool->n_kv_heads;
  p->lg_ps = log2_of(pool->page_size);
  p->err = device_error;
  p->angles = nullptr;
  p->rot = p->interleaved = 0;
  p->q.n_heads = 0;
  return KVQ_OK;
}

kvq_status store(const PagedStoreParams& p, int D, int dtype, void* stream) {
  if (launch_paged_store(p, D, dtype, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_paged_pool_check(const kvq_paged_pool* pool) { return check_pool(pool); }

kvq_status kvq_paged_plan(const int* ctx_len, const int* new_len, int batch, int* block_table,
                          int max_pages, const int* free_pages, int n_free_pages,
                          const int* n_free, int page_size, int n_tokens, int* cu_new,
                          int* seq_len, int* slots, int* n_left, int* device_error, void* stream) {
  return kvq_paged_plan_positions(ctx_len, new_len, batch, block_table, max_pages, free_pages, n_free_pages,
                                  n_free, page_size, n_tokens, cu_new, seq_len, slots, nullptr, n_left,
                                  device_error, stream);
}

kvq_status kvq_paged_plan_positions(const int* ctx_len, const int* new_len, int batch,
                                    int* block_table, int max_pages, const int* free_pages,
                                    int n_free_pages, const int* n_free, int page_size,
                                    int n_tokens, int* cu_new, int* seq_len, int* slots,
                                    int* positions, int* n_left, int* device_error, void* stream) {
  if (batch < 1 || max_pages < 1 || n_free_pages < 0 || n_tokens < 0 || page_size < 1)
    return KVQ_ERR_INVALID_ARG;
  if (!dev_ptr(ctx_len, 4) || !dev_ptr(new_len, 4) || !dev_ptr(block_table, 4) ||
      !dev_ptr(n_free, 4) || !dev_ptr(cu_new, 4) || !dev_ptr(seq_len, 4) || !dev_ptr(n_left, 4) ||
      !aligned(device_error, 4))
    return KVQ_ERR_INVALID_ARG;
  if (n_free_pages > 0 && !dev_ptr(free_pages, 4)) return KVQ_ERR_INVALID_ARG;
  if (n_tokens > 0 && !dev_ptr(slots, 16)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(positions, 16)) return KVQ_ERR_INVALID_ARG;
  // every CTA writes positions while others read the inputs and write the outputs
  if (positions != nullptr) {
    const struct {
      const int* at;
      size_t n;
    } others[] = {{ctx_len, static_cast<size_t>(batch)},
                  {new_len, static_cast<size_t>(batch)},
                  {block_table, static_cast<size_t>(batch) * max_pages},
                  {free_pages, static_cast<size_t>(n_free_pages)},
                  {n_free, 1},
                  {cu_new, static_cast<size_t>(batch) + 1},
                  {seq_len, static_cast<size_t>(batch)},
                  {slots, static_cast<size_t>(n_tokens)},
                  {n_left, 1},
                  {device_error, 1}};
    for (const auto& x : others)
      if (x.at != nullptr && overlap(positions, static_cast<size_t>(n_tokens), x.at, x.n)) return KVQ_ERR_INVALID_ARG;
  }
  // several CTAs read the inputs while the first writes these
  if (seq_len == ctx_len || seq_len == new_len || n_left == n_free || cu_new == ctx_len ||
      cu_new == new_len)
    return KVQ_ERR_INVALID_ARG;
  if (!page_size_ok(page_size) || batch > kPagedMaxBatch || max_pages > INT_MAX / page_size)
    return KVQ_ERR_UNSUPPORTED;
  PagedPlanParams p;
  p.ctx_len = ctx_len;
  p.new_len = new_len;
  p.batch = batch;
  p.table = block_table;
  p.max_pages = max_pages;
  p.free_pages = free_pages;
  p.free_cap = n_free_pages;
  p.n_free = n_free;
  p.lg_ps = log2_of(page_size);
  p.n_tokens = n_tokens;
  p.cu_new = cu_new;
  p.seq_len = seq_len;
  p.slots = slots;
  p.positions = positions;
  p.n_left = n_left;
  p.err = device_error;
  if (launch_paged_plan(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

kvq_status kvq_paged_store(const kvq_paged_pool* pool, const void* k, const void* v, int dtype,
                           long long k_stride, long long v_stride, const int* slots, int n_tokens,
                           int* device_error, void* stream) {
  PagedStoreParams p;
  const kvq_status s = store_params(&p, pool, k, v, dtype, k_stride, v_stride, slots, n_tokens, device_error);
  if (s != KVQ_OK || n_tokens == 0) return s;
  if (n_tokens > kPagedMaxStore) return KVQ_ERR_UNSUPPORTED;
  return store(p, pool->head_dim, dtype, stream);
}

kvq_status kvq_paged_append(const kvq_paged_pool* pool, const kvq_rotary* rotary, const void* k,
                            const void* v, int dtype, long long k_stride, long long v_stride,
                            const int* slots, int n_tokens, const void* q, long long q_stride,
                            void* q_out, long long q_out_stride, int n_q_heads, int* device_error,
                            void* stream) {
  PagedStoreParams p;
  kvq_status s = store_params(&p, pool, k, v, dtype, k_stride, v_stride, slots, n_tokens, device_error);
  if (s != KVQ_OK) return s;
  s = check_rotary(rotary, pool->head_dim, n_tokens);
  if (s != KVQ_OK) return s;
  if (q != nullptr || q_out != nullptr || n_q_heads != 0) {
    if (n_q_heads < 1) return KVQ_ERR_INVALID_ARG;
    s = rotate_params(&p.q, rotary, q, dtype, q_stride, q_out, q_out_stride, n_tokens, n_q_heads, pool->head_dim);
    if (s != KVQ_OK) return s;
    if (pool->n_kv_heads > 65535 - 512) return KVQ_ERR_UNSUPPORTED;  // grid.y: at most a row of CTAs a chunk's token
  }
  if (n_tokens == 0) return KVQ_OK;
  if (n_tokens > kPagedMaxStore) return KVQ_ERR_UNSUPPORTED;
  p.angles = reinterpret_cast<const float2*>(rotary->angles);
  p.rot = rotary->rotary_dim;
  p.interleaved = rotary->interleaved;
  return store(p, pool->head_dim, dtype, stream);
}

kvq_status kvq_paged_workspace_bytes(const kvq_paged_pool* pool, size_t* bytes) {
  if (bytes == nullptr) return KVQ_ERR_INVALID_ARG;
  const kvq_status s = check_pool(pool);
  if (s != KVQ_OK) return s;
  *bytes = workspace_bytes(pool->head_dim);
  return KVQ_OK;
}

kvq_status kvq_paged_attention(const kvq_paged_pool* pool, const void* q, int dtype,
                               long long q_stride, void* out, long long out_stride, int n_tokens,
                               int n_q_heads, const int* block_table, int max_pages,
                               const int* cu_new, const int* seq_len, int batch, int max_new,
                               float softmax_scale, int window, void* workspace,
                               size_t n_workspace, int* device_error, void* stream) {
  return attention(pool, false, q, dtype, q_stride, out, out_stride, n_tokens, n_q_heads, block_table, max_pages, cu_new,
                   seq_len, batch, max_new, softmax_scale, window, workspace, n_workspace, device_error, stream);
}

kvq_status kvq_paged4_pool_check(const kvq_paged4_pool* pool) {
  const kvq_paged_pool c = as_pool(pool);
  return check_pool(pool ? &c : nullptr);
}

kvq_status kvq_paged4_append(const kvq_paged4_pool* pool, const kvq_rotary* rotary, const void* k,
                             const void* v, int dtype, long long k_stride, long long v_stride,
                             const int* slots, int n_tokens, const void* q, long long q_stride,
                             void* q_out, long long q_out_stride, int n_q_heads, int* device_error,
                             void* stream) {
  const kvq_paged_pool c = as_pool(pool);
  PagedStoreParams w;
  kvq_status s = store_params(&w, pool ? &c : nullptr, k, v, dtype, k_stride, v_stride, slots, n_tokens,
                              device_error);
  if (s != KVQ_OK) return s;
  if (!meta_pointers(&c)) return KVQ_ERR_INVALID_ARG;
  Paged4StoreParams p = {};
  const bool queries = q != nullptr || q_out != nullptr || n_q_heads != 0;
  if (rotary != nullptr) {
    s = check_rotary(rotary, c.head_dim, n_tokens);
    if (s != KVQ_OK) return s;
  }
  if (queries) {
    if (rotary == nullptr || n_q_heads < 1) return KVQ_ERR_INVALID_ARG;
    s = rotate_params(&p.q, rotary, q, dtype, q_stride, q_out, q_out_stride, n_tokens, n_q_heads, c.head_dim);
    if (s != KVQ_OK) return s;
    if (n_tokens > INT_MAX / 2) return KVQ_ERR_UNSUPPORTED;  // grid.x: at most two CTAs a token
  }
  if (n_tokens == 0) return KVQ_OK;
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = w.pages[i];
    p.meta[i] = reinterpret_cast<uint32_t*>(w.scale[i]);
    p.x[i] = w.x[i];
    p.stride[i] = w.stride[i];
  }
  p.slots = slots;
  p.n_tokens = n_tokens;
  p.n_pages = c.n_pages;
  p.H = c.n_kv_heads;
  p.lg_ps = w.lg_ps;
  p.err = device_error;
  if (rotary != nullptr) {
    p.angles = reinterpret_cast<const float2*>(rotary->angles);
    p.rot = rotary->rotary_dim;
    p.interleaved = rotary->interleaved;
  }
  if (launch_paged4_append(p, c.head_dim, dtype, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

kvq_status kvq_paged4_read(const kvq_paged4_pool* pool, const int* slots, int n_tokens, void* k_out,
                           void* v_out, int* device_error, void* stream) {
  const kvq_paged_pool c = as_pool(pool);
  const kvq_status s = check_pool(pool ? &c : nullptr);
  if (s != KVQ_OK) return s;
  if (!pool_pointers(&c) || !meta_pointers(&c) || n_tokens < 0 || !aligned(device_error, 4) ||
      !aligned(k_out, 16) || !aligned(v_out, 16))
    return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || (k_out == nullptr && v_out == nullptr)) return KVQ_OK;
  if (!dev_ptr(slots, 4)) return KVQ_ERR_INVALID_ARG;
  Paged4ReadParams p;
  p.codes[0] = static_cast<const uint8_t*>(c.k_pages);
  p.codes[1] = static_cast<const uint8_t*>(c.v_pages);
  p.meta[0] = reinterpret_cast<const uint32_t*>(c.k_scale);
  p.meta[1] = reinterpret_cast<const uint32_t*>(c.v_scale);
  p.out[0] = static_cast<uint16_t*>(k_out);
  p.out[1] = static_cast<uint16_t*>(v_out);
  p.slots = slots;
  p.n_tokens = n_tokens;
  p.n_pages = c.n_pages;
  p.H = c.n_kv_heads;
  p.lg_ps = log2_of(c.page_size);
  p.err = device_error;
  if (launch_paged4_read(p, c.head_dim, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

kvq_status kvq_paged4_workspace_bytes(const kvq_paged4_pool* pool, size_t* bytes) {
  const kvq_paged_pool c = as_pool(pool);
  return kvq_paged_workspace_bytes(pool ? &c : nullptr, bytes);
}

kvq_status kvq_paged4_attention(const kvq_paged4_pool* pool, const void* q, int dtype,
                                long long q_stride, void* out, long long out_stride, int n_tokens,
                                int n_q_heads, const int* block_table, int max_pages,
                                const int* cu_new, const int* seq_len, int batch, int max_new,
                                float softmax_scale, int window, void* workspace,
                                size_t n_workspace, int* device_error, void* stream) {
  const kvq_paged_pool c = as_pool(pool);
  return attention(pool ? &c : nullptr, true, q, dtype, q_stride, out, out_stride, n_tokens, n_q_heads, block_table, max_pages, cu_new,
                   seq_len, batch, max_new, softmax_scale, window, workspace, n_workspace, device_error, stream);
}

kvq_status kvq_debug_set_paged_wait_limit(int limit) {
  g_wait_limit.store(limit < 0 ? UINT32_MAX : static_cast<uint32_t>(limit), std::memory_order_relaxed);
  return KVQ_OK;
}

}  // extern "C"
