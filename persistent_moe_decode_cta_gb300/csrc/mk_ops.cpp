// Host entry points of the multi-token operators (include/mk.h): argument checks, tensor
// maps, launches.  Nothing here allocates device memory or synchronises.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "mk.h"
#include "mk_ops.h"

using namespace mk;

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* sym = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(sym);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int cuda_error(cudaError_t e, const char* what) {
  return e == cudaSuccess ? (int)MK_OK : op_fail(MK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int num_sms(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return cuda_error(e, "device query");
}

int encode(CUtensorMap* tm, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
           const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  auto fn = encoder();
  if (!fn) return op_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return op_fail(MK_ERR_INVALID, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MK_OK;
}

int check_cache(const mk_paged_kv* c, bool pointers) {
  if (!c) return op_fail(MK_ERR_INVALID, "cache is NULL");
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128)
    return op_fail(MK_ERR_UNSUPPORTED, "head_dim %d not in {32, 64, 128}", c->head_dim);
  if (c->batch < 1 || c->batch > kOpMaxBatch) return op_fail(MK_ERR_INVALID, "batch %d not in [1, %d]", c->batch, kOpMaxBatch);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024) return op_fail(MK_ERR_INVALID, "n_kv_heads %d not in [1, 1024]", c->n_kv_heads);
  if (c->max_pages < 1 || c->max_pages > (1 << 26)) return op_fail(MK_ERR_INVALID, "max_pages %d not in [1, 2^26]", c->max_pages);
  if (c->n_pages < 1 || (long long)c->n_pages * c->n_kv_heads * kOpPage > 0x7fffffffll)
    return op_fail(MK_ERR_INVALID, "n_pages %d: need 1 <= n_pages and n_pages * n_kv_heads * 16 < 2^31", c->n_pages);
  if (!pointers) return MK_OK;
  if (!c->k || !c->v || !c->page_table || !c->seq_lens) return op_fail(MK_ERR_INVALID, "NULL cache pointer");
  if (!aligned16(c->k) || !aligned16(c->v)) return op_fail(MK_ERR_INVALID, "K/V pools must be 16-byte aligned");
  return MK_OK;
}

// K and V of `layers` layers in memory of their own: an operator that writes both would write one
// twice, in any order
int check_apart(const mk_paged_kv* c, long long layers) {
  const uintptr_t k = reinterpret_cast<uintptr_t>(c->k), v = reinterpret_cast<uintptr_t>(c->v);
  const unsigned long long bytes = (unsigned long long)layers * c->n_pages * c->n_kv_heads * kOpPage * c->head_dim * 2;
  if ((k < v ? v - k : k - v) < bytes) return op_fail(MK_ERR_INVALID, "the K and V pools overlap");
  return MK_OK;
}

int check_heads(const mk_paged_kv* c, int n_nodes, int n_q_heads) {
  if (n_nodes < 1 || n_nodes > (1 << 24)) return op_fail(MK_ERR_INVALID, "n_nodes %d not in [1, 2^24]", n_nodes);
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads) return op_fail(MK_ERR_INVALID, "n_q_heads %d not a multiple of n_kv_heads %d", n_q_heads, c->n_kv_heads);
  if (n_q_heads > 4096) return op_fail(MK_ERR_INVALID, "n_q_heads %d > 4096", n_q_heads);
  return MK_OK;
}

// a [batch][n_nodes][heads][head_dim] operand: 16-byte aligned, strides multiples of 8
int check_rows(const char* name, const void* ptr, const int64_t* stride, const int64_t* dims) {
  if (!ptr) return op_fail(MK_ERR_INVALID, "%s is NULL", name);
  if (!aligned16(ptr)) return op_fail(MK_ERR_INVALID, "%s must be 16-byte aligned", name);
  for (int i = 0; i < 3; ++i)
    if (dims[i] > 1 && (stride[i] <= 0 || stride[i] % 8 || stride[i] >= (1ll << 38)))
      return op_fail(MK_ERR_INVALID, "%s: stride %lld of dimension %d is not a positive multiple of 8 elements", name, (long long)stride[i], i);
  return MK_OK;
}

// where a call records what its kernels find wrong: the caller's record or the device's own
int set_record(int32_t*& status) {
  return status ? (int)MK_OK : cuda_error(op_record(&status), "error record");
}

// the tile shape of mk_tree_attention for these sizes (device: the SM count)
int tree_shape(const mk_paged_kv* c, const mk_tree_args* a, TreeParams& p) {
  if (!a) return op_fail(MK_ERR_INVALID, "args is NULL");
  int r = check_cache(c, false);
  if (!r) r = check_heads(c, a->n_nodes, a->n_q_heads);
  if (r) return r;
  p.c = *c;
  p.a = *a;
  p.gs = a->n_q_heads / c->n_kv_heads;
  if (p.gs > 128) return op_fail(MK_ERR_UNSUPPORTED, "query group %d > 128", p.gs);
  const int fit = 128 / p.gs;
  p.two = a->n_nodes > fit;
  p.npt = std::min(fit, a->n_nodes);
  const int per = p.npt * (p.two ? 2 : 1);
  p.ntp = (a->n_nodes + per - 1) / per;
  p.team = p.ntp <= 8 ? p.ntp : 1;
  p.words = (a->n_nodes + 31) / 32;
  const double units = (double)c->batch * c->n_kv_heads * p.ntp * ((double)c->max_pages / 8 + 2 + kItemUnits);
  if (units >= 1073741824.0 || (double)c->batch * c->n_kv_heads * p.ntp * 8 >= 1073741824.0)
    return op_fail(MK_ERR_UNSUPPORTED, "batch x heads x nodes x keys exceeds 2^30 work units");
  // (every CTA adds up the work list, 128 entries at a time)
  p.groups = (p.ntp + p.team - 1) / p.team;
  if ((long long)c->batch * p.groups > kOpMaxEntries)
    return op_fail(MK_ERR_UNSUPPORTED, "batch x groups of nodes: %lld > %d", (long long)c->batch * p.groups, kOpMaxEntries);
  const int rc = num_sms(&p.grid);
  if (rc) return rc;
  p.teams = std::max(1, p.grid / p.team);
  return MK_OK;
}

}  // namespace

extern "C" {

int mk_qk_norm_rope(const mk_paged_kv* cache, const mk_rope_args* args, void* stream) {
  int r = check_cache(cache, true);
  if (r) return r;
  if (!args) return op_fail(MK_ERR_INVALID, "args is NULL");
  r = check_heads(cache, args->n_nodes, args->n_q_heads);
  const int64_t dq[3] = {cache->batch, args->n_nodes, args->n_q_heads}, dk[3] = {cache->batch, args->n_nodes, cache->n_kv_heads};
  if (!r) r = check_rows("q", args->q, args->q_stride, dq);
  if (!r) r = check_rows("k", args->k, args->k_stride, dk);
  if (!r) r = check_rows("v", args->v, args->v_stride, dk);
  if (!r) r = check_rows("q_out", args->q_out, args->out_stride, dq);
  if (r) return r;
  if ((long long)cache->batch * args->n_nodes >= 0x7fffffffll - (1 << 20))
    return op_fail(MK_ERR_UNSUPPORTED, "batch x n_nodes does not fit 31 bits");
  if ((args->q_gain && !aligned16(args->q_gain)) || (args->k_gain && !aligned16(args->k_gain)))
    return op_fail(MK_ERR_INVALID, "gains must be 16-byte aligned");
  if (!(args->theta >= 1.0) || !std::isfinite(args->theta)) return op_fail(MK_ERR_INVALID, "theta must be finite and >= 1");
  if (!(args->eps >= 0.f) || !std::isfinite(args->eps)) return op_fail(MK_ERR_INVALID, "eps must be finite and >= 0");
  r = check_apart(cache, 1);
  if (r) return r;
  RopeParams p{};
  p.c = *cache;
  p.a = *args;
  const int half = cache->head_dim / 2;
  // turns per position, as a fraction of 2^64 (the last theta's table is kept: 64 powers take
  // as long as the launch)
  struct Turns {
    double theta = 0;
    int half = 0;
    unsigned long long t[kOpMaxHalf];
  };
  static thread_local Turns table;
  if (table.theta != args->theta || table.half != half) {
    for (int i = 0; i < half; ++i)
      table.t[i] = (unsigned long long)std::ldexp(std::pow(args->theta, -(double)i / half) / (2 * M_PI), 64);
    table.theta = args->theta;
    table.half = half;
  }
  std::copy(table.t, table.t + half, p.turns);
  r = set_record(p.a.status);
  int sms = 0;
  if (!r) r = num_sms(&sms);
  if (r) return r;
  return cuda_error(launch_rope(p, sms, static_cast<cudaStream_t>(stream)), "qk_norm_rope launch");
}

int mk_tree_attention_workspace(const mk_paged_kv* cache, const mk_tree_args* args, size_t* bytes) {
  if (!bytes) return op_fail(MK_ERR_INVALID, "bytes is NULL");
  TreeParams p{};
  const int r = tree_shape(cache, args, p);
  if (r) return r;
  *bytes = tree_workspace_bytes(p);
  return MK_OK;
}

int mk_tree_attention(const mk_paged_kv* cache, const mk_tree_args* args, void* stream) {
  int r = check_cache(cache, true);
  if (r) return r;
  if (!args) return op_fail(MK_ERR_INVALID, "args is NULL");
  r = check_heads(cache, args->n_nodes, args->n_q_heads);
  const int64_t dq[3] = {cache->batch, args->n_nodes, args->n_q_heads};
  if (!r) r = check_rows("q", args->q, args->q_stride, dq);
  if (!r) r = check_rows("out", args->out, args->out_stride, dq);
  if (r) return r;
  if (args->out == args->q) return op_fail(MK_ERR_INVALID, "out must not be q");
  if (!(args->scale >= 0.f) || !std::isfinite(args->scale * 1.4426950408889634f)) return op_fail(MK_ERR_INVALID, "scale must be finite and >= 0");
  if (args->window < 0) return op_fail(MK_ERR_INVALID, "window %d < 0", args->window);
  if (!args->workspace || !aligned16(args->workspace)) return op_fail(MK_ERR_INVALID, "workspace must be 16-byte aligned and not NULL");
  TreeParams p{};
  r = tree_shape(cache, args, p);
  if (r) return r;
  const size_t need = tree_workspace_bytes(p);
  if (args->workspace_bytes < need)
    return op_fail(MK_ERR_INVALID, "workspace has %zu bytes, needs %zu", args->workspace_bytes, need);
  // (a scale of 0 would turn a masked score of -infinity into NaN)
  p.scale_log2 = std::max(args->scale * 1.4426950408889634f, 1e-30f);
  const int hd = cache->head_dim, span = hd == 32 ? 32 : 64;  // elements of a swizzle span
  const CUtensorMapSwizzle sw = hd == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  // queries: column, head, node, sequence; a box is one tile's nodes of one KV head.  (The
  // stride of a dimension of one element is never used, but has to be a valid one.)
  CUtensorMap tq, tk, tv;
  cuuint64_t qd[4] = {(cuuint64_t)hd, (cuuint64_t)args->n_q_heads, (cuuint64_t)args->n_nodes, (cuuint64_t)cache->batch};
  cuuint64_t qs[3];
  for (int i = 0; i < 3; ++i) {
    const int d = 2 - i;  // head, node, sequence
    qs[i] = dq[d] > 1 ? (cuuint64_t)args->q_stride[d] * 2 : (cuuint64_t)hd * 2;
  }
  cuuint32_t qb[4] = {(cuuint32_t)span, (cuuint32_t)p.gs, (cuuint32_t)p.npt, 1};
  r = encode(&tq, args->q, 4, qd, qs, qb, sw);
  // keys: column in the span, row of a group of 8, span, group (a page of a head is two groups)
  cuuint64_t kd[4] = {(cuuint64_t)span, 8, (cuuint64_t)hd / span, (cuuint64_t)cache->n_pages * cache->n_kv_heads * (kOpPage / 8)};
  cuuint64_t ks[3] = {(cuuint64_t)hd * 2, (cuuint64_t)span * 2, (cuuint64_t)hd * 16};
  cuuint32_t kb[4] = {(cuuint32_t)span, 8, (cuuint32_t)(hd / span), kOpPage / 8};
  if (!r) r = encode(&tk, cache->k, 4, kd, ks, kb, sw);
  if (!r) r = encode(&tv, cache->v, 4, kd, ks, kb, sw);
  if (!r) r = set_record(p.a.status);
  if (r) return r;
  return cuda_error(launch_tree(p, tq, tk, tv, static_cast<cudaStream_t>(stream)), "tree_attention launch");
}

int mk_copy_pages(void* k_cache, void* v_cache, int n_layers, int n_pages, int n_kv_heads, int head_dim,
                  const int32_t* src, const int32_t* dst, int n, void* stream) {
  mk_paged_kv c{};
  c.n_pages = n_pages;
  c.n_kv_heads = n_kv_heads;
  c.head_dim = head_dim;
  c.batch = c.max_pages = 1;
  int r = check_cache(&c, false);
  if (r) return r;
  if (!k_cache || !v_cache) return op_fail(MK_ERR_INVALID, "NULL cache pointer");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return op_fail(MK_ERR_INVALID, "K/V pools must be 16-byte aligned");
  if (n_layers < 1 || n_layers > 65535) return op_fail(MK_ERR_INVALID, "n_layers %d not in [1, 65535]", n_layers);
  if (n < 0 || n > n_pages) return op_fail(MK_ERR_INVALID, "%d copies, %d pages", n, n_pages);
  if (n == 0) return MK_OK;
  if (!src || !dst) return op_fail(MK_ERR_INVALID, "NULL page list");
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages)
      return op_fail(MK_ERR_BAD_PAGE, "copy %d: page %d -> %d outside [0, %d)", i, src[i], dst[i], n_pages);
  try {
    // written pages in order: a page that is written twice, or written and read, is refused
    std::vector<int32_t> d(dst, dst + n);
    std::sort(d.begin(), d.end());
    const auto twice = std::adjacent_find(d.begin(), d.end());
    if (twice != d.end()) return op_fail(MK_ERR_INVALID, "page %d is written twice", *twice);
    for (int i = 0; i < n; ++i)
      if (std::binary_search(d.begin(), d.end(), src[i])) return op_fail(MK_ERR_INVALID, "page %d is both read and written", src[i]);
  } catch (const std::bad_alloc&) {
    return op_fail(MK_ERR_OOM, "host memory for %d page ids", n);
  }
  c.k = k_cache;
  c.v = v_cache;
  if (k_cache != v_cache) r = check_apart(&c, n_layers);  // (the same copies twice do no harm)
  if (r) return r;
  const long long page = (long long)n_kv_heads * kOpPage * head_dim * 2;
  return cuda_error(launch_copy_pages(static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), n_layers, page * n_pages,
                                      page, src, dst, n, static_cast<cudaStream_t>(stream)),
                    "copy_pages launch");
}

int mk_commit_nodes(const mk_paged_kv* cache, int n_layers, const int32_t* accepted, int max_accept, int32_t* new_lens,
                    int32_t* status, void* stream) {
  int r = check_cache(cache, true);
  if (r) return r;
  if (n_layers < 1 || n_layers > 65535) return op_fail(MK_ERR_INVALID, "n_layers %d not in [1, 65535]", n_layers);
  if (!accepted || !new_lens) return op_fail(MK_ERR_INVALID, "NULL pointer");
  if (max_accept < 1 || max_accept > kOpMaxAccept) return op_fail(MK_ERR_INVALID, "max_accept %d not in [1, %d]", max_accept, kOpMaxAccept);
  // (a sequence's length is written while other blocks may still have to read)
  const auto overlaps = [&](const int32_t* p, long long n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(new_lens), b = reinterpret_cast<uintptr_t>(p);
    return a < b + n * 4 && b < a + cache->batch * 4ll;
  };
  if (overlaps(cache->seq_lens, cache->batch)) return op_fail(MK_ERR_INVALID, "new_lens must not be seq_lens nor a part of it");
  if (overlaps(accepted, (long long)cache->batch * max_accept) || overlaps(cache->page_table, (long long)cache->batch * cache->max_pages))
    return op_fail(MK_ERR_INVALID, "new_lens must not be a part of accepted or of the page table");
  r = check_apart(cache, n_layers);
  if (r) return r;
  CommitParams p{};
  p.c = *cache;
  p.n_layers = n_layers;
  p.max_accept = max_accept;
  p.accepted = accepted;
  p.new_lens = new_lens;
  p.status = status;
  r = set_record(p.status);
  if (r) return r;
  return cuda_error(launch_commit(p, static_cast<cudaStream_t>(stream)), "commit_nodes launch");
}

int mk_expert_product(const mk_expert_args* a, void* stream) {
  if (!a) return op_fail(MK_ERR_INVALID, "args is NULL");
  if (!a->x || !a->w || !a->offsets || !a->out) return op_fail(MK_ERR_INVALID, "NULL pointer");
  if (a->out == a->x) return op_fail(MK_ERR_INVALID, "out must not be x");
  if (!aligned16(a->x) || !aligned16(a->w) || (a->w_up && !aligned16(a->w_up)))
    return op_fail(MK_ERR_INVALID, "x, w and w_up must be 16-byte aligned");
  if (a->n_experts < 1 || a->n_experts > kOpMaxExperts) return op_fail(MK_ERR_INVALID, "n_experts %d not in [1, %d]", a->n_experts, kOpMaxExperts);
  if (a->n < 1 || a->n > (1 << 24)) return op_fail(MK_ERR_INVALID, "n %d not in [1, 2^24]", a->n);
  if (a->k < 8 || a->k % 8 || a->k > (1 << 24)) return op_fail(MK_ERR_UNSUPPORTED, "k %d is not a positive multiple of 8", a->k);
  if (a->n_rows < 0 || a->n_rows > (1 << 28)) return op_fail(MK_ERR_INVALID, "n_rows %d not in [0, 2^28]", a->n_rows);
  if (a->n_rows == 0) return MK_OK;
  if (a->n_x < 1 || (!a->rows && a->n_x < a->n_rows)) return op_fail(MK_ERR_INVALID, "n_x %d is too small for %d rows", a->n_x, a->n_rows);
  if (a->x_stride < a->k || a->x_stride % 8 || a->x_stride >= (1ll << 38))
    return op_fail(MK_ERR_INVALID, "x_stride %lld: need a multiple of 8, at least k", (long long)a->x_stride);
  if (a->out_stride < a->n) return op_fail(MK_ERR_INVALID, "out_stride %lld < n", (long long)a->out_stride);
  const long long step = a->w_up ? 128 : 256;
  if (((long long)a->n_rows / 128 + a->n_experts) * ((a->n + step - 1) / step) >= 0x7fffffffll - 1024)
    return op_fail(MK_ERR_UNSUPPORTED, "more than 2^31 tiles");
  ExpertParams p{};
  p.a = *a;
  int r = num_sms(&p.grid);
  if (r) return r;
  CUtensorMap tx, tx128, tw, tu;
  cuuint64_t xd[2] = {(cuuint64_t)a->k, (cuuint64_t)a->n_x};
  cuuint64_t xs[1] = {(cuuint64_t)a->x_stride * 2};
  cuuint32_t xb[2] = {64, 32};
  cuuint32_t xb128[2] = {64, 128};
  r = encode(&tx, a->x, 2, xd, xs, xb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!r) r = encode(&tx128, a->x, 2, xd, xs, xb128, CU_TENSOR_MAP_SWIZZLE_128B);
  cuuint64_t wd[3] = {(cuuint64_t)a->k, (cuuint64_t)a->n, (cuuint64_t)a->n_experts};
  cuuint64_t ws[2] = {(cuuint64_t)a->k * 2, (cuuint64_t)a->n * a->k * 2};
  cuuint32_t wb[3] = {64, a->w_up ? 64u : 128u, 1};
  if (!r) r = encode(&tw, a->w, 3, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!r) r = encode(&tu, a->w_up ? a->w_up : a->w, 3, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!r) r = set_record(p.a.status);
  if (r) return r;
  return cuda_error(launch_experts(p, tx, tx128, tw, tu, static_cast<cudaStream_t>(stream)), "expert_product launch");
}

int mk_op_status(int32_t* status_out, void* stream) {
  if (!status_out) return op_fail(MK_ERR_INVALID, "status_out is NULL");
  const auto st = static_cast<cudaStream_t>(stream);
  int32_t* record = nullptr;
  int r = set_record(record);
  if (r) return r;
  r = cuda_error(cudaMemcpyAsync(status_out, record, 4 * sizeof(int32_t), cudaMemcpyDeviceToHost, st), "error record");
  if (!r) r = cuda_error(cudaStreamSynchronize(st), "error record");
  if (!r && status_out[0]) {
    r = cuda_error(cudaMemsetAsync(record, 0, 4 * sizeof(int32_t), st), "error record");
    if (!r) r = cuda_error(cudaStreamSynchronize(st), "error record");
  }
  return r;
}

}  // extern "C"
