// Moving K/V inside the paged cache: whole pages (copy-on-write of a fork, moving a
// sequence) and the nodes of an accepted draft path.  Both only move bytes.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // 16-byte loads in flight per thread: a block moves 16 KB at a time

// The (source, destination) pairs travel in the kernel's parameters, so that a call takes
// host arrays without a copy of its own and a captured call keeps them.
template <int N>
struct PagePairs {
  int32_t src[N], dst[N];
};

// One block per (pair, layer, K or V, 16 KB of the page).  HBM bounds it: 512 pages of 48 layers (1.6 GB
// moved) 231 us, 7.0 TB/s; 8 pages 4.2 us.
template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ PagePairs<N> pairs, uint4* k, uint4* v,
                                                                  long long layer_vecs, int page_vecs, int parts) {
  const int pair = blockIdx.x / parts, part = blockIdx.x - pair * parts;
  uint4* pool = (blockIdx.z ? v : k) + (long long)blockIdx.y * layer_vecs;
  const uint4* src = pool + (long long)pairs.src[pair] * page_vecs;
  uint4* dst = pool + (long long)pairs.dst[pair] * page_vecs;
  const int i0 = part * kCopyThreads * kCopyVecs + threadIdx.x;
  uint4 x[kCopyVecs];
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int j = 0; j < kCopyVecs; ++j)
    if (i0 + j * kCopyThreads < page_vecs) x[j] = op_ld16_once(src + i0 + j * kCopyThreads);
#pragma unroll
  for (int j = 0; j < kCopyVecs; ++j)
    if (i0 + j * kCopyThreads < page_vecs) __stcs(dst + i0 + j * kCopyThreads, x[j]);
}

template <int N>
cudaError_t copy_some(uint8_t* k, uint8_t* v, int n_layers, long long layer_bytes, long long page_bytes,
                      const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
  PagePairs<N> pairs;
  for (int i = 0; i < n; ++i) {
    pairs.src[i] = src[i];
    pairs.dst[i] = dst[i];
  }
  const int vecs = (int)(page_bytes / 16);
  const int parts = (vecs + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs);
  return launch_early(copy_pages_kernel<N>, dim3((unsigned)(n * parts), (unsigned)n_layers, 2), kCopyThreads, 0, st, pairs,
                      reinterpret_cast<uint4*>(k), reinterpret_cast<uint4*>(v), layer_bytes / 16, vecs, parts);
}

constexpr int kCommitThreads = 128;

// One block per (sequence, KV head, layer, K or V).  The accepted rows of its slice are
// staged in shared memory, all of them before the first is written back, so that the path
// may name the nodes in any order.  A chain of loads (path, page table, rows) bounds it: 8 sequences of 48
// layers 6.7 us.
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CommitParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ int s_count;
  const int hd = p.c.head_dim, vecs = hd / 8;
  int* from = reinterpret_cast<int*>(raw);          // [max_accept] page * n_kv_heads of the node
  int* to = from + p.max_accept;                    // ... and of its new place
  uint4* rows = reinterpret_cast<uint4*>(raw + ((2 * p.max_accept * 4 + 15) & ~15));
  const int b = blockIdx.x / p.c.n_kv_heads, kvh = blockIdx.x - b * p.c.n_kv_heads;
  pdl_wait();
  pdl_trigger();
  const int len = op_ld(p.c.seq_lens + b);
  const int32_t* acc = p.accepted + (long long)b * p.max_accept;
  if (threadIdx.x == 0) s_count = p.max_accept;
  __syncthreads();
  for (int i = threadIdx.x; i < p.max_accept; i += kCommitThreads)
    if (op_ld(acc + i) < 0) atomicMin(&s_count, i);
  __syncthreads();
  const int count = s_count;
  int bad = 0;
  const int32_t* table = p.c.page_table + (long long)b * p.c.max_pages;
  for (int i = threadIdx.x; i < 2 * count; i += kCommitThreads) {
    const int a = i < count ? op_ld(acc + i) : i - count;
    const long long at = (long long)len + a;
    if (len < 0 || at >= 16ll * p.c.max_pages) {
      op_error(p.status, MK_ERR_INVALID, b, a, len);
      bad = 1;
      continue;
    }
    const int page = op_ld(table + at / kOpPage);
    if (page < 0 || page >= p.c.n_pages) {
      op_error(p.status, MK_ERR_BAD_PAGE, b, (int)(at / kOpPage), page);
      bad = 1;
      continue;
    }
    (i < count ? from : to - count)[i] = page * p.c.n_kv_heads;
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.y == 0 && blockIdx.z == 0 && kvh == 0 && threadIdx.x == 0) p.new_lens[b] = len + (bad ? 0 : count);
  if (bad) return;
  const long long layer_vecs = (long long)p.c.n_pages * p.c.n_kv_heads * kOpPage * vecs;
  uint4* pool = static_cast<uint4*>(blockIdx.z ? p.c.v : p.c.k) + (long long)blockIdx.y * layer_vecs;
  for (int i = threadIdx.x; i < count * vecs; i += kCommitThreads) {
    const int r = i / vecs, c = i - r * vecs;
    const int slot = (int)(((long long)len + op_ld(acc + r)) % kOpPage);
    rows[i] = pool[((long long)(from[r] + kvh) * kOpPage + slot) * vecs + c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < count * vecs; i += kCommitThreads) {
    const int r = i / vecs, c = i - r * vecs;
    pool[((long long)(to[r] + kvh) * kOpPage + (len + r) % kOpPage) * vecs + c] = rows[i];
  }
}

// What calls without a record of their own find wrong.
__device__ int32_t own_record[4];

}  // namespace

cudaError_t op_record(int32_t** record) {
  static std::atomic<int32_t*> known[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *record = dev < 64 ? known[dev].load(std::memory_order_acquire) : nullptr;
  if (*record) return cudaSuccess;
  e = cudaGetSymbolAddress(reinterpret_cast<void**>(record), own_record);
  if (e == cudaSuccess && dev < 64) known[dev].store(*record, std::memory_order_release);
  return e;
}

cudaError_t launch_copy_pages(uint8_t* k, uint8_t* v, int n_layers, long long layer_bytes, long long page_bytes,
                              const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
  // few pairs: a small parameter block, which a launch has to carry every time
  constexpr int kFew = 64, kMany = 2000;
  for (int i = 0; i < n;) {
    const int m = n - i <= kFew ? n - i : n - i < kMany ? n - i : kMany;
    const cudaError_t e = m <= kFew ? copy_some<kFew>(k, v, n_layers, layer_bytes, page_bytes, src + i, dst + i, m, st)
                                    : copy_some<kMany>(k, v, n_layers, layer_bytes, page_bytes, src + i, dst + i, m, st);
    if (e != cudaSuccess) return e;
    i += m;
  }
  return cudaSuccess;
}

cudaError_t launch_commit(const CommitParams& p, cudaStream_t st) {
  const size_t smem = ((2 * (size_t)p.max_accept * 4 + 15) & ~(size_t)15) + (size_t)p.max_accept * p.c.head_dim * 2;
  if (smem > 48 * 1024) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(commit_kernel, kOpMaxAccept * (2 * 4 + 2 * 2 * kOpMaxHalf), done);  // the most of any call
    if (e != cudaSuccess) return e;
  }
  return launch_early(commit_kernel, dim3((unsigned)(p.c.batch * p.c.n_kv_heads), (unsigned)p.n_layers, 2), kCommitThreads, smem, st, p);
}

}  // namespace mk
