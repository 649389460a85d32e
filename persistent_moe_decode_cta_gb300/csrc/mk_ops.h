// Internal interface between the host entry points of the multi-token operators
// (mk_ops.cpp) and their kernels.  Every launch_* function returns the CUDA error of the
// launch; argument checks are the caller's.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mk.h"

namespace mk {

// sets the message of mk_last_error(NULL) and returns `code` (mk_host.cpp)
int op_fail(int code, const char* fmt, ...);

// Allow `kernel` that much dynamic shared memory, once per device (`done`: a bit per device).
template <class K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch `kernel` so that its prologue may run beside the end of the kernel before it on the
// stream (griddepcontrol.wait in the kernel is where it waits for that one).
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kOpPage = 16;            // tokens per cache page
constexpr int kOpMaxBatch = 65535;     // sequences of one call
constexpr int kOpMaxEntries = 65536;   // of the attention's work list: sequences x groups of nodes
constexpr int kItemUnits = 6;          // of the attention's work list: what an item counts for beside its key blocks
constexpr int kOpMaxExperts = 256;     // experts of one call (as mk_create)
constexpr int kOpMaxAccept = 512;      // accepted nodes per sequence (staged in shared memory)
constexpr int kOpMaxHalf = 64;         // head_dim / 2 at most

// The current device's own error record, int32[4] (mk_cache_pages.cu).
cudaError_t op_record(int32_t** record);

// ------------------------------------------------------------------ qk_norm_rope
struct RopeParams {
  mk_paged_kv c;
  mk_rope_args a;
  unsigned long long turns[kOpMaxHalf];  // theta^(-2i/hd) / 2pi as a 64-bit binary fraction
};
cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t st);

// ------------------------------------------------------------------ tree_attention
struct TreeParams {
  mk_paged_kv c;
  mk_tree_args a;
  int gs;          // query heads per KV head
  int npt;         // nodes per 128-row tile
  int two;         // 1: a CTA works on two row tiles at once; 0: on one, with two key streams
  int ntp;         // row-tile groups per (sequence, KV head)
  int team;        // tile groups that walk a run of keys together
  int teams;       // such teams in the grid
  int groups;      // entries of the work list per sequence
  int words;       // mask words per node
  int grid;        // CTAs
  float scale_log2;
  float* part;     // partial results: [grid][2][tiles][hd / 4][128] float4
  float2* part_ml; // [grid][2][tiles][128] (running maximum, sum)
  int* table;      // prefix sums of the work list, written for the join
};
size_t tree_workspace_bytes(const TreeParams& p);
cudaError_t launch_tree(TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t st);

// ------------------------------------------------------------------ cache pages
cudaError_t launch_copy_pages(uint8_t* k, uint8_t* v, int n_layers, long long layer_bytes, long long page_bytes,
                              const int32_t* src, const int32_t* dst, int n, cudaStream_t st);
struct CommitParams {
  mk_paged_kv c;   // k, v: the whole pools
  int n_layers, max_accept;
  const int32_t* accepted;
  int32_t* new_lens;
  int32_t* status;
};
cudaError_t launch_commit(const CommitParams& p, cudaStream_t st);

// ------------------------------------------------------------------ expert_product
struct ExpertParams {
  mk_expert_args a;
  int grid;
};
cudaError_t launch_experts(const ExpertParams& p, const CUtensorMap& tx, const CUtensorMap& tx128, const CUtensorMap& tw,
                           const CUtensorMap& tu, cudaStream_t st);

}  // namespace mk
