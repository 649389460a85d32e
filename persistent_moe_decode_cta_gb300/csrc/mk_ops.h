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

// Allow `kernel` clusters of more than 8 blocks, likewise.
template <class K>
cudaError_t allow_wide_clusters(K* kernel, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Clusters of `ctas` blocks that can run at once, one block an SM (`known`: by device, 0: not asked for yet).  Fewer than the SMs
// divided by their size: a cluster lies within a group of SMs that share a switch.
template <class K>
cudaError_t active_clusters(K* kernel, int ctas, int threads, size_t smem, std::atomic<int> (&known)[64], int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *n = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
  if (*n > 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
  if (e == cudaSuccess && dev < 64) known[dev].store(*n, std::memory_order_release);
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

// The same in clusters of `ctas` blocks.
template <class... P, class... A>
cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int ctas, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
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
  // Results as sums of two bf16 rows: where the second part of each lies, in elements behind the first (0: one rounded row), and
  // whether the rows of x come in such pairs, whose products are added.
  int64_t rest;
  int pairs;
};
cudaError_t launch_experts(const ExpertParams& p, const CUtensorMap& tx, const CUtensorMap& tx128, const CUtensorMap& tw,
                           const CUtensorMap& tu, cudaStream_t st);

// ------------------------------------------------------------------ linear
// One expert that has every row, and what happens to its results.  (mk_experts.cu)
struct LinearEpi {
  const uint16_t* bias;      // [n] or NULL
  const uint16_t* residual;  // [m][n] or NULL
  int64_t residual_stride;
  int act, out_float;
  int vec;                   // residual and out can be read and written four values at a time
  int tile_rows;             // of a tile, at most (a multiple of 32)
};
// The same for few rows (mk_linear.cu).
struct SplitParams {
  LinearEpi epi;
  void* out;
  int64_t out_stride;
  int32_t* status;
  int m, n, k;
  // from split_shape: row tiles of `rows` (a multiple of 16, also the copies' height), outputs' tiles, columns' chunks of 64 and how
  // many slices they are cut into
  int rows, box, w_tiles, r_tiles, chunks, slices, stages, tmem_cols, ring, smem;
  int long_sums;  // float32 results of more than 512 columns a slice
};
cudaError_t split_shape(SplitParams& p, int sms, bool* fits);
cudaError_t launch_linear_split(const SplitParams& p, const CUtensorMap& tx, const CUtensorMap& tw, cudaStream_t st);
cudaError_t launch_linear_pairs(const ExpertParams& p, const LinearEpi& epi, const CUtensorMap& tx, const CUtensorMap& tx128,
                                const CUtensorMap& tw, cudaStream_t st);

// ------------------------------------------------------------------ moe_layer
constexpr int kMoeTokens = 256;   // tokens of one call
constexpr int kMoeTopK = 16;
constexpr int kMoeFew = 8;        // ... of both products in one kernel
constexpr int kMoeWidest = 8192;  // d_model: the tokens stay in shared memory
struct MoeParams {
  mk_moe_args a;
  int grid;          // CTAs of the products
  int groups;        // few tokens: groups of eight rows of h an expert, else 0
  int width, slots;  // few tokens: output columns of a CTA's block, slots of a warp's ring
  int vec;           // residual and out can be read and written four values at a time
  int32_t* ids;      // the caller's or the workspace's
  float* weights;
  uint16_t* h;       // [moe_h_rows][d_ff] bf16: silu(gate) * up, of few tokens times c, as sums of two values
  uint32_t* sync;    // counters, zeroed by the router
  // more tokens
  int32_t *offsets, *offsets_h, *rows, *places;  // an expert's rows, and of h, two each; the token of a row; the row of a token's j-th expert
  float* y;          // [rows][d_model]
};
struct MoeMaps {
  CUtensorMap gate, up, down, h;
};
size_t moe_workspace_bytes(const mk_moe_args& a);
long long moe_h_rows(const mk_moe_args& a);
void moe_shape(MoeParams& p);  // fills what follows `grid`
cudaError_t launch_moe_router(const MoeParams& p, cudaStream_t st);
cudaError_t launch_moe_few(const MoeParams& p, const MoeMaps& m, cudaStream_t st);
cudaError_t launch_moe_sum(const MoeParams& p, cudaStream_t st);

// ------------------------------------------------------------------ verify_nodes
constexpr int kVerifyVocab = 1 << 18;
struct VerifyParams {
  mk_verify_args a;
  int grid;        // SMs
  float4* parts;   // [batch][n_nodes][pieces] (largest, sum, index of the largest) of a piece of a row
  int pieces;      // of a row
};
size_t verify_workspace_bytes(const mk_verify_args& a);
cudaError_t launch_verify(VerifyParams& p, cudaStream_t st);

}  // namespace mk
