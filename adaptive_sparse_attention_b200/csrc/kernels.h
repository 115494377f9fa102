// kernels.h -- host-side launchers of the entmax attention kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "common.cuh"

namespace ea {

// dtype: 0 = fp32, 1 = bf16.  Each returns cudaSuccess or the launch error.
cudaError_t launch_tau_simt(const Problem& P, int dtype, cudaStream_t s);
cudaError_t launch_tau_fallback(const Problem& P, int dtype, int num_ctas, cudaStream_t s);
cudaError_t launch_out_simt(const Problem& P, int dtype, cudaStream_t s);

// Tensor-core (tcgen05) kernels, bf16 only, d in {64, 128}.
cudaError_t launch_tau_tc(const Problem& P, cudaStream_t s);
// Multi-sweep tau search on the tensor cores for the overflow queue (one CTA per SM at most).
cudaError_t launch_tau_tc_fallback(const Problem& P, int num_ctas, cudaStream_t s);
cudaError_t launch_out_tc(const Problem& P, cudaStream_t s);
// Output of the query tiles that are not pending, from the support lists the tau pass recorded
// (bf16 values, d in {64, 128}).
cudaError_t launch_out_support(const Problem& P, cudaStream_t s);
// Warm-up keys of the tensor-core tau pass (P.norms, P.warm); nothing when P.warm_levels == 0.
cudaError_t launch_warm(const Problem& P, cudaStream_t s);

// Backward pass on the CUDA cores: delta (fp32 per query row), then dq (fp32, written) and dk,
// dv (fp32, accumulated: zero them first).  g is the upstream gradient in the input dtype.
cudaError_t launch_bwd(const Problem& P, int dtype, const void* g, float* delta, float* dq,
                       float* dk, float* dv, cudaStream_t s);

// FP8 screen of the tau pass (screen.cu, bf16, d = 128): e4m3 copies of q (per row) and k (per
// 128-key tile) with their scales and error norms, then per query tile the ascending list of key
// tiles the bf16 tau pass must visit and its count.  q8 [q rows][128] bytes, qst float4 [q rows],
// k8 [kv rows][128] bytes, kst float4 [(B or 1) Hkv slots], list [tiles][nkt_max], count [tiles].
cudaError_t launch_screen(const Problem& P, void* q8, void* qst, void* k8, void* kst, int* list,
                          int* count, cudaStream_t s);

// Entmax block routing over chunk summaries (pi fp32 [B, Hq, T, nc], tau fp32 [B, Hq, T]);
// with scores_ready the rows of pi already hold z = (alpha - 1) scaling q . sigma / sqrt(d).
cudaError_t launch_route_chunks(const void* q, const void* sig, float* pi, float* tau, int B,
                                int Hq, int Hkv, int T, int d, int nc, int chunk, float alpha,
                                int n_iter, int causal, int diag, float scaling, int dtype,
                                int scores_ready, cudaStream_t s);
// z = zscale q . sigma for every (query row, chunk) into z [B, Hq, T, nc] on the tensor cores
// (bf16, d in {64, 128}, q and sig 16-byte aligned); status: the device status word.
cudaError_t launch_route_scores_tc(const void* q, const void* sig, float* z, int B, int Hq,
                                   int Hkv, int T, int d, int nc, float zscale, int* status,
                                   cudaStream_t s);

// Row-wise alpha-entmax of a [rows, n] matrix x (row stride ldx elements) into p (row stride
// ldp); dtype 0 = fp32, 1 = bf16 for both x and p; tau may be null.
cudaError_t launch_entmax_rows(const void* x, int64_t ldx, void* p, int64_t ldp, float* tau,
                               int rows, int n, float alpha, int n_iter, int dtype,
                               cudaStream_t s);

// Paged key-value cache (paged.cu, decode.cuh).  Its kernels are a few microseconds each and follow
// one another in a decoding step, so they are launched with programmatic stream serialization: a
// kernel's blocks may be set up as soon as all blocks of the kernel before it in the stream have
// ended, and wait (serial_wait, before their first access to memory) until that kernel's writes are
// visible.  An append of 64 tokens takes 3.2 us instead of 4.1, a request of 1000 tokens 8.6
// instead of 10.6, four ragged ones on the split kernels 36.4 instead of 40.6.  No kernel lets the next one be set up earlier
// (griddepcontrol.launch_dependents): the early blocks crowd the SMs that are free first, which
// cost the page tables of 1000 requests 11.4 instead of 6.8 us and 64 requests of 16384 tokens 266
// instead of 261.
template <typename K, typename... A>
cudaError_t launch_serial(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                          const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void serial_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif
// Allows a kernel more than 48 KB of shared memory, once per device and always the most that any of
// its launches takes: the limit is the process's, and another thread may be about to launch with it.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

constexpr int kMaxRequests = 8192;  // prefix sums over the batch live in shared memory

// Block tables and slot maps of a step (entmax_attn_page_tables).
struct PageTables {
  const int32_t* lens;        // [B] tokens held
  const int32_t* new_lens;    // [B] tokens to add
  const int32_t* free_pages;  // [n_free]
  const int32_t* free_start;  // [1] first free entry not yet taken
  int32_t* tables;            // [B][table_stride]
  int64_t table_stride;
  int64_t table_tokens;       // tokens a table row addresses (W page_size)
  int64_t* slots;             // [n_new], padded: [B][n_new]
  int32_t* lens_out;          // [B]
  int32_t* cu_new;            // [B + 1]
  int32_t* free_next;         // [1]
  int n_free, B, page_size, n_new, padded;
};
cudaError_t launch_page_tables(const PageTables& P, cudaStream_t s);

// New tokens' keys and values into their slots (entmax_attn_paged_append); strides in bytes.
struct PagedAppend {
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  const int64_t* slots;
  int* status;
  int64_t stride_b, stride_h, stride_t;
  int64_t page_stride, head_stride, slot_stride;
  int64_t n_slots;  // num_pages page_size
  int n_tokens, T, Hkv, page_size;
};
cudaError_t launch_paged_append(const PagedAppend& P, int row_bytes, cudaStream_t s);

// One-token attention over the paged cache (entmax_attn_decode); strides in elements.
constexpr int kDecodeScoreWarps = 148 * 16;  // warps of the score kernel: 16 on each SM
// Keys of a request: key numbers, rounded up to units of 16 and by what the join reads ahead, fit an
// int.
constexpr int kMaxKeys = 0x7fffffff - 4095;
struct DecodeProblem {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* tables;
  const int32_t* lens;
  void* out;
  float* tau;
  int* status;
  int64_t q_stride_b, q_stride_h;
  int64_t page_stride, head_stride, slot_stride;
  int64_t table_stride;
  int num_pages, page_size;
  int B, Hq, Hkv, G, max_len;
  int head_blocks, heads_per_block;  // query heads of a kv head are scored 8 or 16 at a time
  float alpha, beta, c;
  int score_warps;
  int cluster;      // blocks per cluster of the one-launch kernel; 0 = the split kernels
  int join_blocks;  // blocks of 8 warps per head of the split kernels' join (1 or 4); 0 = a warp
  // workspace
  int32_t* pre;         // [B + 1] prefix sums of the requests' 16-key units
  int2* parts;          // (count, max bits) [heads_per_block][score_warps + groups], groups = B Hkv
                        // head_blocks; the cluster kernel keeps its own in shared memory
  int2* cand;           // [B][Hq][cand_stride] (z bits, key)
  int64_t cand_stride;  // max_len rounded up to 16
};
cudaError_t launch_decode_bf16_64(const DecodeProblem& P, cudaStream_t s);
cudaError_t launch_decode_bf16_128(const DecodeProblem& P, cudaStream_t s);
cudaError_t launch_decode_fp32_64(const DecodeProblem& P, cudaStream_t s);
cudaError_t launch_decode_fp32_128(const DecodeProblem& P, cudaStream_t s);

// Records e as the string entmax_attn_last_cuda_error reports and returns ENTMAX_ATTN_ECUDA.
int record_cuda_error(cudaError_t e);

inline int beta_kind(float beta) {
  if (beta == 1.f) return kBetaOne;
  if (beta == 2.f) return kBetaTwo;
  if (fabsf(beta - 3.f) <= kNearIntFrac) return kBetaNear3;
  return kBetaGeneral;
}

}  // namespace ea
