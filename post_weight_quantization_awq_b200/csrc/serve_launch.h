// Internal launchers of the serving operators (host side): the adapter
// product, the mixture-of-experts layer and the norms around a block.  Every
// launcher only enqueues work on `stream` and returns the launch error, if any.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "awq_device.cuh"

namespace awq {

// DevStatus flag: an adapter id outside [-1, n_adapters) (beside awq_device.cuh's kDev* bits)
constexpr uint32_t kDevBadAdapter = 1u << 4;

// Sets a kernel's dynamic shared memory limit once per device (two threads that
// come first both set it).
template <class K>
inline cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

// A kernel launched by launch_after is set up while the kernel before it on the
// stream ends; pdl_wait() returns when that one has ended with all its results
// visible, and comes before the first access to memory.  pdl_launch() lets the next
// such kernel start: called behind the block's own pdl_wait(), so that all work before
// this kernel has ended by then, and the next one may read that work's results (not this
// kernel's) before its own pdl_wait(), from L2 (ld.cg, cp.async.cg, TMA).
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), int64_t blocks, int threads, size_t smem, cudaStream_t stream,
                                const A &...args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct LoraArgs {
  const __half *X;
  int64_t T, in, ldx;
  const int32_t *qweight, *qzeros;
  const __half *scales;
  int64_t out;
  int group;
  const __half *A, *B;
  const float *c;
  const int32_t *ids;
  int rank, adapters;
  __half *Y;
  int64_t ldy;
  float *U;       // workspace: [T, rank] fp32
  DevStatus *st;
  uint32_t max_polls;
};
// Y = X W^T + c_a (X A_a^T) B_a^T; in % 64 == 0, out % 32 == 0, rank % 8 == 0.
// Up to kLoraStreamT tokens it streams the packed words; `U` then holds [T, rank] fp32.
constexpr int64_t kLoraStreamT = 64;
cudaError_t launch_lora(const LoraArgs &a, int num_sms, cudaStream_t stream);
// More tokens: `U` holds lora_prefill_ws() bytes.
size_t lora_prefill_ws(int64_t T, int64_t in, int64_t out, int rank);
cudaError_t launch_lora_prefill(const LoraArgs &a, int num_sms, cudaStream_t stream);

struct NormArgs {
  const __half *R, *V, *post, *gate, *pre;
  int64_t ldr, ldv, ldg, T, d, ldro, ldno;
  float c, eps;
  __half *R_out, *N_out;
};
cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t stream);

constexpr int kMoeMaxTokens = 64, kMoeMaxTopK = 16, kMoeMaxExperts = 256;

struct MoeArgs {
  const __half *X;
  int64_t ldx;
  const uint8_t *mask;     // [T] or NULL
  const __half *router;    // [experts, hidden]
  const int32_t *gu_q, *gu_z;
  const __half *gu_s;
  const int32_t *dn_q, *dn_z;
  const __half *dn_s;
  int T, experts, top_k, group, renormalize;
  int64_t hidden, inter;
  __half *Y;
  int64_t ldy;
  int32_t *ids;
  float *weights;
  // workspace
  DevStatus *st;           // 512 bytes cleared by the launch: status word,
  uint32_t *barrier;       // 4 counters,
  int *tok_count;          // [T] logits written
  double *logits;
  __half *H;
  float *sums, *dn_sums;        // [pairs, 2 inter]; [2 pairs, hidden]
  float *partial, *dn_partial;  // [blocks, 2, rows, 512] each
  uint32_t max_polls;
};
struct MoeLayout {
  size_t logits, H, sums, dn_sums, partial, dn_partial, end;
};
MoeLayout moe_layout(int64_t T, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k, int num_sms);
cudaError_t launch_moe(const MoeArgs &a, int num_sms, cudaStream_t stream);

}  // namespace awq
