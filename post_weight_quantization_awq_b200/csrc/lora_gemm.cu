// Low-rank adapters of many requests beside one packed projection:
//
//   Y[t][o] = RN16( sum_j X[t][j] (q - z) s  +  c_a sum_r U[t][r] B_a[o][r] ),
//   U[t][r] = sum_j X[t][j] A_a[r][j],  a = ids[t]  (-1: no adapter)
//
// Two launches.  lora_shrink_kernel computes c_a U in fp32; it lets its
// successor start at once (programmatic dependent launch), which meanwhile
// streams the packed weights and waits for U only before its epilogue.
#include <cooperative_groups.h>

#include "serve_launch.h"
#include "w4_stream.cuh"

namespace awq {
namespace {
namespace cg = cooperative_groups;
using namespace w4s;

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&y[i]));
    s = fmaf(p.x, q.x, s);
    s = fmaf(p.y, q.y, s);
  }
  return s;
}

// One warp per (token, rank row).
__global__ void __launch_bounds__(256) lora_shrink_kernel(const LoraArgs a) {
  pdl_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{};
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = i / a.rank, r = i - t * a.rank;
  if (t >= a.T) return;
  const int id = a.ids[t];
  if (id < 0 || id >= a.adapters) return;  // never read
  const uint4 *x = reinterpret_cast<const uint4 *>(a.X + t * a.ldx);
  const uint4 *w = reinterpret_cast<const uint4 *>(a.A + ((int64_t)id * a.rank + r) * a.in);
  float s = 0.0f;
  for (int64_t k = lane; k < a.in / 8; k += 32) s = dot8(__ldg(x + k), __ldg(w + k), s);
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (lane == 0) a.U[t * a.rank + r] = a.c[id] * s;
}

// A cluster of `splits` blocks covers 256 outputs x MAXTOK tokens, each block
// a range of input rows; the blocks' fp32 sums meet through distributed shared
// memory in rank order.
template <int NT, Split SP, int MAXTOK, int STAGES, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) lora_stream_kernel(const __grid_constant__ LoraArgs a,
                                                                     const int splits) {
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)(blockIdx.x % (unsigned)splits);
  const int64_t tile = blockIdx.x / (unsigned)splits;
  const int64_t t0 = (int64_t)blockIdx.y * MAXTOK;
  const int n = (int)(a.T - t0 < MAXTOK ? a.T - t0 : MAXTOK);
  Weights w{a.qweight, a.qzeros, a.scales, a.out / 8, group_shift(a.group),
            tile * 32, a.out / 8, tile * 32 + 16, a.out / 8};
  const Rows x{a.X + t0 * a.ldx, a.ldx, nullptr, n};
  // input rows of this rank, in units of 256 (128) rows so that groups stay whole
  const int64_t unit = a.in >= 512 * splits ? 256 : 128, units = (a.in + unit - 1) / unit;
  const int64_t k0 = units * rank / splits * unit;
  int64_t k1 = units * (rank + 1) / splits * unit;
  if (k1 > a.in) k1 = a.in;
  Acc<NT> acc;
  product<NT, SP, MAXTOK, STAGES>(acc, smem, w, x, (int)k0, (int)(k1 > k0 ? k1 : k0));
  float *red = reinterpret_cast<float *>(smem);
  store_sums<NT, SP>(acc, red);
  pdl_wait();  // U and the cleared status word
  if (blockIdx.x == 0) {
    for (int t = threadIdx.x; t < n; t += kThreads) {
      const int id = a.ids[t0 + t];
      if (id < -1 || id >= a.adapters) dev_fail(a.st, kDevBadAdapter, 0xE01u);
    }
  }
  cluster.sync();
  for (int i = rank * kThreads + threadIdx.x; i < n * (kTileN / 2); i += splits * kThreads) {
    const int t = i / (kTileN / 2), oo = 2 * (i % (kTileN / 2));
    const int64_t o = tile * kTileN + oo;
    if (o >= a.out) continue;
    float s0 = 0.0f, s1 = 0.0f;
    for (int s = 0; s < splits; ++s) {
      const float *p = cluster.map_shared_rank(red, s) + t * kRedPitch + oo;
      s0 += p[0];
      s1 += p[1];
    }
    const int id = a.ids[t0 + t];
    if (id >= 0 && id < a.adapters) {
      const float4 *u = reinterpret_cast<const float4 *>(a.U + (t0 + t) * a.rank);
      const uint4 *b0 = reinterpret_cast<const uint4 *>(a.B + ((int64_t)id * a.out + o) * a.rank);
      const uint4 *b1 = b0 + a.rank / 8;
      float l0 = 0.0f, l1 = 0.0f;
      for (int k = 0; k < a.rank / 8; ++k) {
        const float4 ua = u[2 * k], ub = u[2 * k + 1];
        const float uu[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
        const uint4 p = __ldg(b0 + k), q = __ldg(b1 + k);
        const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&pw[e]));
          const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&qw[e]));
          l0 = fmaf(uu[2 * e], f.x, l0);
          l0 = fmaf(uu[2 * e + 1], f.y, l0);
          l1 = fmaf(uu[2 * e], h.x, l1);
          l1 = fmaf(uu[2 * e + 1], h.y, l1);
        }
      }
      s0 += l0;
      s1 += l1;
    }
    *reinterpret_cast<__half2 *>(a.Y + (t0 + t) * a.ldy + o) = __floats2half2_rn(s0, s1);
  }
  cluster.sync();  // no block leaves while its sums are read
}

template <int NT, Split SP, int MAXTOK, int STAGES, int MINB>
cudaError_t launch_stream(const LoraArgs &a, int num_sms, cudaStream_t stream) {
  static bool done[64];
  constexpr size_t kSmem = STAGES * stage_bytes(MAXTOK);
  static_assert((size_t)MAXTOK * kRedPitch * 4 <= kSmem, "the sums reuse the ring");
  auto kernel = lora_stream_kernel<NT, SP, MAXTOK, STAGES, MINB>;
  cudaError_t e = allow_smem(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.out + kTileN - 1) / kTileN, ttiles = (a.T + MAXTOK - 1) / MAXTOK;
  int64_t s = (int64_t)num_sms * MINB / (tiles * ttiles);
  const int64_t most = (a.in + 127) / 128;
  s = s > 8 ? 8 : s;
  s = s > most ? most : s;
  s = s < 1 ? 1 : s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)s;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * s), (unsigned)ttiles);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, (int)s);
}
}  // namespace

cudaError_t launch_lora(const LoraArgs &a, int num_sms, cudaStream_t stream) {
  const int64_t blocks = (a.T * a.rank + 7) / 8;
  lora_shrink_kernel<<<(unsigned)blocks, 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.T <= 8) return launch_stream<1, Split::kK, 8, 4, 2>(a, num_sms, stream);
  if (a.T <= 16) return launch_stream<2, Split::kK, 16, 4, 2>(a, num_sms, stream);
  if (a.T <= 32) return launch_stream<2, Split::kTok, 32, 3, 2>(a, num_sms, stream);
  if (a.T <= 48) return launch_stream<3, Split::kTok, 48, 4, 1>(a, num_sms, stream);
  return launch_stream<4, Split::kTok, 64, 4, 1>(a, num_sms, stream);
}

}  // namespace awq
