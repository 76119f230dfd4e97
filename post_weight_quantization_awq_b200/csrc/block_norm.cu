// A block's exit and the next block's entrance in one pass over a token row:
//
//   v' = v rsqrt(mean v^2 + eps) post     (or v, without a norm after the block)
//   r' = r + c gate v'                    (gate: per channel, per token, or 1)
//   n  = r' rsqrt(mean r'^2 + eps) pre
//
// with r' stored as the next residual and n as the next block's input; pre is
// the norm weight into which awq_fold_inv_scale folds 1/s.
//
// Bytes: r and v read once, r' and n written once (8 bytes an element, 2 more
// with a per-token gate); everything between stays in registers, in fp32, and
// n is taken from the unrounded r'.  A row belongs to one team of threads (a
// warp for short rows, up to a block of 1024 for long ones), VPT 16-byte
// vectors to a thread, so both reductions are a warp butterfly and, past one
// warp, one exchange through shared memory.  Every element is read before it
// is written by the thread that owns it, so r' may overwrite r and n may
// overwrite v.
//
// Measured: 16384 rows of 4096 in 82-83 us = 6.5 TB/s, bound by HBM; 333 rows of 5120
// with a gate by token 4.5 us, one row 2.3 us, bound by latency.
#include "serve_launch.h"

namespace awq {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Sum over the row's team.  `red` has one slot per warp; two buffers used in
// turn make one barrier enough.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float *red) {
  v = warp_sum(v);
  if (TEAM == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < TEAM / 32 ? red[lane] : 0.0f;
  return warp_sum(v);
}

__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ROWS rows per block, TEAM threads per row.
template <int TEAM, int ROWS, int VPT>
__global__ void __launch_bounds__(TEAM *ROWS) block_norm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  pdl_wait();
  const int lane = threadIdx.x % TEAM;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TEAM;
  if (row >= a.T) return;  // ROWS > 1 only with TEAM = 32: no barrier is missed
  const int nvec = (int)(a.d / 8);
  const float inv_d = 1.0f / (float)a.d;
  const uint4 *R = reinterpret_cast<const uint4 *>(a.R + row * a.ldr);
  const uint4 *V = a.V ? reinterpret_cast<const uint4 *>(a.V + row * a.ldv) : nullptr;
  uint4 rv[VPT], vv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * TEAM;
    rv[i] = vv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < nvec && AWQ_IN_BOUNDS(row < a.T && 8 * (c + 1) <= a.d, 0xB080u)) {
      rv[i] = R[c];
      if (V) vv[i] = V[c];
    }
  }
  float f = a.c;  // c, times v's norm factor
  if (a.post) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float x[8];
      unpack8(vv[i], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
    }
    s = team_sum<TEAM>(s, red[0]);
    f = rsqrtf(fmaf(s, inv_d, a.eps));
  }
  const uint4 *G = a.gate ? reinterpret_cast<const uint4 *>(a.gate + row * a.ldg) : nullptr;
  float r[VPT][8];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * TEAM;
    unpack8(rv[i], r[i]);
    if (V && c < nvec) {
      float x[8], w[8];
      unpack8(vv[i], x);
      if (a.post) {
        unpack8(__ldg(reinterpret_cast<const uint4 *>(a.post) + c), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = a.c * (x[k] * f * w[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = a.c * x[k];
      }
      if (G) {
        unpack8(G[c], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= w[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] += x[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(r[i][k], r[i][k], s);
    if (a.R_out && c < nvec && AWQ_IN_BOUNDS(row < a.T && 8 * (c + 1) <= a.d, 0xB081u))
      reinterpret_cast<uint4 *>(a.R_out + row * a.ldro)[c] = pack8(r[i]);
  }
  if (!a.N_out) return;
  s = team_sum<TEAM>(s, red[1]);
  const float h = rsqrtf(fmaf(s, inv_d, a.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * TEAM;
    if (c < nvec && AWQ_IN_BOUNDS(row < a.T && 8 * (c + 1) <= a.d, 0xB082u)) {
      float w[8];
      if (a.pre)
        unpack8(__ldg(reinterpret_cast<const uint4 *>(a.pre) + c), w);
      else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 1.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] *= r[i][k] * h;
      reinterpret_cast<uint4 *>(a.N_out + row * a.ldno)[c] = pack8(w);
    }
  }
}

template <int TEAM, int ROWS, int VPT>
cudaError_t go(const NormArgs &a, cudaStream_t stream) {
  return launch_after(block_norm_kernel<TEAM, ROWS, VPT>, (a.T + ROWS - 1) / ROWS, TEAM * ROWS, 0, stream, a);
}
}  // namespace

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t stream) {
  const int64_t nvec = a.d / 8;
  if (nvec <= 32) return go<32, 4, 1>(a, stream);
  if (nvec <= 64) return go<32, 4, 2>(a, stream);
  if (nvec <= 128) return go<128, 1, 1>(a, stream);
  if (nvec <= 256) return go<256, 1, 1>(a, stream);
  if (nvec <= 512) return go<256, 1, 2>(a, stream);
  if (nvec <= 1024) return go<512, 1, 2>(a, stream);
  if (nvec <= 2048) return go<1024, 1, 2>(a, stream);
  if (nvec <= 4096) return go<1024, 1, 4>(a, stream);
  return cudaErrorInvalidValue;
}

AWQ_BOUNDS_READER(bounds_status_norm)

}  // namespace awq
