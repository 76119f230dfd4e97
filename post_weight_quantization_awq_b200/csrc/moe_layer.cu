// A whole mixture-of-experts layer on packed 4-bit experts for a few tokens,
// one cooperative kernel:
//
//   l = x Wr^T;  the k largest logits (ties to the lowest expert), p = softmax
//   over all experts (divided by the chosen ones' sum when renormalize);
//   y = sum_k p_k down_e( RN16( silu(x gate_e) * (x up_e) ) )
//
// The layer is bound by reading the met experts' words once.  Phases, between
// grid barriers:
//   router   a warp per (token, expert): fp32 products summed in fp64, so that
//            a choice next to a border is the definition's;
//   choice   every block redoes the top-k and the experts' token lists in
//            shared memory (nothing to wait for a second time);
//   gate|up  tiles of 128 gate and the same 128 up outputs of one expert over
//            its tokens, in units of 128 input rows.  The units of all tiles
//            are dealt out evenly and in order, so a block computes the end of
//            one tile, whole tiles, and the start of another; tiles that are
//            split meet as fp32 partial sums, added in block order by the last
//            block to arrive, which also applies silu(g) u;
//   down     tiles of 256 outputs whose inner axis runs over all met experts;
//            each expert's sums are weighted with p in fp32 and added to the
//            block's rows of the tile;
//   combine  the blocks' rows of a tile added in block order, one rounding.
// Sums are added in an order fixed by the sizes and the routing alone.
#include <cuda_runtime.h>

#include "serve_launch.h"
#include "w4_stream.cuh"

namespace awq {
namespace {
using namespace w4s;

constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMaxSeg = kMoeMaxExperts + kMaxPairs / 32;  // (expert, up to 32 tokens) entries

struct MoeShared {
  int16_t id[kMaxPairs];     // chosen expert of (token, slot), -1: masked row
  float wt[kMaxPairs];
  int16_t pair[kMaxPairs];   // the entries' (token, slot) pairs, expert by expert
  int row[32];               // rows of X or H of the running product
  int16_t count[kMoeMaxExperts];
  int16_t seg_expert[kMaxSeg], seg_first[kMaxSeg], seg_n[kMaxSeg];
  int n_seg;
  int flag;
};

// All blocks meet (counter from 0 to gridDim.x); false when the wait ran out.
__device__ __forceinline__ bool grid_barrier(uint32_t *counter, MoeShared *sh, DevStatus *st, uint32_t max_polls,
                                             uint32_t site) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    uint32_t v;
    asm volatile("atom.add.release.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(counter) : "memory");
    const uint64_t t0 = global_ns(), limit = (uint64_t)max_polls * 64u;
    bool ok = true;
    for (;;) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= gridDim.x) break;
      if (global_ns() - t0 > limit) {
        dev_fail(st, kDevTimeout, site);
        ok = false;
        break;
      }
    }
    __threadfence();
    sh->flag = ok;
  }
  __syncthreads();
  return sh->flag != 0;
}

__device__ __forceinline__ double dot8d(uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&y[i]));
    s = fmaf(p.x, q.x, s);
    s = fmaf(p.y, q.y, s);
  }
  return (double)s;
}

__device__ void router(const MoeArgs &a) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32);
  for (int i = blockIdx.x + gridDim.x * (threadIdx.x >> 5); i < a.T * a.experts; i += warps) {
    const int t = i / a.experts, e = i - t * a.experts;
    if (a.mask && !a.mask[t]) continue;
    const uint4 *x = reinterpret_cast<const uint4 *>(a.X + t * a.ldx);
    const uint4 *w = reinterpret_cast<const uint4 *>(a.router + (int64_t)e * a.hidden);
    double s = 0.0;
    for (int k = lane; k < a.hidden / 8; k += 32) s += dot8d(__ldg(x + k), __ldg(w + k));
#pragma unroll
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lane == 0) a.logits[i] = s + 0.0;  // -0 becomes 0: the order below is of bit patterns
  }
}

// Top-k of one token by a warp; a lane holds experts lane, lane + 32, ...
__device__ void choose(const MoeArgs &a, MoeShared *sh, int t) {
  const int lane = threadIdx.x & 31;
  constexpr int PER = kMoeMaxExperts / 32;
  if (a.mask && !a.mask[t]) {
    if (lane < a.top_k) {
      sh->id[t * a.top_k + lane] = -1;
      sh->wt[t * a.top_k + lane] = 0.0f;
    }
    return;
  }
  // fp64 bit patterns in an order-preserving form; NaN sorts by its bits
  long long key[PER];
  double top = -INFINITY;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    key[j] = LLONG_MIN;
    if (e < a.experts) {
      const double l = __ldcg(a.logits + (int64_t)t * a.experts + e);
      const long long b = __double_as_longlong(l);
      key[j] = b ^ ((b >> 63) & 0x7fffffffffffffffLL);
      top = fmax(top, l);
    }
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, m));
  // exp(l - top): the fp64 difference as two floats, exp of the first exact to
  // fp32 and the second's factor 1 + lo
  float sum = 0.0f;
  auto weight = [&](long long kk) {
    const long long b = kk ^ ((kk >> 63) & 0x7fffffffffffffffLL);
    const double d = __longlong_as_double(b) - top;
    const float hi = (float)d;
    const float ex = expf(hi);
    return fmaf(ex, isfinite(hi) ? (float)(d - (double)hi) : 0.0f, ex);
  };
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (lane + 32 * j < a.experts) sum += weight(key[j]);
#pragma unroll
  for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  uint32_t taken = 0;
  float mine = 0.0f, chosen = 0.0f;
  int my_id = -1;
  for (int s = 0; s < a.top_k; ++s) {
    long long best = LLONG_MIN;
    int at = 0x7fff;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 32 * j;
      if (e < a.experts && !((taken >> j) & 1u) && (at == 0x7fff || key[j] > best)) {
        best = key[j];
        at = e;
      }
    }
    // largest high word, then low word, then lowest expert
    const int hi = (int)(best >> 32);
    const bool have = at != 0x7fff;
    const int mhi = __reduce_max_sync(0xffffffffu, have ? hi : INT_MIN);
    const bool in1 = have && hi == mhi;
    const uint32_t mlo = __reduce_max_sync(0xffffffffu, in1 ? (uint32_t)best : 0u);
    const bool in2 = in1 && (uint32_t)best == mlo;
    const uint32_t e = __reduce_min_sync(0xffffffffu, in2 ? (uint32_t)at : 0x7fffu);
    if ((e & 31u) == (uint32_t)lane) taken |= 1u << (e >> 5);
    const long long kk = ((long long)mhi << 32) | (long long)mlo;
    const float w = weight(kk);
    chosen += w;
    if (lane == s) {
      mine = w;
      my_id = (int)e;
    }
  }
  if (lane < a.top_k) {
    sh->id[t * a.top_k + lane] = (int16_t)my_id;
    sh->wt[t * a.top_k + lane] = mine / (a.renormalize ? chosen : sum);
  }
}

// The experts' token lists, and the entries (expert, at most 32 tokens).
__device__ void make_lists(const MoeArgs &a, MoeShared *sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.T * a.top_k;
  for (int e = warp; e < a.experts; e += kThreads / 32) {
    int n = 0;
    for (int c = 0; c < pairs; c += 32) n += __popc(__ballot_sync(0xffffffffu, c + lane < pairs && sh->id[c + lane] == e));
    if (lane == 0) sh->count[e] = (int16_t)n;
  }
  __syncthreads();
  if (warp == 0) {  // first pair of each expert and its entries
    int first = 0, segs = 0;
    for (int c = 0; c < a.experts; c += 32) {
      const int n = c + lane < a.experts ? sh->count[c + lane] : 0;
      const int m = (n + 31) / 32;
      int pn = n, pm = m;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, pn, d), v = __shfl_up_sync(0xffffffffu, pm, d);
        if (lane >= d) {
          pn += u;
          pm += v;
        }
      }
      for (int j = 0; j < m; ++j) {
        const int at = segs + pm - m + j;
        sh->seg_expert[at] = (int16_t)(c + lane);
        sh->seg_first[at] = (int16_t)(first + pn - n + 32 * j);
        sh->seg_n[at] = (int16_t)(n - 32 * j < 32 ? n - 32 * j : 32);
      }
      if (c + lane < a.experts) sh->count[c + lane] = (int16_t)(first + pn - n);  // now: first pair
      first += __shfl_sync(0xffffffffu, pn, 31);
      segs += __shfl_sync(0xffffffffu, pm, 31);
    }
    if (lane == 0) sh->n_seg = segs;
  }
  __syncthreads();
  for (int e = warp; e < a.experts; e += kThreads / 32) {
    int at = sh->count[e];
    for (int c = 0; c < pairs; c += 32) {
      const bool hit = c + lane < pairs && sh->id[c + lane] == e;
      const uint32_t b = __ballot_sync(0xffffffffu, hit);
      if (hit) sh->pair[at + __popc(b & ((1u << lane) - 1u))] = (int16_t)(c + lane);
      at += __popc(b);
    }
  }
  __syncthreads();
}

// red[token][output] of the tile over rows [k0, k1), n tokens.
template <int NT>
__device__ __forceinline__ void tile_sums(uint8_t *smem, const Weights &w, const Rows &x, int k0, int k1) {
  float *red = reinterpret_cast<float *>(smem);
  Acc<NT> acc;
  if (NT == 1 || x.n <= 16) {
    product<NT, Split::kK, NT * 8, 4>(acc, smem, w, x, k0, k1);
    store_sums<NT, Split::kK>(acc, red);
  } else {
    product<NT, Split::kTok, 2 * NT * 8, 3>(acc, smem, w, x, k0, k1);
    store_sums<NT, Split::kTok>(acc, red);
  }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Units of a phase dealt out evenly: block b takes [b quota, (b + 1) quota).
__device__ __forceinline__ int64_t quota_of(int64_t units, int64_t per_tile) {
  int64_t q = (units + gridDim.x - 1) / gridDim.x;
  q = (q + 1) / 2 * 2;  // both K halves of a block busy
  return q < 1 ? 1 : (q > per_tile && units / per_tile <= gridDim.x ? per_tile : q);
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 2) moe_kernel(const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  MoeShared *sh = reinterpret_cast<MoeShared *>(smem + kMoeRing);
  const int tid = threadIdx.x;
  DevStatus *st = a.st;
  const int shift = group_shift(a.group);
  const int64_t itiles = (a.inter + 127) / 128, htiles = (a.hidden + kTileN - 1) / kTileN;
  const int64_t kgh = (a.hidden + 127) / 128, kgi = (a.inter + 127) / 128;

  // counters of split gate|up tiles
  for (int64_t i = blockIdx.x * (int64_t)kThreads + tid; i < a.max_seg * itiles; i += (int64_t)gridDim.x * kThreads)
    a.tile_count[i] = 0;
  router(a);
  if (!grid_barrier(a.barrier + 0, sh, st, a.max_polls, 0xE10u)) return;
  for (int t = tid >> 5; t < a.T; t += kThreads / 32) choose(a, sh, t);
  __syncthreads();
  make_lists(a, sh);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.T * a.top_k; i += kThreads) {
      a.ids[i] = sh->id[i];
      a.weights[i] = sh->wt[i];
    }
  const int n_seg = sh->n_seg;

  // ---------------------------------------------------------------- gate|up
  {
    const int64_t units = n_seg * itiles * kgh, quota = quota_of(units, kgh);
    int64_t u = (int64_t)blockIdx.x * quota;
    const int64_t u_end = u + quota < units ? u + quota : units;
    float *red = reinterpret_cast<float *>(smem);
    const int64_t wo = 2 * a.inter / 8;
    while (u < u_end) {
      const int64_t tile = u / kgh, g0 = u - tile * kgh;
      const int64_t g1 = g0 + (u_end - u) < kgh ? g0 + (u_end - u) : kgh;
      const int s = (int)(tile / itiles);
      const int64_t it = tile - s * itiles;
      const int e = sh->seg_expert[s], p0 = sh->seg_first[s], n = sh->seg_n[s];
      __syncthreads();
      if (tid < n) sh->row[tid] = sh->pair[p0 + tid] / a.top_k;
      __syncthreads();
      Weights w{a.gu_q + e * a.hidden * wo, a.gu_z + e * (a.hidden / a.group) * wo,
                a.gu_s + e * (a.hidden / a.group) * wo * 8, wo, shift, it * 16, wo / 2, wo / 2 + it * 16, wo};
      Rows x{a.X, a.ldx, sh->row, n};
      const int k1 = (int)(g1 * 128 < a.hidden ? g1 * 128 : a.hidden);
      tile_sums<NT>(smem, w, x, (int)g0 * 128, k1);
      bool done = true;
      const int64_t b0 = tile * kgh / quota, b1 = ((tile + 1) * kgh - 1) / quota;  // the tile's blocks
      const int rows = NT == 1 ? 8 : 32;
      if (b0 != b1) {
        float *slot = a.partial + ((int64_t)blockIdx.x * 2 + (g0 == 0)) * rows * kTileN;
        for (int t = 0; t < n; ++t) slot[t * kTileN + tid] = red[t * kRedPitch + tid];
        __threadfence();
        __syncthreads();
        if (tid == 0) sh->flag = atomicAdd(a.tile_count + tile, 1) == (int)(b1 - b0);
        __syncthreads();
        done = sh->flag != 0;
        if (done) {
          __threadfence();
          for (int t = 0; t < n; ++t) {
            float v = 0.0f;
            for (int64_t b = b0; b <= b1; ++b)
              v += __ldcg(a.partial + (b * 2 + (b == b0)) * rows * kTileN + t * kTileN + tid);
            red[t * kRedPitch + tid] = v;
          }
          __syncthreads();
        }
      }
      if (done)
        for (int i = tid; i < n * 128; i += kThreads) {
          const int t = i >> 7, c = i & 127;
          if (it * 128 + c < a.inter)
            a.H[(int64_t)sh->pair[p0 + t] * a.inter + it * 128 + c] =
                __float2half_rn(silu_mul(red[t * kRedPitch + c], red[t * kRedPitch + 128 + c]));
        }
      u += g1 - g0;
    }
  }
  if (!grid_barrier(a.barrier + 1, sh, st, a.max_polls, 0xE11u)) return;

  // ------------------------------------------------------------------- down
  const int64_t per_tile = n_seg * kgi, units = htiles * per_tile;
  const int64_t quota = per_tile ? quota_of(units, per_tile) : 1;
  {
    int64_t u = (int64_t)blockIdx.x * quota;
    const int64_t u_end = u + quota < units ? u + quota : units;
    const float *red = reinterpret_cast<const float *>(smem);
    const int64_t wo = a.hidden / 8;
    float *slot = nullptr;
    int64_t cur = -1;
    while (u < u_end) {
      const int64_t tile = u / per_tile, in_tile = u - tile * per_tile;
      if (tile != cur) {  // this block's rows of the tile: thread tid owns column tid
        cur = tile;
        slot = a.partial + ((int64_t)blockIdx.x * 2 + (in_tile == 0)) * a.T * kTileN;
        for (int t = 0; t < a.T; ++t) slot[t * kTileN + tid] = 0.0f;
      }
      const int s = (int)(in_tile / kgi);
      const int64_t g0 = in_tile - s * kgi;
      const int64_t g1 = g0 + (u_end - u) < kgi ? g0 + (u_end - u) : kgi;
      const int e = sh->seg_expert[s], p0 = sh->seg_first[s], n = sh->seg_n[s];
      __syncthreads();
      if (tid < n) sh->row[tid] = sh->pair[p0 + tid];
      __syncthreads();
      Weights w{a.dn_q + e * a.inter * wo, a.dn_z + e * (a.inter / a.group) * wo,
                a.dn_s + e * (a.inter / a.group) * wo * 8, wo, shift, tile * 32, wo, tile * 32 + 16, wo};
      Rows x{a.H, a.inter, sh->row, n};
      const int k1 = (int)(g1 * 128 < a.inter ? g1 * 128 : a.inter);
      tile_sums<NT>(smem, w, x, (int)g0 * 128, k1);
      for (int t = 0; t < n; ++t) {
        const int p = sh->pair[p0 + t];
        float *d = slot + (p / a.top_k) * kTileN + tid;
        *d = fmaf(sh->wt[p], red[t * kRedPitch + tid], *d);
      }
      u += g1 - g0;
    }
  }
  if (!grid_barrier(a.barrier + 2, sh, st, a.max_polls, 0xE12u)) return;

  // ---------------------------------------------------------------- combine
  const int64_t half = a.hidden / 2;
  for (int64_t i = blockIdx.x * (int64_t)kThreads + tid; i < a.T * half; i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / half, o = 2 * (i - t * half), tile = o / kTileN;
    float2 v = make_float2(0.0f, 0.0f);
    if (units) {
      const int64_t b0 = tile * per_tile / quota, b1 = ((tile + 1) * per_tile - 1) / quota;
      for (int64_t b = b0; b <= b1; ++b) {
        // a block that starts inside the tile uses its first slot for it
        const float2 p = __ldcg(reinterpret_cast<const float2 *>(
            a.partial + ((b * 2 + (b * quota <= tile * per_tile)) * a.T + t) * kTileN + (o - tile * kTileN)));
        v.x += p.x;
        v.y += p.y;
      }
    }
    *reinterpret_cast<__half2 *>(a.Y + t * a.ldy + o) = __floats2half2_rn(v.x, v.y);
  }
}

template <int NT>
cudaError_t go(const MoeArgs &a, int blocks, cudaStream_t stream) {
  static bool done[64];
  cudaError_t e = allow_smem(moe_kernel<NT>, kMoeRing + sizeof(MoeShared), done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMoeRing + sizeof(MoeShared);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel<NT>, a);
}

static_assert(kMoeRing >= 4 * stage_bytes(16) && kMoeRing >= 3 * stage_bytes(32), "ring");
static_assert(32 * kRedPitch * 4 <= kMoeRing, "the sums reuse the ring");
static_assert(2 * (kMoeRing + sizeof(MoeShared) + 1024) <= 233472, "two blocks per SM");
}  // namespace

cudaError_t launch_moe(const MoeArgs &a, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(a.st, 0, 256, stream);  // status word and barrier counters
  if (e != cudaSuccess) return e;
  return a.T <= 8 ? go<1>(a, 2 * num_sms, stream) : go<2>(a, 2 * num_sms, stream);
}

MoeLayout moe_layout(int64_t T, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k, int num_sms) {
  MoeLayout l;
  const int64_t pairs = T * top_k;
  l.max_seg = (experts < pairs ? experts : pairs) + pairs / 32;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  size_t off = 256;
  l.logits = off;
  off = up(off + sizeof(double) * (size_t)(T * experts));
  l.tile_count = off;
  off = up(off + sizeof(int) * (size_t)(l.max_seg * ((inter + 127) / 128)));
  l.H = off;
  off = up(off + sizeof(__half) * (size_t)(pairs * inter));
  l.partial = off;
  const int64_t rows = i64max_(T, T <= 8 ? 8 : 32);
  off = up(off + sizeof(float) * (size_t)(2 * num_sms * 2 * rows * kTileN));
  l.end = off;
  return l;
}

}  // namespace awq
