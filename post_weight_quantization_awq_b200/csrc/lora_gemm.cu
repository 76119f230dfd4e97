// Low-rank adapters of many requests beside one packed projection:
//
//   Y[t][o] = RN16( sum_j X[t][j] (q - z) s  +  c_a sum_r U[t][r] B_a[o][r] ),
//   U[t][r] = sum_j X[t][j] A_a[r][j],  a = ids[t]  (-1: no adapter)
//
// lora_shrink_kernel computes U and lets its successor start at once (programmatic
// dependent launch), which meanwhile streams the words and waits for U only before
// its epilogue.  (One launch, in which the blocks of a cluster compute U over their
// input rows while the first words travel, took longer for every adapter: 13.6 against
// 12.3 us for 1 token at rank 16, 18.5 against 14.2 at rank 64, since every output
// tile's cluster reads all of A.)
//
// Measured at 4096 x 4096, rank 16: 10.7 us for 1 token (9.6 without an adapter), 13.7
// for 16, where the words are 1.4 us: bound by the latency of the launches, the loads and
// the sums that meet.  45 tokens on 4096 x 12288, rank 64: 39.5 us, bound by the core's
// instructions.
#include <cooperative_groups.h>

#include "awq_launch.h"
#include "serve_launch.h"
#include "w4_stream.cuh"

namespace awq {
namespace {
namespace cg = cooperative_groups;
using namespace w4s;

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

// U of one token and kShrinkR rank rows a block: the 8 warps take eighths of the
// input, all loads of a warp in flight at once, and meet in shared memory.
constexpr int kShrinkR = 8;
__global__ void __launch_bounds__(256) lora_shrink_kernel(const LoraArgs a) {
  __shared__ float part[8][kShrinkR];
  pdl_wait();  // the work before this call: its results are the stream kernel's inputs too
  pdl_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{};
  const int chunks = a.rank / kShrinkR, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x / chunks;
  const int r0 = (int)(blockIdx.x - t * chunks) * kShrinkR;
  const int id = a.ids[t];
  if (id < 0 || id >= a.adapters) return;  // never read
  const float scale = __ldg(a.c + id);
  const int n = (int)(a.in / 8), c0 = n * warp / 8, c1 = n * (warp + 1) / 8;  // 16-byte chunks
  const uint4 *x = reinterpret_cast<const uint4 *>(a.X + t * a.ldx);
  const uint4 *w = reinterpret_cast<const uint4 *>(a.A + ((int64_t)id * a.rank + r0) * a.in);
  float s[kShrinkR];
#pragma unroll
  for (int r = 0; r < kShrinkR; ++r) s[r] = 0.0f;
#pragma unroll 2
  for (int k = c0 + lane; k < c1; k += 32) {
    const uint4 xv = __ldg(x + k);
    uint4 wv[kShrinkR];
#pragma unroll
    for (int r = 0; r < kShrinkR; ++r) wv[r] = __ldg(w + (int64_t)r * n + k);
#pragma unroll
    for (int r = 0; r < kShrinkR; ++r) s[r] = dot8(xv, wv[r], s[r]);
  }
#pragma unroll
  for (int r = 0; r < kShrinkR; ++r) {
#pragma unroll
    for (int m = 16; m; m >>= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], m);
    if (lane == 0) part[warp][r] = s[r];
  }
  __syncthreads();
  if (threadIdx.x < kShrinkR && AWQ_IN_BOUNDS(t < a.T && r0 + kShrinkR <= a.rank, 0xB0A0u)) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) u += part[i][threadIdx.x];
    a.U[t * a.rank + r0 + threadIdx.x] = scale * u;
  }
}

// One output's part of a token's adapter in fp32, term by term; 0 where U and B_a are
// finite throughout.
__device__ __noinline__ float non_finite_dot(const float *u, const __half *b, int rank) {
  float s = 0.0f;
  bool any = false;
  for (int r = 0; r < rank; ++r) {
    const float x = u[r], y = __half2float(b[r]);
    any |= !isfinite(x) || !isfinite(y);
    s = fmaf(x, y, s);
  }
  return any ? s : 0.0f;
}

// A cluster of `splits` blocks covers 256 outputs x MAXTOK tokens, each block
// a range of input rows and a share of the adapters; the blocks' fp32 sums meet
// through distributed shared memory in rank order.
//
// The adapters' part joins the accumulators on the tensor cores too: B_a's rows
// are A operands straight from global memory, and U (fp32) is an fp16 pair
// hi + lo of 22 bits under a power of two of its token, so nothing is rounded
// away and no U overflows.  An adapter's sums are added for its own tokens only.  With an
// infinity or a NaN in U or B_a a pair's product is not the value's (0 x infinity is NaN):
// a sum that is not finite is left out and made in fp32 afterwards.
template <Mode M, int NT, int MAXTOK, int STAGES>
struct LoraShared {
  static constexpr uint32_t kRing = STAGES * stage_bytes<M, MAXTOK>();
  static constexpr uint32_t kRed = (MAXTOK * kRedPitch * 4 + 15) / 16 * 16;  // in the ring, after the product
  static constexpr int kUPitch = 2 * (256 + 8);                               // bytes of a token's hi (lo) row
  static constexpr uint32_t kU = 2 * MAXTOK * kUPitch;                        // behind it
  static constexpr uint32_t kTail = sizeof(RingBars<STAGES>) + MAXTOK * 16 + 16 + kLoraStreamT * 4;
  static constexpr uint32_t kBytes = 1024 + kRing + kTail;
  static_assert(kRed + kU <= kRing, "the sums and U reuse the ring");
};

template <Mode M, int NT, int MAXTOK, int STAGES, int MINB, int SHIFT>
__global__ void __launch_bounds__(kThreads, MINB)
    lora_stream_kernel(const __grid_constant__ LoraArgs a, const __grid_constant__ CUtensorMap map, const int splits) {
  using L = LoraShared<M, NT, MAXTOK, STAGES>;
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  float *red = reinterpret_cast<float *>(ring);
  uint8_t *uhl = ring + L::kRed;
  auto *bars = reinterpret_cast<RingBars<STAGES> *>(ring + L::kRing);
  // the tokens stand in the order of their adapters, so that one's tokens fill whole
  // token tiles; this block's are the places [t0, t0 + n)
  int *ids = reinterpret_cast<int *>(bars + 1);  // adapter of the token at a place, -1: none
  int *perm = ids + MAXTOK;                      // its row of X
  int *list = perm + MAXTOK;                     // the different adapters' first place | end << 16
  float *uscale = reinterpret_cast<float *>(list + MAXTOK);
  int *n_list = reinterpret_cast<int *>(uscale + MAXTOK);
  int *all_ids = n_list + 4;                     // all tokens' adapters
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)(blockIdx.x % (unsigned)splits);
  const int64_t tile = blockIdx.x / (unsigned)splits;
  const int64_t t0 = (int64_t)blockIdx.y * MAXTOK;
  const int n = (int)(a.T - t0 < MAXTOK ? a.T - t0 : MAXTOK);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) ring_init(bars);
  __syncthreads();
  // input rows of this rank, in units of 256 (128) rows so that groups stay whole
  const int64_t unit = a.in >= 512 * splits ? 256 : 128, units = (a.in + unit - 1) / unit;
  const int k0 = (int)(units * rank / splits * unit);
  const int k1 = (int)i64min(units * (rank + 1) / splits * unit, a.in);
  if (tid >= kConsumers) {
    Producer<M, MAXTOK> p(Weights{&map, 0, a.qzeros, a.scales, a.out / 8, (int)a.in, SHIFT,
                  (int)(tile * 32), (int)(a.out / 8), (int)(tile * 32), (int)(a.out / 8)});
    RingPos pos;
    // the first words do not wait for the tokens' order
    const int ahead = min(num_stages<M>(max(k1 - k0, 0)), STAGES);
    for (int s = 0; s < ahead; ++s)
      p.issue_words(smem_u32(ring) + s * stage_bytes<M, MAXTOK>(), &bars->full[s], k0, k1, s);
    asm volatile("bar.sync 2, 288;" ::: "memory");
    p.rows(a.X, a.ldx, a.T, n, [&](int t) { return perm[t]; });
    p.run(pos, smem_u32(ring), bars, k0, k1, a.max_polls, nullptr, ahead);
    if (*reinterpret_cast<volatile int *>(&bars->abort)) ring_drain(bars, pos);
  } else {
    RingPos pos;
    Acc<NT> acc;
    // The tokens' order, while the first words travel.  What is read before pdl_wait() (ids,
    // token rows, words) comes from L2: it is where the work before the shrink kernel has
    // left its results when that kernel lets this one start, and an L1 need not know of them
    if (tid < a.T) {
      const int id = __ldcg(a.ids + tid);
      all_ids[tid] = id >= 0 && id < a.adapters ? id : -1;
    }
    if (tid < MAXTOK) ids[tid] = -1;
    consumer_sync();
    if (tid < a.T) {
      const int id = all_ids[tid];
      int at = -(int)t0;
      for (int s = 0; s < a.T; ++s) at += all_ids[s] < id || (all_ids[s] == id && s < tid);
      if (at >= 0 && at < n) {
        ids[at] = id;
        perm[at] = tid;
      }
    }
    asm volatile("bar.sync 2, 288;" ::: "memory");
    if (warp == 0) {
      int count = 0;
      for (int c = 0; c < n; c += 32) {
        const int t = c + lane, id = t < n ? ids[t] : -1;
        const bool first = id >= 0 && (t == 0 || ids[t - 1] != id);
        const uint32_t b = __ballot_sync(0xffffffffu, first);
        if (first) {
          int end = t + 1;
          while (end < n && ids[end] == id) ++end;
          list[count + __popc(b & ((1u << lane) - 1u))] = t | end << 16;
        }
        count += __popc(b);
      }
      if (lane == 0) *n_list = count;
    }
    consume<M, NT, MAXTOK, STAGES, SHIFT>(acc, pos, ring, bars, k0, k1, true, a.max_polls, nullptr);
    pdl_wait();  // U and the cleared status word
    consumer_sync();
    const int r32 = (a.rank + 31) / 32 * 32;
    {  // a team of threads to a token, all tokens at once
      constexpr int kTeam = MAXTOK <= 8 ? 32 : MAXTOK <= 16 ? 16 : MAXTOK <= 32 ? 8 : 4;
      const int t = tid / kTeam, part = tid % kTeam;
      const bool on = t < n && ids[t] >= 0 && AWQ_IN_BOUNDS(perm[t] >= 0 && perm[t] < a.T, 0xB0A2u);
      const float4 *u = reinterpret_cast<const float4 *>(a.U + (on ? perm[t] : 0) * a.rank);
      uint32_t m = 0;  // the largest magnitude's bits; a NaN's are larger than all
#pragma unroll 4
      for (int k = part; k < a.rank / 4; k += kTeam)
        if (on) {
          const float4 v = u[k];
          m = max(max(m, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu)),
                  max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
        }
#pragma unroll
      for (int d = kTeam / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      // 2^e with |u| / 2^e below 4, NaN where U has one
      const int e = min(max((int)(m >> 23) - 127, -126), 126);
      const float up = m > 0x7f800000u ? __uint_as_float(m) : __uint_as_float((uint32_t)(127 + e) << 23);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      if (t < MAXTOK) {
        if (part == 0) uscale[t] = up;
        __half2 *d = reinterpret_cast<__half2 *>(uhl + t * L::kUPitch);
#pragma unroll 4
        for (int k = part; k < r32 / 4; k += kTeam) {
          const float4 v = on && 4 * k < a.rank ? u[k] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          const float w[4] = {v.x * down, v.y * down, v.z * down, v.w * down};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 hi = __floats2half2_rn(w[2 * i], w[2 * i + 1]);
            const float2 f = __half22float2(hi);
            d[2 * k + i] = hi;
            d[2 * k + i + L::kU / 8] = __floats2half2_rn(isfinite(f.x) ? w[2 * i] - f.x : 0.0f, isfinite(f.y) ? w[2 * i + 1] - f.y : 0.0f);
          }
        }
      }
    }
    consumer_sync();
    const int nw = warp & 3, half = warp >> 2, g = lane >> 2, q = lane & 3;
    const int64_t o0 = tile * kBoxN + (nw * 8 + g) * 8;
    const int tt = M == Mode::kTok ? half * NT * 8 : 0;  // this warp's first token column
    const int step = M == Mode::kK ? 2 * splits : splits, first = M == Mode::kK ? 2 * rank + half : rank;
    // 32 rank rows a step, a lane's 16 bytes at 8q of a row of B_a (or of U) being
    // its fragments of two MMAs
    const uint8_t *ul = uhl + (tt + g) * L::kUPitch + q * 16;
    bool left_out = false;
    for (int j = first; j < *n_list; j += step) {
      const int lo = list[j] & 0xffff, hi = list[j] >> 16, id = ids[lo];
      if (hi <= tt || lo >= tt + 8 * NT) continue;  // none of this warp's tokens
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc.grp[p][x][c] = 0.0f;
      const __half *bp = a.B + ((int64_t)id * a.out + o0) * a.rank + 8 * q;
      // out % 32 == 0: the 8 outputs are all in or all out
      const bool o_ok = o0 < a.out && AWQ_IN_BOUNDS(id >= 0 && id < a.adapters && o0 + 8 <= a.out, 0xB0A1u);
#pragma unroll 1
      for (int k = 0; k < r32; k += 32) {
        uint4 af[8];
#pragma unroll
        for (int o = 0; o < 8; ++o)
          af[o] = o_ok && k + 8 * q < a.rank ? __ldg(reinterpret_cast<const uint4 *>(bp + (int64_t)o * a.rank + k))
                                             : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (hi <= tt + 8 * x || lo >= tt + 8 * x + 8) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // hi, lo
            const uint4 b = *reinterpret_cast<const uint4 *>(ul + h * (L::kU / 2) + x * 8 * L::kUPitch + k * 2);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              mma16816(acc.grp[p][x], af[p].x, af[p + 4].x, af[p].y, af[p + 4].y, b.x, b.y);
              mma16816(acc.grp[p][x], af[p].z, af[p + 4].z, af[p].w, af[p + 4].w, b.z, b.w);
            }
          }
        }
      }
      const auto each_sum = [&](auto f) {  // of this adapter's tokens
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = tt + x * 8 + 2 * q + e;
            if (t < lo || t >= hi) continue;
            const float sc = uscale[t];
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
              for (int h = 0; h < 2; ++h) f(sc, acc.grp[p][x][e + 2 * h], acc.out[p][x][e + 2 * h]);
          }
      };
      float bad[8] = {};  // NaN where a sum is not finite (of whichever token: fewer tests)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int c = 0; c < 4; ++c) bad[2 * p + (c & 1)] = fmaf(0.0f, acc.grp[p][x][c], bad[2 * p + (c & 1)]);
      const float odd = ((bad[0] + bad[1]) + (bad[2] + bad[3])) + ((bad[4] + bad[5]) + (bad[6] + bad[7]));
      if (__any_sync(0xffffffffu, odd != 0.0f))
        each_sum([&](float sc, float &v, float &) {
          if (isfinite(v)) return;
          v = 0.0f;
          left_out |= !isnan(sc);  // NaN in U: all its outputs are
        });
      each_sum([&](float sc, float v, float &out) { out = fmaf(sc, v, out); });
    }
    // The sums left out, in a loop of their own: beside the MMAs they cost 20 % (36 tokens
    // with 31 adapters of rank 64)
    if (__any_sync(0xffffffffu, left_out)) {
      for (int j = first; j < *n_list; j += step) {
        const int lo = list[j] & 0xffff, hi = list[j] >> 16;
        if (o0 >= a.out) break;
        const __half *b = a.B + ((int64_t)ids[lo] * a.out + o0) * a.rank;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = tt + x * 8 + 2 * q + e;
            if (t < lo || t >= hi || isnan(uscale[t])) continue;
            const float *u = a.U + perm[t] * a.rank;
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
              for (int h = 0; h < 2; ++h) acc.out[p][x][e + 2 * h] += non_finite_dot(u, b + (p + 4 * h) * a.rank, a.rank);
          }
      }
      __syncwarp();
    }
    store_sums<M, NT>(acc, red);
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && warp == kConsumers / 32) {
    pdl_wait();
    for (int t = lane; t < a.T; t += 32) {
      const int id = a.ids[t];
      if (id < -1 || id >= a.adapters) dev_fail(a.st, kDevBadAdapter, 0xE01u);
    }
  }
  cluster.sync();
  // A wait of the ring that ran out.  It may have done so before the shrink kernel cleared
  // the status word; this thread has seen that kernel end
  if (tid == 0 && *reinterpret_cast<volatile int *>(&bars->abort)) dev_fail(a.st, kDevTimeout, 0xE21u);
  for (int i = rank * kConsumers + tid; tid < kConsumers && i < n * (kBoxN / 2); i += splits * kConsumers) {
    const int t = i / (kBoxN / 2), oo = 2 * (i % (kBoxN / 2));
    const int64_t o = tile * kBoxN + oo;
    if (o >= a.out || !AWQ_IN_BOUNDS(o + 2 <= a.out && perm[t] >= 0 && perm[t] < a.T, 0xB0A3u)) continue;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      const float *p = cluster.map_shared_rank(red, s) + t * kRedPitch + oo;
      s0 += p[0];
      s1 += p[1];
    }
    *reinterpret_cast<__half2 *>(a.Y + perm[t] * a.ldy + o) = __floats2half2_rn(s0, s1);
  }
  cluster.sync();  // no block leaves while its sums are read
}

// The most blocks of a cluster (up to 8) with which `clusters` of them run at
// once: a second wave costs a whole pass (16 clusters of 8 blocks do not fit the
// GPCs at one block per SM: 15.5 us for the last to start).
template <class K>
int cluster_size(K kernel, size_t smem, int64_t clusters, int64_t most, std::atomic<int> (&fit)[64][9]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  for (int s = (int)(most < 8 ? most : 8); s > 1; --s) {
    int known = fit[dev][s];  // 0: not asked yet
    if (!known) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)s);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)s;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
      }
      fit[dev][s] = known = n + 1;
    }
    if (known > clusters) return s;
  }
  return 1;
}

// The blocks that share a tile (and a group of MAXTOK tokens), and the time of the
// whole in cycles of its steps, measured: 252, 313 and 400 for 2, 3 and 4 token tiles.
struct Split {
  int s;
  int64_t groups, cycles;
};
template <Mode M, int NT, int MAXTOK, int STAGES, int MINB, int SHIFT>
struct Stream {
  static constexpr size_t kSmem = LoraShared<M, NT, MAXTOK, STAGES>::kBytes;
  static_assert(MINB * (kSmem + 1024) <= 233472, "resident blocks");
  static constexpr auto kernel = lora_stream_kernel<M, NT, MAXTOK, STAGES, MINB, SHIFT>;

  static cudaError_t split(const LoraArgs &a, int num_sms, Split &p) {
    static std::atomic<bool> done[64];
    static std::atomic<int> fit[64][9];
    const cudaError_t e = allow_smem(kernel, kSmem, done);
    if (e != cudaSuccess) return e;
    p.groups = (a.T + MAXTOK - 1) / MAXTOK;
    const int64_t clusters = (a.out + kBoxN - 1) / kBoxN * p.groups;
    p.s = cluster_size(kernel, kSmem, clusters, (a.in + 127) / 128, fit);
    const int64_t waves = (clusters * p.s + num_sms * MINB - 1) / (num_sms * MINB);
    p.cycles = waves * ((a.in + p.s - 1) / p.s) / (M == Mode::kTok ? 16 : 32) * (NT <= 2 ? 252 : NT == 3 ? 313 : 400);
    return cudaSuccess;
  }

  static cudaError_t launch(const LoraArgs &a, const Split &p, cudaStream_t stream) {
    CUtensorMap map;  // the words as pairs of 16-bit values
    cudaError_t e = make_tmap_f16_box(&map, a.qweight, a.in, a.out / 4, a.out / 4, 64, kBoxK);
    if (e != cudaSuccess) return e;
    e = launch_after(lora_shrink_kernel, a.T * (a.rank / kShrinkR), 256, 0, stream, a);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.s;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.out + kBoxN - 1) / kBoxN * p.s), (unsigned)p.groups);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, map, p.s);
  }

  static cudaError_t run(const LoraArgs &a, int num_sms, cudaStream_t stream) {
    Split p;
    const cudaError_t e = split(a, num_sms, p);
    return e != cudaSuccess ? e : launch(a, p, stream);
  }
};

// 17 tokens and more: all of them in one block, or 16 in each of several blocks of a
// tile, whichever fills the SMs better (45 tokens on 4096 x 12288: 45 us in 48 clusters
// of 2, since 48 of 3 do not fit, 37 us in 3 groups of 16; on 4096 x 32768, rank 16, 70 us
// in 128 blocks, 101 in groups).
template <class Whole, class Groups>
cudaError_t launch_wide(const LoraArgs &a, int num_sms, cudaStream_t stream) {
  Split w, g;
  cudaError_t e = Whole::split(a, num_sms, w);
  if (e == cudaSuccess) e = Groups::split(a, num_sms, g);
  if (e != cudaSuccess) return e;
  return g.cycles < w.cycles ? Groups::launch(a, g, stream) : Whole::launch(a, w, stream);
}

template <int SHIFT>
cudaError_t launch_group(const LoraArgs &a, int num_sms, cudaStream_t stream) {
  if (a.T <= 8) return Stream<Mode::kK, 1, 8, 4, 2, SHIFT>::run(a, num_sms, stream);
  using Groups = Stream<Mode::kK, 2, 16, 8, 1, SHIFT>;
  if (a.T <= 16) return Groups::run(a, num_sms, stream);
  if (a.T <= 32) return launch_wide<Stream<Mode::kTok, 2, 32, 6, 1, SHIFT>, Groups>(a, num_sms, stream);
  if (a.T <= 48) return launch_wide<Stream<Mode::kTok, 3, 48, 6, 1, SHIFT>, Groups>(a, num_sms, stream);
  return launch_wide<Stream<Mode::kTok, 4, 64, 5, 1, SHIFT>, Groups>(a, num_sms, stream);
}
}  // namespace

cudaError_t launch_lora(const LoraArgs &a, int num_sms, cudaStream_t stream) {
  return a.group == 128  ? launch_group<7>(a, num_sms, stream)
         : a.group == 64 ? launch_group<6>(a, num_sms, stream)
                         : launch_group<5>(a, num_sms, stream);
}

AWQ_BOUNDS_READER(bounds_status_lora)

}  // namespace awq
