// A whole mixture-of-experts layer on packed 4-bit experts for a few tokens,
// one cooperative kernel (and one that clears its status word and counters):
//
//   l = x Wr^T;  the k largest logits (ties to the lowest expert), p = softmax
//   over all experts (divided by the chosen ones' sum when renormalize);
//   y = sum_k p_k down_e( RN16( silu(x gate_e) * (x up_e) ) )
//
// The layer is bound by reading the met experts' words once.  Phases, between
// grid barriers:
//   router   a warp per (token, expert): exact products summed in fp64, so that
//            a choice next to a border is the definition's; the warp that
//            writes a token's last logit picks its experts;
//   lists    every block makes the experts' token lists in shared memory;
//   gate|up  tiles of 512 consecutive outputs (256 bytes of every row: 128-byte
//            pieces of rows read HBM at 4.6-5.0 TB/s, 256-byte ones at 6.1-6.6),
//            gate's and up's of one expert in turn, in units of 128 input rows.
//            The units are dealt out evenly by cost and in order; fp32 sums go
//            to L2.  While the blocks meet, the producer warps load the first
//            words of the next phase;
//   H        silu(g) u from the sums of the blocks that share a tile, added in
//            block order: each block makes what its down units read, or, where
//            that would be made too many times over, all blocks make all of it
//            between two barriers;
//   down     the same over hidden's tiles and all met experts;
//   combine  a token's experts' sums, weighted with p in fp32, one rounding.
// Sums are added in an order fixed by the sizes and the routing alone.
//
// Measured, 4096 -> 11008 and two of eight experts: 58 us for 1 token (139 MB of
// words and steps; 5.3 TB/s while gate|up streams, the rest are phases that wait
// for each other), 241 us for 64 (557 MB; 252-313 cycles for 16 rows x 512 outputs
// by 8 warps, bound by their instructions and the latency of mma.sync).
#include <climits>
#include <cuda_runtime.h>
#include <type_traits>

#include "awq_launch.h"
#include "serve_launch.h"
#include "w4_stream.cuh"

namespace awq {
namespace {
using namespace w4s;

constexpr int kTile = 2 * kBoxN;  // outputs of a block's tile
constexpr int kCap = 24;          // tokens of an entry: three token tiles are what 168 registers hold

// Up to 8 tokens (V = 1), or more: the (token, slot) pairs and the entries (an
// expert and up to kTok of its tokens) at most, the depth of the ring, the
// resident blocks of an SM.
template <int V>
struct Cfg {
  static constexpr int kTok = V == 1 ? 8 : kCap;
  static constexpr int kPairs = (V == 1 ? 8 : kMoeMaxTokens) * kMoeMaxTopK;
  static constexpr int kSegs = V == 1 ? kPairs : kMoeMaxExperts + kPairs / kCap + 1;
  static constexpr int kStages = V == 1 ? 5 : 9;
  static constexpr int kBlocks = V == 1 ? 2 : 1;
  static constexpr uint32_t kStage = stage_bytes<Mode::kN, kTok>();
  static constexpr uint32_t kRing = kStages * kStage;
};

// Where every block computes all logits itself: one to a warp.  Up to 8 logits of hidden
// 1024 to 16384 a layer takes 1.7 us less to 0.3 more than with logits made together (1
// token on eight experts of hidden 1024: 21.2 us, 22.2 together; on two of 16384: 45.8 and
// 47.5); with 32 logits 2.1 more.
constexpr int kAloneLogits = kThreads / 32;
// Where every block makes the values of H that its down units read: this many values in
// all, each counted once for every tile of down.  Up to 45 000 a layer takes 0.3 to 0.8 us
// less than with H made once between two barriers (1 token, 2048 -> 1408: 23.4 us, 24.2
// between barriers), from 65 000 0.4 to 8 more (1 token, 4096 -> 11008: 58.8 and 56.9; 32
// tokens, 2048 -> 2048, all of eight: 88.8 and 80.7), but for 64 tokens on one or two
// tiles of hidden (0.5 to 2.6 less).
constexpr int64_t kOwnH = 3 << 14;
constexpr int kPieceH = 128;  // channels of H made at a time; divides a tile

template <int V>
struct MoeLists {
  using C = Cfg<V>;
  float wt[C::kPairs];
  int16_t pair[C::kPairs];   // the entries' pairs, expert by expert
  int16_t where[C::kPairs];  // position of a pair among them
  int count[kMoeMaxExperts];
  int16_t seg_expert[C::kSegs], seg_first[C::kSegs], seg_n[C::kSegs];
  int seg_cost[C::kSegs + 1];  // cost of a unit, summed over the entries before
  double logit[kAloneLogits];
  int n_seg;
  int flag;
};

template <int V>
constexpr uint32_t moe_smem() {
  constexpr uint32_t n = 1024 + Cfg<V>::kRing + sizeof(RingBars<Cfg<V>::kStages>) + sizeof(MoeLists<V>);
  static_assert(Cfg<V>::kBlocks * (n + 1024) <= 233472, "resident blocks");
  return n;
}

// All blocks meet (counter from 0 to gridDim.x); false when the wait ran out.  The
// release and the acquire cover the block's other threads through its barriers.
__device__ __forceinline__ bool grid_barrier(uint32_t *counter, int *flag, DevStatus *st, uint32_t max_polls,
                                             uint32_t site) {
  __syncthreads();
  if (threadIdx.x == 0) {
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
    *flag = ok;
  }
  __syncthreads();
  return *flag != 0;
}

// Products of fp16 values are exact in fp32; their sum is fp64.
__device__ __forceinline__ double dot8d(uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  double s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&y[i]));
    s[i] = (double)__fmul_rn(p.x, q.x) + (double)__fmul_rn(p.y, q.y);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The logit of one (token, expert) pair by a warp.
__device__ __forceinline__ double warp_logit(const MoeArgs &a, int t, int e) {
  const int lane = threadIdx.x & 31;
  const uint4 *x = reinterpret_cast<const uint4 *>(a.X + t * a.ldx);
  const uint4 *w = reinterpret_cast<const uint4 *>(a.router + (int64_t)e * a.hidden);
  double s = 0.0;
#pragma unroll 8
  for (int k = lane; k < a.hidden / 8; k += 32) s += dot8d(__ldg(x + k), __ldg(w + k));
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s + 0.0;  // -0 becomes 0: the choice compares bit patterns
}

// Top-k of one token by a warp; a lane holds experts lane, lane + 32, ...  The
// choices go to id(slot, expert, weight).
template <class Put>
__device__ __forceinline__ void choose(const MoeArgs &a, const double *logits, bool masked, Put put) {
  const int lane = threadIdx.x & 31;
  constexpr int PER = kMoeMaxExperts / 32;
  if (masked) {
    if (lane < a.top_k) put(lane, -1, 0.0f);
    return;
  }
  // fp64 bit patterns in an order-preserving form; NaN sorts by its bits
  long long key[PER];
  double top = -INFINITY;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    key[j] = LLONG_MIN;
    if (32 * j < a.experts && lane + 32 * j < a.experts) {
      const double l = __isGlobal(logits) ? __ldcg(logits + lane + 32 * j) : logits[lane + 32 * j];
      const long long b = __double_as_longlong(l);
      key[j] = b ^ ((b >> 63) & 0x7fffffffffffffffLL);
      top = fmax(top, l);
    }
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, m));
  // exp(l - top): the fp64 difference as two floats, exp of the first exact to
  // fp32 and the second's factor 1 + lo
  const auto weight = [&](long long kk) {
    const long long b = kk ^ ((kk >> 63) & 0x7fffffffffffffffLL);
    const double d = __longlong_as_double(b) - top;
    const float hi = (float)d;
    const float ex = expf(hi);
    return fmaf(ex, isfinite(hi) ? (float)(d - (double)hi) : 0.0f, ex);
  };
  uint32_t taken = 0;
  long long my_key = 0;
  int my_id = -1;
  for (int s = 0; s < a.top_k; ++s) {
    long long best = LLONG_MIN;
    int at = 0x7fff;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (32 * j >= a.experts) break;
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
    if (lane == s) {
      my_key = ((long long)mhi << 32) | (long long)mlo;
      my_id = (int)e;
    }
  }
  const float mine = lane < a.top_k ? weight(my_key) : 0.0f;
  float sum = 0.0f;
  if (a.renormalize) {
    sum = mine;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (32 * j < a.experts && lane + 32 * j < a.experts) sum += weight(key[j]);
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if (lane < a.top_k) put(lane, my_id, mine / sum);
}

// Past 8 tokens: the warp that writes a token's last logit picks its experts.
__device__ void router(const MoeArgs &a) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32);
  for (int i = blockIdx.x + gridDim.x * (threadIdx.x >> 5); i < a.T * a.experts; i += warps) {
    const int t = i / a.experts, e = i - t * a.experts;
    const bool masked = a.mask && !a.mask[t];
    int last = masked && e == 0;
    if (!masked) {
      const double s = warp_logit(a, t, e);
      if (lane == 0 && AWQ_IN_BOUNDS(t < a.T && e < a.experts, 0xB0D0u)) {
        a.logits[i] = s;
        __threadfence();
        last = atomicAdd(a.tok_count + t, 1) == a.experts - 1;
      }
      last = __shfl_sync(0xffffffffu, last, 0);
    }
    if (last && AWQ_IN_BOUNDS(t < a.T, 0xB0D1u)) {
      __threadfence();
      choose(a, a.logits + (int64_t)t * a.experts, masked, [&](int slot, int id, float w) {
        a.ids[t * a.top_k + slot] = id;
        a.weights[t * a.top_k + slot] = w;
      });
    }
  }
}

// Time of a unit of 128 input rows by its token tiles, measured: 207, 252 and
// 313 cycles a step for 1, 2 and 3 tiles with 8 warps on an SM.
__host__ __device__ constexpr int unit_cost(int n) { return n <= 8 ? 3 : n <= 16 ? 4 : 5; }

// The experts' token lists, and the entries.  Every block makes its own: an
// expert's pairs stand in rising order, since blocks that share a tile must agree
// on the rows.
template <int V>
__device__ void make_lists(const MoeArgs &a, MoeLists<V> *sh) {
  constexpr int cap = Cfg<V>::kTok;
  const int tid = threadIdx.x, lane = tid & 31;
  const int pairs = a.T * a.top_k;
  for (int e = tid; e < a.experts; e += kThreads) sh->count[e] = 0;
  if (V != 1)
    for (int i = tid; i < pairs; i += kThreads) {
      sh->pair[i] = (int16_t)__ldcg(a.ids + i);  // for now: its expert
      sh->wt[i] = __ldcg(a.weights + i);
    }
  __syncthreads();
  if (tid < 32) {  // a pair's place among its expert's
    for (int c = 0; c < pairs; c += 32) {
      const int i = c + lane, id = i < pairs ? sh->pair[i] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id), before = same & ((1u << lane) - 1u);
      const int base = id >= 0 ? sh->count[id] : 0;
      __syncwarp();
      if (id >= 0 && !before) sh->count[id] = base + __popc(same);
      if (i < pairs) sh->where[i] = (int16_t)(id >= 0 ? base + __popc(before) : -1);
      __syncwarp();
    }
  }
  __syncthreads();
  if (tid < 32) {  // first pair of each expert and its entries
    int first = 0, segs = 0, costs = 0;
    for (int c = 0; c < a.experts; c += 32) {
      const int n = c + lane < a.experts ? sh->count[c + lane] : 0;
      const int m = (n + cap - 1) / cap;
      int cost = 0;
      for (int j = 0; j < m; ++j) cost += unit_cost(n - cap * j < cap ? n - cap * j : cap);
      int pn = n, pm = m, pc = cost;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, pn, d), v = __shfl_up_sync(0xffffffffu, pm, d),
                  x = __shfl_up_sync(0xffffffffu, pc, d);
        if (lane >= d) {
          pn += u;
          pm += v;
          pc += x;
        }
      }
      int before = costs + pc - cost;
      for (int j = 0; j < m; ++j) {
        const int s = segs + pm - m + j;
        sh->seg_expert[s] = (int16_t)(c + lane);
        sh->seg_first[s] = (int16_t)(first + pn - n + cap * j);
        sh->seg_n[s] = (int16_t)(n - cap * j < cap ? n - cap * j : cap);
        sh->seg_cost[s] = before;
        before += unit_cost(sh->seg_n[s]);
      }
      if (c + lane < a.experts) sh->count[c + lane] = first + pn - n;  // now: first pair
      first += __shfl_sync(0xffffffffu, pn, 31);
      segs += __shfl_sync(0xffffffffu, pm, 31);
      costs += __shfl_sync(0xffffffffu, pc, 31);
    }
    if (lane == 0) {
      sh->n_seg = segs;
      sh->seg_cost[segs] = costs;
    }
  }
  __syncthreads();
  constexpr int PER = (Cfg<V>::kPairs + kThreads - 1) / kThreads;
  int id[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) id[j] = tid + j * kThreads < pairs ? sh->pair[tid + j * kThreads] : -1;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (id[j] >= 0) {
      const int i = tid + j * kThreads, at = sh->count[id[j]] + sh->where[i];
      sh->pair[at] = (int16_t)i;
      sh->where[i] = (int16_t)at;
    }
  __syncthreads();
}

// Rows of the down product's left side: a value of H is an fp16 and, where the
// token tile has the columns to spare, the fp16 of what its rounding left
// (two rows for a token: free, since the instruction computes 8 columns).
__device__ __forceinline__ int h_rows(int n) { return 2 * n <= 8 ? 2 * n : n; }

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// ceil(x / c) for a unit's cost c, x >= 0
__device__ __forceinline__ int units_of(int x, int c) { return c == 3 ? (x + 2) / 3 : c == 4 ? (x + 3) / 4 : (x + 4) / 5; }

// The units of a phase in their order: by (entry, tile) pair, a "stretch" of
// `len` units of 128 input rows, gate|up with the entry outermost (and gate's
// tile before up's), down with the tile outermost.  Blocks take even shares of
// the units' cost.  Costs stay below 2^26 (about 300 entries of 5, 256 tiles, 128
// units; or 32 tiles, 512 units): 32 bits.
struct Stretch {
  int seg, tile;
  int before;  // the cost of all units before it
};

template <int V, bool DOWN>
struct Work {
  const MoeLists<V> *sh;
  int n_seg, tiles, len;  // tiles: gate|up 2 x the pairs of tiles, down the tiles
  int quota;

  __device__ __forceinline__ Work(const MoeLists<V> *l, int tiles_, int len_)
      : sh(l), n_seg(l->n_seg), tiles(tiles_), len(len_) {
    const int total = sh->seg_cost[n_seg] * tiles * len;
    quota = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    // at least a unit's cost, so that every block between a stretch's first and last has a unit of it
    quota = max(quota, unit_cost(Cfg<V>::kTok));
  }
  __device__ __forceinline__ int cost(int seg) const { return sh->seg_cost[seg + 1] - sh->seg_cost[seg]; }
  __device__ __forceinline__ Stretch at(int seg, int tile) const {
    const int c = sh->seg_cost[seg];
    return {seg, tile, (DOWN ? tile * sh->seg_cost[n_seg] + c : c * tiles + tile * cost(seg)) * len};
  }
  // The units of a stretch that block b takes: those whose cost offset lies in
  // its share [b quota, (b + 1) quota).
  __device__ __forceinline__ void units(const Stretch &s, int b, int &u0, int &u1) const {
    const int d = b * quota - s.before, c = cost(s.seg);
    u0 = d <= 0 ? 0 : min(units_of(d, c), len);
    u1 = d + quota <= 0 ? 0 : min(units_of(d + quota, c), len);
  }
  // The blocks of a stretch's first and last unit: all that take part in it.
  __device__ __forceinline__ int2 blocks(const Stretch &s) const {
    return make_int2(s.before / quota, (s.before + (len - 1) * cost(s.seg)) / quota);
  }
  // The last stretch that begins at or before block b's share.
  __device__ __forceinline__ Stretch first_of(int b) const {
    const int at_cost = b * quota, scale = DOWN ? len : tiles * len;
    const int per_tile = sh->seg_cost[n_seg] * len, tile = DOWN ? min(at_cost / per_tile, tiles - 1) : 0;
    const int rest = at_cost - tile * per_tile;
    int lo = 0, hi = n_seg;
    while (hi - lo > 1) {
      const int m = (lo + hi) / 2;
      if (sh->seg_cost[m] * scale <= rest)
        lo = m;
      else
        hi = m;
    }
    return at(lo, DOWN ? tile : min((rest - sh->seg_cost[lo] * scale) / (cost(lo) * len), tiles - 1));
  }
  __device__ __forceinline__ bool next(Stretch &s) const {  // false behind the last one
    s.before += cost(s.seg) * len;
    int &inner = DOWN ? s.seg : s.tile, &outer = DOWN ? s.tile : s.seg;
    if (++inner < (DOWN ? n_seg : tiles)) return true;
    inner = 0;
    return ++outer < (DOWN ? tiles : n_seg);
  }
};

// Block b's stretches of a phase, in order: f(stretch, first unit, end).
template <class W, class F>
__device__ __forceinline__ void each_stretch(const W &w, int b, F f) {
  if (!w.n_seg) return;
  Stretch s = w.first_of(b);
  do {
    int u0, u1;
    w.units(s, b, u0, u1);
    if (u0 < u1)
      f(s, u0, u1);
    else if (u0 < w.len)
      break;  // the block's share has ended
  } while (w.next(s));
}

// Sums of n0 and n1 parts, each in its parts' order, the loads of four of each in
// flight together: p0(i) and p1(i) point at part i.
template <class P0, class P1>
__device__ __forceinline__ void sum_parts(int n0, P0 p0, int n1, P1 p1, float4 &s0, float4 &s1) {
  s0 = s1 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const auto add = [](float4 &s, const float4 &v) {
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  };
  for (int k = 0; k < n0 || k < n1; k += 4) {
    float4 v[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = w[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k + j < n0) v[j] = __ldcg(reinterpret_cast<const float4 *>(p0(k + j)));
      if (k + j < n1) w[j] = __ldcg(reinterpret_cast<const float4 *>(p1(k + j)));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      add(s0, v[j]);
      add(s1, w[j]);
    }
  }
}

template <int V, int SHIFT>
__global__ void __launch_bounds__(kThreads, Cfg<V>::kBlocks)
    moe_kernel(const __grid_constant__ MoeArgs a, const __grid_constant__ CUtensorMap gu_map,
               const __grid_constant__ CUtensorMap dn_map) {
  using C = Cfg<V>;
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  auto *bars = reinterpret_cast<RingBars<C::kStages> *>(ring + C::kRing);
  auto *sh = reinterpret_cast<MoeLists<V> *>(bars + 1);
  const uint32_t ring_u = smem_u32(ring);
  const int tid = threadIdx.x;
  DevStatus *st = a.st;
  const int hidden = (int)a.hidden, inter = (int)a.inter;
  const int itiles = (inter + kTile - 1) / kTile, htiles = (hidden + kTile - 1) / kTile;
  const int kgh = (hidden + 127) / 128, kgi = (inter + 127) / 128;

  if (tid == 0) {
    ring_init(bars);
    tma_prefetch_desc(&gu_map);
    tma_prefetch_desc(&dn_map);
  }
  if (V == 1) {
    // A few tokens: every block chooses for itself, from logits that the blocks
    // compute together, or each on its own where that is cheaper than meeting
    // (a barrier is 1.8 us)
    const int warp = tid >> 5, lane = tid & 31;
    const bool alone = a.T * a.experts <= kAloneLogits;
    const int first = alone ? warp : (int)blockIdx.x + (int)gridDim.x * warp;
    const int step = (alone ? 1 : (int)gridDim.x) * (kThreads / 32);
    for (int i = first; i < a.T * a.experts; i += step) {
      const int t = i / a.experts;
      if (a.mask && !a.mask[t]) continue;
      const double l = warp_logit(a, t, i - t * a.experts);
      if (lane == 0) (alone ? sh->logit : a.logits)[i] = l;
    }
    if (alone)
      __syncthreads();
    else if (!grid_barrier(a.barrier + 0, &sh->flag, st, a.max_polls, 0xE10u))
      return;
    for (int t = warp; t < a.T; t += kThreads / 32)
      choose(a, (alone ? sh->logit : a.logits) + (int64_t)t * a.experts, a.mask && !a.mask[t],
             [&](int slot, int id, float w) {
               sh->pair[t * a.top_k + slot] = (int16_t)id;
               sh->wt[t * a.top_k + slot] = w;
               if (blockIdx.x == 0) {
                 a.ids[t * a.top_k + slot] = id;
                 a.weights[t * a.top_k + slot] = w;
               }
             });
  } else {
    router(a);
    if (!grid_barrier(a.barrier + 0, &sh->flag, st, a.max_polls, 0xE10u)) return;
  }
  make_lists<V>(a, sh);

  const Work<V, false> up(sh, 2 * itiles, kgh);
  const Work<V, true> down(sh, htiles, kgi);
  const int wi = inter / 8, wh = hidden / 8;  // word columns
  const int64_t pitch_gu = 2 * a.inter;  // a row of the gate|up sums
  // the words of a stretch
  const auto up_weights = [&](const Stretch &s) {
    const int e = AWQ_IN_BOUNDS(s.seg < sh->n_seg && sh->seg_expert[s.seg] >= 0 && sh->seg_expert[s.seg] < a.experts, 0xB0D2u)
                      ? sh->seg_expert[s.seg] : 0;
    const int tile = AWQ_IN_BOUNDS(s.tile < 2 * itiles, 0xB0D3u) ? s.tile : 0;
    const int64_t groups = (int64_t)e * (hidden / a.group);
    const int c0 = (tile & 1) * wi + (tile >> 1) * 64, end = (tile & 1) ? 2 * wi : wi;
    return Weights{&gu_map, e * hidden, a.gu_z + groups * 2 * wi, a.gu_s + groups * 2 * inter, 2 * wi, hidden, SHIFT,
                   c0, end, c0 + 32, end};
  };
  const auto down_weights = [&](const Stretch &s) {
    const int e = AWQ_IN_BOUNDS(s.seg < sh->n_seg && sh->seg_expert[s.seg] >= 0 && sh->seg_expert[s.seg] < a.experts, 0xB0D4u)
                      ? sh->seg_expert[s.seg] : 0;
    const int c0 = AWQ_IN_BOUNDS(s.tile < htiles, 0xB0D5u) ? s.tile * 64 : 0;
    const int64_t groups = (int64_t)e * (inter / a.group);
    return Weights{&dn_map, e * inter, a.dn_z + groups * wh, a.dn_s + groups * hidden, wh, inter, SHIFT, c0, wh, c0 + 32, wh};
  };
  const bool own_h = (int64_t)a.T * a.top_k * inter * htiles <= kOwnH;
  bool ok = true;

  if (tid >= kConsumers) {
    // ------------------------------------------------------------ producer
    RingPos pos;
    each_stretch(up, (int)blockIdx.x, [&](const Stretch &s, int u0, int u1) {
      Producer<Mode::kN, C::kTok> p(up_weights(s));
      const int seg = s.seg, p0 = sh->seg_first[seg];
      p.rows(a.X, a.ldx, a.T, sh->seg_n[seg], [&](int t) { return sh->pair[p0 + t] / a.top_k; });
      p.template run<C::kStages>(pos, ring_u, bars, u0 * 128, min(u1 * 128, hidden), a.max_polls, st);
    });
    // the first words of the down product do not wait for H
    int ahead = 0;
    bool met = false;
    const auto meet = [&] {
      met = true;
      ok = grid_barrier(a.barrier + 1, &sh->flag, st, a.max_polls, 0xE11u);
      if (ok && own_h)
        asm volatile("bar.sync 2, 288;" ::: "memory");  // H of this block's ranges is there
      else if (ok)
        ok = grid_barrier(a.barrier + 2, &sh->flag, st, a.max_polls, 0xE13u);
    };
    each_stretch(down, (int)blockIdx.x, [&](const Stretch &s, int u0, int u1) {
      Producer<Mode::kN, C::kTok> p(down_weights(s));
      const int k0 = u0 * 128, k1 = min(u1 * 128, inter);
      if (!met) {
        RingPos r = pos;
        const int most = min(num_stages<Mode::kN>(k1 - k0), C::kStages);
        while (ahead < most && ring_wait(bars, &bars->empty[r.slot], r.phase ^ 1u, a.max_polls, st, 0xE22u)) {
          p.issue_words(ring_u + r.slot * C::kStage, &bars->full[r.slot], k0, k1, ahead++);
          r.next<C::kStages>();
        }
        meet();
      }
      if (!ok) return;
      const int seg = s.seg, p0 = sh->seg_first[seg], n = sh->seg_n[seg], pairs = a.T * a.top_k;
      p.rows(a.H, inter, 2 * pairs, h_rows(n),
             [&](int t) { return t < n ? sh->pair[p0 + t] : pairs + sh->pair[p0 + t - n]; });
      p.template run<C::kStages>(pos, ring_u, bars, k0, k1, a.max_polls, st, ahead);
      ahead = 0;
    });
    if (!met) meet();
    for (int i = 0; i < ahead; ++i) pos.next<C::kStages>();
    if (!ok || *reinterpret_cast<volatile int *>(&bars->abort)) ring_drain(bars, pos);
  } else {
    // ------------------------------------------------------------ consumers
    const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int lane_col = (warp >> 2) * kBoxN + ((warp & 3) * 8 + g) * 8;  // first of this lane's 8 outputs in a tile
    RingPos pos;
    // sums of rows [k0, k1) into d(token row) + column, for `rows` token rows and `cols` outputs
    const auto sums = [&](int rows, int k0, int k1, int cols, auto dst) {
      const auto run = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        Acc<NT> acc;
        consume<Mode::kN, NT, C::kTok, C::kStages, SHIFT>(acc, pos, ring, bars, k0, k1, cols > kBoxN, a.max_polls, st);
        if (lane_col >= cols) return;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = n * 8 + 2 * q + e;
            float v[8];
            outputs8<NT>(acc, n, e, v);
            if (t < rows && AWQ_IN_BOUNDS(rows <= C::kTok && lane_col + 8 <= cols, 0xB0D6u)) {
              float4 *d = reinterpret_cast<float4 *>(dst(t) + lane_col);
              __stcg(d, make_float4(v[0], v[1], v[2], v[3]));
              __stcg(d + 1, make_float4(v[4], v[5], v[6], v[7]));
            }
          }
      };
      if (V == 1 || rows <= 8)
        run(std::integral_constant<int, 1>{});
      else if (rows <= 16)
        run(std::integral_constant<int, 2>{});
      else
        run(std::integral_constant<int, 3>{});
    };
    // a block's two partial tiles: one it enters inside, one it leaves inside
    const auto slot = [&](int64_t b, int which) { return a.partial + (b * 2 + which) * C::kTok * kTile; };
    const auto dn_slot = [&](int64_t b, int which) { return a.dn_partial + (b * 2 + which) * C::kTok * kTile; };

    each_stretch(up, (int)blockIdx.x, [&](const Stretch &s, int u0, int u1) {
      const int seg = s.seg, tile = s.tile, p0 = sh->seg_first[seg], n = sh->seg_n[seg];
      const int ch = (tile >> 1) * kTile, cols = min(kTile, inter - ch);  // the tile's channels
      const bool whole = u0 == 0 && u1 == up.len;
      float *part = slot(blockIdx.x, u0 == 0);
      float *gu = a.sums + (tile & 1) * a.inter + ch;
      sums(n, u0 * 128, min(u1 * 128, hidden), cols, [&](int t) {
        return whole ? gu + sh->pair[p0 + t] * pitch_gu : part + t * kTile;
      });
    });
    // H of entry seg, channels [c0, c1): the sums of the blocks that share gate's and
    // up's tile, silu(g) u, and what its rounding leaves
    const auto finish = [&](int seg, int c0, int c1) {
      const int n = sh->seg_n[seg], p0 = sh->seg_first[seg], quads = (c1 - c0) / 4;
      const bool rest_too = h_rows(n) > n;
      for (int i = tid; i < n * quads; i += kConsumers) {
        const int t = i / quads, c = c0 + 4 * (i - t * quads), ch = c / kTile * kTile;
        const int64_t row = sh->pair[p0 + t];
        if (!AWQ_IN_BOUNDS(row >= 0 && row < a.T * a.top_k && c + 4 <= inter, 0xB0D7u)) continue;
        const int2 gb = up.blocks(up.at(seg, 2 * (c / kTile))), ub = up.blocks(up.at(seg, 2 * (c / kTile) + 1));
        if (!AWQ_IN_BOUNDS(gb.x >= 0 && ub.x >= 0 && gb.y < (int)gridDim.x && ub.y < (int)gridDim.x && t < C::kTok, 0xB0D8u)) continue;
        // part j: a whole tile's sums, or those of the j-th of its blocks, which but for the first enter inside it
        const auto part = [&](int2 b, int64_t off) {
          return [=](int j) {
            return b.x == b.y ? a.sums + row * pitch_gu + off + c : slot(b.x + j, j == 0) + t * kTile + c - ch;
          };
        };
        float4 gv, uv;
        sum_parts(gb.y - gb.x + 1, part(gb, 0), ub.y - ub.x + 1, part(ub, a.inter), gv, uv);
        const float h[4] = {silu_mul(gv.x, uv.x), silu_mul(gv.y, uv.y), silu_mul(gv.z, uv.z), silu_mul(gv.w, uv.w)};
        __align__(8) __half hi[4], rest[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hi[k] = __float2half_rn(h[k]);
          const float v = __half2float(hi[k]);
          rest[k] = __float2half_rn(isfinite(v) ? h[k] - v : 0.0f);
        }
        __half *d = a.H + row * inter + c;
        *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<const uint2 *>(hi);
        if (rest_too) *reinterpret_cast<uint2 *>(d + (int64_t)a.T * a.top_k * inter) = *reinterpret_cast<const uint2 *>(rest);
      }
    };
    ok = grid_barrier(a.barrier + 1, &sh->flag, st, a.max_polls, 0xE11u);
    if (ok && own_h) {  // other blocks may write the same values
      each_stretch(down, (int)blockIdx.x, [&](const Stretch &s, int u0, int u1) {
        finish(s.seg, u0 * 128, min(u1 * 128, inter));
      });
      asm volatile("bar.sync 2, 288;" ::: "memory");  // the producer waits for it
    } else if (ok) {
      const int pieces = (inter + kPieceH - 1) / kPieceH;
      for (int i = blockIdx.x; i < up.n_seg * pieces; i += gridDim.x) {
        const int c = i % pieces * kPieceH;
        finish(i / pieces, c, min(c + kPieceH, inter));
      }
      ok = grid_barrier(a.barrier + 2, &sh->flag, st, a.max_polls, 0xE13u);
    }
    if (ok)
      each_stretch(down, (int)blockIdx.x, [&](const Stretch &s, int u0, int u1) {
        const int seg = s.seg, ch = s.tile * kTile, p0 = sh->seg_first[seg], n = sh->seg_n[seg];
        const bool whole = u0 == 0 && u1 == down.len;
        float *part = dn_slot(blockIdx.x, u0 == 0);
        const int rows = h_rows(n), pairs = a.T * a.top_k;
        sums(rows, u0 * 128, min(u1 * 128, inter), min(kTile, hidden - ch), [&](int t) {
          // the remainders' sums have rows of their own
          return whole ? a.dn_sums + (int64_t)(t < n ? sh->pair[p0 + t] : pairs + sh->pair[p0 + t - n]) * hidden + ch
                       : part + t * kTile;
        });
      });
  }
  if (!ok) return;
  if (!grid_barrier(a.barrier + 3, &sh->flag, st, a.max_polls, 0xE12u)) return;

  // ---------------------------------------------------------------- combine
  // A warp takes 32 / kp quads of four outputs, kp lanes to a quad: a token's choices
  // side by side (their sums meet in a fixed tree)
  int kp = 1;
  while (kp < a.top_k) kp *= 2;
  const int quads = hidden / 4, qw = 32 / kp, groups = (quads + qw - 1) / qw;
  const int lane = tid & 31, k = lane / qw;
  for (int i = blockIdx.x + gridDim.x * (tid >> 5); i < a.T * groups; i += gridDim.x * (kThreads / 32)) {
    const int t = i / groups, quad = (i - t * groups) * qw + lane % qw, o = 4 * quad;
    const int p = t * a.top_k + k, at = quad < quads && k < a.top_k ? sh->where[p] : -1;  // -1: a masked row
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (at >= 0) {
      int seg = 0, hi = down.n_seg;  // the entry that holds position `at`
      while (hi - seg > 1) {
        const int m = (seg + hi) / 2;
        if (sh->seg_first[m] <= at)
          seg = m;
        else
          hi = m;
      }
      const int n = sh->seg_n[seg], row = at - sh->seg_first[seg];
      const int2 db = down.blocks(down.at(seg, o / kTile));
      const int parts = db.y - db.x + 1, w = o % kTile;
      const bool in = AWQ_IN_BOUNDS(db.x >= 0 && db.y < (int)gridDim.x && row < n && h_rows(n) <= C::kTok && p < a.T * a.top_k, 0xB0D9u);
      const auto part = [&](int j, int rest) -> const float * {
        return parts == 1 ? a.dn_sums + (int64_t)(rest * a.T * a.top_k + p) * hidden + o
                          : a.dn_partial + (((int64_t)db.x + j) * 2 + (j == 0)) * C::kTok * kTile + (rest * n + row) * kTile + w;
      };
      float4 v, r;
      sum_parts(in ? parts : 0, [&](int j) { return part(j, 0); }, in && h_rows(n) > n ? parts : 0, [&](int j) { return part(j, 1); }, v, r);
      const float pw = sh->wt[p];
      y = make_float4(pw * (v.x + r.x), pw * (v.y + r.y), pw * (v.z + r.z), pw * (v.w + r.w));
    }
    for (int d = qw; d < 32; d *= 2) {
      y.x += __shfl_xor_sync(0xffffffffu, y.x, d);
      y.y += __shfl_xor_sync(0xffffffffu, y.y, d);
      y.z += __shfl_xor_sync(0xffffffffu, y.z, d);
      y.w += __shfl_xor_sync(0xffffffffu, y.w, d);
    }
    if (k == 0 && quad < quads && AWQ_IN_BOUNDS(t < a.T && o + 4 <= hidden, 0xB0DAu)) {
      const __half2 h0 = __floats2half2_rn(y.x, y.y), h1 = __floats2half2_rn(y.z, y.w);
      *reinterpret_cast<uint2 *>(a.Y + t * a.ldy + o) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
    }
  }
}

// The status word and the counters, 512 bytes
__global__ void moe_clear_kernel(uint4 *ws) {
  pdl_wait();
  ws[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
}

template <int V, int SHIFT>
cudaError_t go(const MoeArgs &a, int num_sms, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  cudaError_t e = allow_smem(moe_kernel<V, SHIFT>, moe_smem<V>(), done);
  if (e != cudaSuccess) return e;
  CUtensorMap gu, dn;  // the words of all experts as pairs of 16-bit values
  e = make_tmap_f16_box(&gu, a.gu_q, a.experts * a.hidden, a.inter / 2, a.inter / 2, 64, kBoxK);
  if (e != cudaSuccess) return e;
  e = make_tmap_f16_box(&dn, a.dn_q, a.experts * a.inter, a.hidden / 4, a.hidden / 4, 64, kBoxK);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(Cfg<V>::kBlocks * num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = moe_smem<V>();
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel<V, SHIFT>, a, gu, dn);
}
template <int V>
cudaError_t go_group(const MoeArgs &a, int num_sms, cudaStream_t stream) {
  return a.group == 128  ? go<V, 7>(a, num_sms, stream)
         : a.group == 64 ? go<V, 6>(a, num_sms, stream)
                         : go<V, 5>(a, num_sms, stream);
}
}  // namespace

cudaError_t launch_moe(const MoeArgs &a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_after(moe_clear_kernel, 1, 32, 0, stream, reinterpret_cast<uint4 *>(a.st));
  if (e != cudaSuccess) return e;
  return a.T <= 8 ? go_group<1>(a, num_sms, stream) : go_group<2>(a, num_sms, stream);
}

AWQ_BOUNDS_READER(bounds_status_moe)

MoeLayout moe_layout(int64_t T, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k, int num_sms) {
  MoeLayout l;
  const int64_t pairs = T * top_k;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  size_t off = 512;
  l.logits = off;
  off = up(off + sizeof(double) * (size_t)(T * experts));
  l.H = off;  // and the remainders
  off = up(off + 2 * sizeof(__half) * (size_t)(pairs * inter));
  l.sums = off;  // whole tiles' sums: gate|up, and down (the remainders' apart)
  off = up(off + 2 * sizeof(float) * (size_t)(pairs * inter));
  l.dn_sums = off;
  off = up(off + 2 * sizeof(float) * (size_t)(pairs * hidden));
  const int64_t blocks = T <= 8 ? 2 * num_sms : num_sms, rows = T <= 8 ? 8 : kCap;
  l.partial = off;  // split tiles' sums, by block
  off = up(off + sizeof(float) * (size_t)(blocks * 2 * rows * kTile));
  l.dn_partial = off;
  off = up(off + sizeof(float) * (size_t)(blocks * 2 * rows * kTile));
  l.end = off;
  return l;
}

}  // namespace awq
