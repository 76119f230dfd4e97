// The adapter product for many tokens (more than 64), on the 5th-generation
// tensor cores:
//
//   Y = X Wd^T + sum over the tile's adapters a of mask_a(U) B_a^T,
//   Wd = RN16((q - z) scale),  U[t] = RN16( c_a (x_t A_a^T) ),  a = ids[t]
//
// (a row of U past fp16's range stays fp32, and its part is added to the accumulators).
//
// Three launches.  lora_shrink_mma_kernel computes U and, for every token tile of
// the product, the list of the adapters its rows carry; beside it (programmatic
// dependent launch) lora_dequant_kernel dequantises W once, in x out work instead
// of once per token tile.
// lora_gemm_kernel: the low-rank part is K steps like any other, appended to a
// tile's K loop for each adapter on its list: A is U's rows, which the waiting
// epilogue warps write to shared memory from registers, those of other adapters as
// zeros, B is B_a's rows by TMA.  No partial result leaves the accumulators, so the whole is
// rounded once, and the part costs rank / in of the product for rows that stand
// together by adapter.
//
// Measured, replayed: 138 us for 1531 tokens on 4096 x 11008 at rank 32 (the product
// 110, two rounds of 256 x 256 tiles on 148 SMs, 735 ns a step of 64 columns = 1.69
// PFLOP/s while a tile is at work), 245-251 us for 8192 on 4096 x 4096 at rank 16 (product
// 213); bound by the tensor cores at the clock they hold.  Tiles with values that leave the
// product (non-finite B, rows of U past fp16) are stored 8 columns at a time with those
// terms added in fp32: 253 us for the 1531 tokens with one infinity in one adapter's B, 1.2
// ms with every row of U past fp16.
#include <cuda.h>

#include "awq_launch.h"
#include "serve_launch.h"
#include "w4_dequant.cuh"

namespace awq {
namespace {

// ---------------------------------------------------------------------------
// Preparation
// ---------------------------------------------------------------------------
constexpr int kShT = 16;      // tokens of a shrink block
constexpr int kShR = 32;      // rank rows of a pass
constexpr int kShWarps = 16;
constexpr int kShThreads = kShWarps * 32;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The different adapters of n <= 256 ids (shared memory), in order of appearance,
// into list; returns how many.  All threads of the block.
__device__ int adapter_list(const int *ids, int n, int *list, int *scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int id = tid < n ? ids[tid] : -1;
  bool first = id >= 0;
  for (int s = 0; s < tid && first; ++s) first = ids[s] != id;
  const uint32_t b = __ballot_sync(0xffffffffu, first);
  if (lane == 0 && warp < 8) scratch[warp] = __popc(b);
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < 8; ++w) {
    at += w < warp ? scratch[w] : 0;
    total += scratch[w];
  }
  if (first) list[at + __popc(b & ((1u << lane) - 1u))] = id;
  __syncthreads();
  return total;
}

// 8 NX rank rows of one adapter: X (16 rows) times A_a^T on mma.sync over this
// warp's steps of 32 columns, the loads of four steps in flight together.  A lane
// loads 16 bytes of a row: the 8 columns 8q .. 8q + 7 of a step are its fragments of
// two MMAs, the order of k inside a step being free as long as both operands agree.
template <int NX>
__device__ __forceinline__ void shrink_pass(float (&acc)[4][4], const __half *x0, const __half *x1, const __half *ar,
                                            int64_t in, int s0, int s1) {
  for (int s = s0; s < s1; s += 4) {
    uint4 xa[4], xb[4], av[4][NX];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s + i < s1) {
        xa[i] = __ldg(reinterpret_cast<const uint4 *>(x0 + 32 * (s + i)));
        xb[i] = __ldg(reinterpret_cast<const uint4 *>(x1 + 32 * (s + i)));
#pragma unroll
        for (int x = 0; x < NX; ++x) av[i][x] = __ldg(reinterpret_cast<const uint4 *>(ar + 8 * x * in + 32 * (s + i)));
      } else {
        xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int x = 0; x < NX; ++x) av[i][x] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        mma16816(acc[x], xa[i].x, xb[i].x, xa[i].y, xb[i].y, av[i][x].x, av[i][x].y);
        mma16816(acc[x], xa[i].z, xb[i].z, xa[i].w, xb[i].w, av[i][x].z, av[i][x].w);
      }
  }
}

// The rank rows of an adapter go in passes of 32, then 16 and 8: the i-th one's first
// row and its rows.
__device__ __forceinline__ int2 shrink_rows(int rank, int i) {
  const int full = rank / 32, left = rank % 32;
  if (i < full) return make_int2(32 * i, 32);
  if (i == full && left >= 16) return make_int2(32 * full, 16);
  return make_int2(rank - 8, 8);
}
__host__ __device__ constexpr int shrink_passes(int rank) { return rank / 32 + (rank / 16 & 1) + (rank / 8 & 1); }

// U of 16 tokens for the adapters among them: items of an adapter and a pass.
// `split` of the 16 warps share an item's K, so that each has at least four steps of
// it, and the others take other items.  `shares` blocks deal the items of the same
// tokens out between them (this is the `share`-th).
__device__ void shrink_block(const LoraArgs &a, int64_t t0, int share, int shares, uint8_t *smem) {
  float *red = reinterpret_cast<float *>(smem);  // [16][16][kShR + 1]
  int *ids = reinterpret_cast<int *>(smem + kShWarps * kShT * (kShR + 1) * 4);
  int *list = ids + 256, *scratch = list + 256;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int n = (int)i64min(kShT, a.T - t0);
  if (tid < kShT) {
    const int id = tid < n ? a.ids[t0 + tid] : -1;
    ids[tid] = id >= 0 && id < a.adapters ? id : -1;
  }
  __syncthreads();
  const int passes = shrink_passes(a.rank), items = adapter_list(ids, n, list, scratch) * passes;
  const int steps = (int)(a.in / 32);
  int split = kShWarps;
  while (split > 1 && split * 4 > steps) split /= 2;
  const int teams = kShWarps / split, team = warp / split, part = warp - team * split;
  const int s0 = steps * part / split, s1 = steps * (part + 1) / split;
  // rows g and g + 8 (the last one again past the end)
  const __half *x0 = a.X + (t0 + min(g, n - 1)) * a.ldx + 8 * q, *x1 = a.X + (t0 + min(g + 8, n - 1)) * a.ldx + 8 * q;
  for (int i0 = share * teams; i0 < items; i0 += shares * teams) {
    if (i0 + team < items && AWQ_IN_BOUNDS(list[(i0 + team) / passes] >= 0 && list[(i0 + team) / passes] < a.adapters, 0xB0B1u)) {
      const int j = (i0 + team) / passes;
      const int2 rows = shrink_rows(a.rank, i0 + team - j * passes);
      float acc[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[x][c] = 0.0f;
      const __half *ar = a.A + ((int64_t)list[j] * a.rank + rows.x + g) * a.in + 8 * q;
      if (rows.y == 32)
        shrink_pass<4>(acc, x0, x1, ar, a.in, s0, s1);
      else if (rows.y == 16)
        shrink_pass<2>(acc, x0, x1, ar, a.in, s0, s1);
      else
        shrink_pass<1>(acc, x0, x1, ar, a.in, s0, s1);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          red[(warp * kShT + g + 8 * (c >> 1)) * (kShR + 1) + 8 * x + 2 * q + (c & 1)] = acc[x][c];
    }
    __syncthreads();
    for (int i = tid; i < min(teams, items - i0) * kShT * kShR; i += kShThreads) {
      const int m = i / (kShT * kShR), t = i / kShR % kShT, r = i % kShR, j = (i0 + m) / passes, id = list[j];
      const int2 rows = shrink_rows(a.rank, i0 + m - j * passes);
      if (r >= rows.y || t >= n || ids[t] != id) continue;
      if (!AWQ_IN_BOUNDS(t0 + t < a.T && rows.x + r < a.rank, 0xB0B0u)) continue;
      float v = 0.0f;
      for (int w = 0; w < split; ++w) v += red[((m * split + w) * kShT + t) * (kShR + 1) + r];
      const int64_t at = (t0 + t) * a.rank + rows.x + r;
      const float u = a.c[id] * v;
      a.U[at] = u;
      __half h = __float2half_rn(u);
      if (u != 0.0f && __heq(h, __float2half_rn(0.0f))) h = __float2half_rn(copysignf(0x1p-24f, u));  // past_fp16
      reinterpret_cast<__half *>(a.U + a.T * a.rank)[at] = h;
    }
    __syncthreads();
  }
}

constexpr int kShrinkSmem = kShWarps * kShT * (kShR + 1) * 4 + (256 + 256 + 16) * 4;

// Blocks [0, n_shrink shares): U; the rest: the lists of `bm`-row tiles,
// lists[tile][bm + 1] = count, ids.
__global__ void __launch_bounds__(kShThreads)
    lora_shrink_mma_kernel(const LoraArgs a, int n_shrink, int shares, int bm, int *lists) {
  __shared__ __align__(16) uint8_t smem[kShrinkSmem];
  pdl_wait();
  pdl_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.st = DevStatus{};
  int64_t b = blockIdx.x;
  if (b < (int64_t)n_shrink * shares) {
    shrink_block(a, b % n_shrink * kShT, (int)(b / n_shrink), shares, smem);
    return;
  }
  b -= (int64_t)n_shrink * shares;
  int *ids = reinterpret_cast<int *>(smem), *list = ids + 256, *scratch = list + 256;
  const int64_t t0 = b * bm;
  const int n = (int)i64min(bm, a.T - t0), tid = threadIdx.x;
  const int id = tid < n ? a.ids[t0 + tid] : -1;
  if (tid < 256) ids[tid] = id >= 0 && id < a.adapters ? id : -1;
  __syncthreads();
  const int count = adapter_list(ids, n, list, scratch);
  if (!AWQ_IN_BOUNDS(t0 < a.T && count <= n, 0xB0B2u)) return;
  int *dst = lists + b * (bm + 1);
  if (tid == 0) dst[0] = count;
  if (tid < count) dst[1 + tid] = list[tid];
}

__global__ void __launch_bounds__(256) lora_dequant_kernel(const LoraArgs a, __half *Wd) {
  __shared__ __align__(16) __half tile[kWideIn * kWideOut];
  const int64_t tiles_o = (a.out + kWideOut - 1) / kWideOut, b = blockIdx.x;
  dequant_wide(tile, a.qweight, a.qzeros, a.scales, a.in, a.out, a.group, b % tiles_o * kWideOut,
               b / tiles_o * kWideIn, Wd);
  pdl_wait();  // its end is the shrink product's too
}

// ---------------------------------------------------------------------------
// Product.  One block per SM, persistent over BM x BN tiles: warp 0 TMA, warp 1
// MMA, warps 2..9 write the adapters' A operands and store the tile.
// ---------------------------------------------------------------------------
constexpr int PK = 64;
constexpr uint32_t kPDrain = 1u << 22;
constexpr int kGroupM = 16;  // token tiles whose X stays in L2 while the output tiles stream past

template <int BM, int BN>
struct PCfg {
  static constexpr int kMT = BM / 128;  // MMAs of M = 128 per K substep
  static constexpr uint32_t kA = BM * PK * 2, kB = BN * PK * 2;
  static constexpr int kStages = (int)(196608 / (kA + kB));
  static constexpr int kAccs = 512 / (kMT * BN) >= 2 ? 2 : 1;  // tiles in tensor memory
  static constexpr uint32_t kCols = kAccs * kMT * BN;
  static constexpr uint32_t kOut = 8 * 4096;  // 32 rows x 64 columns of each storing warp
  static constexpr uint32_t kBytes = 1024 + kStages * (kA + kB) + kOut + 512;
};

template <int STAGES>
struct __align__(8) PTail {
  uint64_t full[STAGES], empty[STAGES];  // words of X and Wd; read
  uint64_t ufull[STAGES], masked[STAGES];  // B_a landed; U written
  uint64_t tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort_flag;
  // the last tile, by i % 4 of the block's i-th (the warps are at most two apart), in which
  // B has values that are not finite, or rows of U are past fp16: i + 1
  volatile int odd[4];
};

// Of the two fp16 of w, the sign bits of those that are infinite or NaN.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }

// A row of B_a's landed box (16-byte chunks i, i + STEP, .. of `chunks`, swizzled by the
// row): non-zero where a value is not finite.
template <int STEP>
__device__ __forceinline__ uint32_t row_non_finite(const uint8_t *row, int swizzle, int first, int chunks) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 8; i += STEP)
    if (first + i < chunks) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + (((first + i) ^ swizzle) * 16));
      any |= non_finite(v.x) | non_finite(v.y) | non_finite(v.z) | non_finite(v.w);
    }
  return any;
}

// The same row with 0 for what is not finite.
__device__ __noinline__ void make_finite(uint8_t *row, int swizzle, int i, int step, int chunks) {
  for (; i < chunks; i += step) {
    uint32_t *p = reinterpret_cast<uint32_t *>(row + ((i ^ swizzle) * 16));
    for (int k = 0; k < 4; ++k) p[k] &= ~((non_finite(p[k]) >> 15) * 0xFFFFu);
  }
}

// 8 columns of tensor memory, waited for.
__device__ __forceinline__ void tmem_columns8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Whether a row of U is no operand of fp16: its largest value past the type's range, or so
// small that the type's smallest step, 2^-24, is no longer small beside it (a value that
// rounds to 0 is stored as that step, so that the row's fp16 form tells).  A row with a NaN
// is one: all its outputs are NaN.
__device__ __forceinline__ bool past_fp16(const __half *u, int rank) {
  uint32_t m = 0;
#pragma unroll 4
  for (int r = 0; r < rank; r += 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(u + r));
    m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), __vmaxu2(__vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu));
  }
  m = max(m & 0xFFFFu, m >> 16);
  return m == 0x7C00u || (m != 0 && m < 0x0C00u);  // infinity; 2^-12
}

// Adds to v the terms U[t][r] B_a[o][r] of 8 outputs (b: the first one's row) that are not
// in the product: those that make_finite took out, or all of a row of U past fp16.
__device__ __noinline__ void left_out(float (&v)[8], const float *u, const __half *b, int rank, bool all) {
  for (int r = 0; r < rank; r += 8) {
    uint4 w[8];
    const float4 x0 = __ldg(reinterpret_cast<const float4 *>(u + r)), x1 = __ldg(reinterpret_cast<const float4 *>(u + r) + 1);
    const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(b + (int64_t)i * rank + r));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      if (!all && !(non_finite(h[0]) | non_finite(h[1]) | non_finite(h[2]) | non_finite(h[3]))) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float y = __half2float(__ushort_as_half((unsigned short)(h[k / 2] >> (16 * (k & 1)))));
        if (all || !isfinite(y)) v[i] = fmaf(x[k], y, v[i]);
      }
    }
  }
}

template <int STAGES>
__device__ __forceinline__ void p_abort(PTail<STAGES> *t, DevStatus *st, uint32_t where) {
  dev_fail(st, kDevTimeout, where);
  *reinterpret_cast<volatile int *>(&t->abort_flag) = 1;
}

struct PrefillArgs {
  const int32_t *ids;
  const float *U;   // [T, rank], and as fp16
  const __half *U16, *B;
  const int *lists;
  int64_t T, out, ldy;
  int adapters, rank, num_m, num_n, num_kb;
  __half *Y;
  DevStatus *st;
  uint32_t max_polls;
};

__device__ __forceinline__ void p_tile(int tile, int num_m, int num_n, int &m, int &n) {
  const int per = kGroupM * num_n, grp = tile / per, first = grp * kGroupM;
  const int gm = min(kGroupM, num_m - first), local = tile - grp * per;
  m = first + local % gm;
  n = local / gm;
}

template <int BM, int BN>
__global__ void __launch_bounds__(320, 1)
    lora_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ PrefillArgs a) {
  using C = PCfg<BM, BN>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *sA = smem, *sB = smem + STAGES * C::kA;
  uint8_t *sOut = sB + STAGES * C::kB;
  auto *tail = reinterpret_cast<PTail<STAGES> *>(sOut + C::kOut);
  volatile int *abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = a.num_m * a.num_n;
  const int rsteps = (a.rank + PK - 1) / PK;  // K steps of an adapter

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
      mbar_init(&tail->ufull[s], 1);
      mbar_init(&tail->masked[s], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->tfull[i], 2);  // the MMAs' end, and the issuing thread
      mbar_init(&tail->tempty[i], 8);
    }
    mbar_init(&tail->done, 1);
    tail->abort_flag = 0;
    for (int i = 0; i < 4; ++i) tail->odd[i] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&tail->tmem, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem;
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t step = 0, fphase = 0, uphase = 0, last_u = 0;  // per stage: phases, and whose copy is the last
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        int m, n;
        p_tile(tile, a.num_m, a.num_n, m, n);
        const int *list = a.lists + (int64_t)m * (BM + 1);
        const int steps = a.num_kb + list[0] * rsteps;
        for (int k = 0; k < steps; ++k, ++step) {
          const int s = step % STAGES;
          if (!mbar_wait_long(&tail->empty[s], ((step / STAGES) & 1u) ^ 1u, a.max_polls, abort_flag)) {
            p_abort(tail, a.st, 0xE30u);
            ok = false;
            break;
          }
          const bool low = k >= a.num_kb;
          uint64_t *bar = low ? &tail->ufull[s] : &tail->full[s];
          mbar_arrive_expect_tx(bar, low ? C::kB : C::kA + C::kB);
          if (!low) {
            tma_load_2d(sA + s * C::kA, &tmX, bar, k * PK, m * BM);
            tma_load_2d(sB + s * C::kB, &tmW, bar, k * PK, n * BN);
          } else {
            const int e = (k - a.num_kb) / rsteps, r = (k - a.num_kb) % rsteps;
            // rows past this adapter's outputs are the next one's: their columns are not stored
            tma_load_2d(sB + s * C::kB, &tmB, bar, r * PK, (int)(list[1 + e] * a.out + n * BN));
          }
          (low ? uphase : fphase) ^= 1u << s;
          last_u = (last_u & ~(1u << s)) | (low ? 1u << s : 0u);
        }
      }
      if (!ok || *abort_flag)  // own copies in flight
        for (uint32_t s = 0; s < STAGES && s < step; ++s) {
          const bool low = (last_u >> s) & 1u;
          (void)mbar_wait_bounded(low ? &tail->ufull[s] : &tail->full[s],
                                  (((low ? uphase : fphase) >> s) & 1u) ^ 1u, kPDrain, nullptr);
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t step = 0, fphase = 0, mphase = 0;  // phases per stage
      constexpr uint32_t idesc = idesc_f16_f32(128, BN);
      int it = 0;
      bool ok = true, issued = false;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, ++it) {
        int m, n;
        p_tile(tile, a.num_m, a.num_n, m, n);
        const int steps = a.num_kb + a.lists[(int64_t)m * (BM + 1)] * rsteps;
        const int acc = it % C::kAccs;
        if (!mbar_wait_long(&tail->tempty[acc], ((it / C::kAccs) & 1) ^ 1u, a.max_polls, abort_flag)) {
          p_abort(tail, a.st, 0xE31u);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + acc * (C::kMT * BN);
        for (int k = 0; k < steps; ++k, ++step) {
          const int s = step % STAGES;
          bool got;
          int subs = PK / 16;
          if (k < a.num_kb) {
            got = mbar_wait_bounded(&tail->full[s], (fphase >> s) & 1u, a.max_polls, abort_flag);
            fphase ^= 1u << s;
          } else {
            got = mbar_wait_long(&tail->masked[s], (mphase >> s) & 1u, a.max_polls, abort_flag);
            mphase ^= 1u << s;
            const int left = a.rank - (k - a.num_kb) % rsteps * PK;  // the rest of the box is zero
            subs = left < PK ? (left + 15) / 16 : PK / 16;
          }
          if (!got) {
            p_abort(tail, a.st, 0xE32u);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(sA + s * C::kA), sb = smem_u32(sB + s * C::kB);
          for (int kk = 0; kk < subs; ++kk) {
            const uint64_t bd = smem_desc_k_sw128(sb + kk * 32);
#pragma unroll
            for (int h = 0; h < C::kMT; ++h)
              tc_mma_f16(d + h * BN, smem_desc_k_sw128(sa + h * 128 * PK * 2 + kk * 32), bd, idesc,
                         (k | kk) != 0 ? 1u : 0u);
          }
          issued = true;
          tc_commit(&tail->empty[s]);
        }
        if (!ok) break;
        tc_commit(&tail->tfull[acc]);
        mbar_arrive(&tail->tfull[acc]);  // hands on what the `masked` arrivals showed this thread (odd)
      }
      if (issued) {
        tc_commit(&tail->done);
        (void)mbar_wait_bounded(&tail->done, 0, kPDrain, nullptr);
      }
    }
  } else {
    // warps 2..9: lane quarter q of tensor memory; with two MMA halves warps 2..5
    // and 6..9 take one each, else half of the columns each
    const int q = warp & 3, part = (warp - 2) >> 2, tid = threadIdx.x - 64;
    uint32_t step = 0, uphase = 0;
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, ++it) {
      int m, n;
      p_tile(tile, a.num_m, a.num_n, m, n);
      const int *list = a.lists + (int64_t)m * (BM + 1);
      const int count = list[0];
      step += a.num_kb;
      if (count) {
        const int64_t row = (int64_t)m * BM + tid;  // tid >= BM: no row
        int id = tid < BM && row < a.T ? a.ids[row] : -1;
        if (!AWQ_IN_BOUNDS(count <= BM, 0xB0B5u)) id = -1;
        const uint4 *u = reinterpret_cast<const uint4 *>(a.U16 + row * a.rank);
        const auto chunk = [&](int i) {  // 8 values of this row's U
          return id >= 0 && 8 * i < a.rank ? __ldg(u + i) : make_uint4(0u, 0u, 0u, 0u);
        };
        const bool past = id >= 0 && past_fp16(a.U16 + row * a.rank, a.rank);
        int next = list[1];
        for (int e = 0; e < count && ok; ++e) {
          const bool mine = id == next && !past;
          if (id == next && past) tail->odd[it & 3] = it + 1;
          if (e + 1 < count) next = list[2 + e];
          for (int r = 0; r < rsteps; ++r, ++step) {
            const int s = step % STAGES, left = min(PK, a.rank - r * PK);
            uint4 v[PK / 8];  // on its way while B_a is
#pragma unroll
            for (int i = 0; i < PK / 8; ++i) v[i] = mine ? chunk(PK / 8 * r + i) : make_uint4(0u, 0u, 0u, 0u);
            int got = 1;
            if (lane == 0) got = mbar_wait_long(&tail->ufull[s], (uphase >> s) & 1u, a.max_polls, abort_flag);
            uphase ^= 1u << s;
            got = __shfl_sync(0xffffffffu, got, 0);
            if (!got) {
              if (lane == 0) p_abort(tail, a.st, 0xE33u);
              ok = false;
              break;
            }
            __syncwarp();
            // The other rows' zeros meet B_a too, and 0 x infinity is NaN: what is not finite
            // leaves the box, and is added to the adapter's own rows at the end (0.13 us a step of
            // 128 rows; looking the adapters over beforehand would read B_a once more)
            const int chunks = n * BN + tid % BN < a.out ? left / 8 : 0;
            uint8_t *brow = sB + s * C::kB + tid % BN * (PK * 2);
            const uint32_t bad = row_non_finite<256 / BN>(brow, tid & 7, tid / BN, chunks);
            if (tid < BM) {
              uint4 *d = reinterpret_cast<uint4 *>(sA + s * C::kA + tid * (PK * 2));
#pragma unroll
              for (int i = 0; i < PK / 8; ++i)  // 128-byte swizzle; the MMAs of 16 columns that are issued
                if (8 * (i & ~1) < left) d[i ^ (tid & 7)] = v[i];
            }
            if (__any_sync(0xffffffffu, bad != 0)) {
              make_finite(brow, tid & 7, tid / BN, 256 / BN, chunks);
              tail->odd[it & 3] = it + 1;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail->masked[s]);
          }
        }
        if (!ok) break;
      }
      const int acc = it % C::kAccs;
      int got = 1;
      if (lane == 0) got = mbar_wait_long(&tail->tfull[acc], (it / C::kAccs) & 1u, a.max_polls, abort_flag);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        if (lane == 0) p_abort(tail, a.st, 0xE34u);
        break;
      }
      tc_fence_after();
      // A lane has a row's values: 64 columns at a time go through shared memory (16-byte
      // chunks exchanged by the row, so that both sides meet all banks), whose rows the
      // warp stores 128 bytes at a time: 3 us a tile, 6.5 with each lane storing its row
      const int64_t t = (int64_t)m * BM + (C::kMT == 2 ? part * 128 : 0) + q * 32;
      const int c0 = C::kMT == 2 ? 0 : part * (BN / 2), c1 = C::kMT == 2 ? BN : c0 + BN / 2;
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + acc * (C::kMT * BN) + (C::kMT == 2 ? part * BN : 0);
      uint8_t *stage = sOut + (warp - 2) * 4096;
      const bool odd = count && tail->odd[it & 3] == it + 1;
      if (odd) {  // a lane its row, 8 columns at a time, with what is not in the product
        const int id = t + lane < a.T ? a.ids[t + lane] : -1;
        const bool on = id >= 0 && id < a.adapters;
        const float *u = a.U + (t + lane) * a.rank;
        const bool past = on && past_fp16(a.U16 + (t + lane) * a.rank, a.rank);
#pragma unroll 1
        for (int c = c0; c < c1; c += 8) {
          float v[8];
          tmem_columns8(d + c, v);
          const int64_t o = (int64_t)n * BN + c;
          if (t + lane < a.T && o < a.out && AWQ_IN_BOUNDS(o + 8 <= a.out, 0xB0B4u)) {
            if (on) left_out(v, u, a.B + (id * a.out + o) * a.rank, a.rank, past);
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const __half2 p = __floats2half2_rn(v[2 * h], v[2 * h + 1]);
              w[h] = *reinterpret_cast<const uint32_t *>(&p);
            }
            *reinterpret_cast<uint4 *>(a.Y + (t + lane) * a.ldy + o) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
        }
      }
#pragma unroll 1
      for (int c = odd ? c1 : c0; c < c1; c += 64) {
        float v[64];
        tmem_ld_32x32b_x32(d + c, *reinterpret_cast<float(*)[32]>(v));
        tmem_ld_32x32b_x32(d + c + 32, *reinterpret_cast<float(*)[32]>(v + 32));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const __half2 p = __floats2half2_rn(v[8 * i + 2 * h], v[8 * i + 2 * h + 1]);
            w[h] = *reinterpret_cast<const uint32_t *>(&p);
          }
          *reinterpret_cast<uint4 *>(stage + lane * 128 + ((i ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int64_t o = (int64_t)n * BN + c + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          if (t + row < a.T && o < a.out && AWQ_IN_BOUNDS(o + 8 <= a.out, 0xB0B3u))
            *reinterpret_cast<uint4 *>(a.Y + (t + row) * a.ldy + o) =
                *reinterpret_cast<const uint4 *>(stage + row * 128 + (((lane & 7) ^ (row & 7)) * 16));
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->tempty[acc]);
    }
  }
  for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * blockDim.x)
    if (a.ids[t] < -1 || a.ids[t] >= a.adapters) dev_fail(a.st, kDevBadAdapter, 0xE02u);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int BM, int BN>
cudaError_t launch_product(const LoraArgs &a, const int *lists, const __half *Wd, int num_sms, cudaStream_t stream) {
  using C = PCfg<BM, BN>;
  static std::atomic<bool> done[64];
  static_assert(sizeof(PTail<C::kStages>) <= 512 && C::kBytes <= 232448, "shared memory");
  cudaError_t e = allow_smem(lora_gemm_kernel<BM, BN>, C::kBytes, done);
  if (e != cudaSuccess) return e;
  CUtensorMap x, w, b;
  if ((e = make_tmap_f16_box(&x, a.X, a.T, a.in, a.ldx, PK, BM)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_box(&w, Wd, a.out, a.in, a.in, PK, BN)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_box(&b, a.B, (int64_t)a.adapters * a.out, a.rank, a.rank, PK, BN)) != cudaSuccess) return e;
  const PrefillArgs p = {a.ids, a.U, reinterpret_cast<const __half *>(a.U + a.T * a.rank), a.B, lists, a.T, a.out, a.ldy, a.adapters, a.rank, (int)((a.T + BM - 1) / BM),
                         (int)((a.out + BN - 1) / BN), (int)(a.in / PK), a.Y, a.st, a.max_polls};
  const int64_t tiles = (int64_t)p.num_m * p.num_n;
  return launch_after(lora_gemm_kernel<BM, BN>, i64min(tiles, num_sms), 320, C::kBytes, stream, x, w, b, p);
}
}  // namespace

// Token rows of a tile of the product.  A step of 64 columns of a 256 x 256 tile takes
// 735 ns (the tensor cores' rate at the clock they hold), one of a 128 x 128 tile 490
// (L2 feeds 148 SMs at 9.7 TB/s), and the SMs work in rounds of tiles: 785 tokens on 2816
// x 6176 take 92 us in three rounds of the small tiles and 48 in one of the large.
int lora_prefill_bm(int64_t T, int64_t out, int num_sms) {
  const auto rounds = [&](int64_t b) { return (((T + b - 1) / b) * ((out + b - 1) / b) + num_sms - 1) / num_sms; };
  return rounds(256) * 735 <= rounds(128) * 490 ? 256 : 128;
}

size_t lora_prefill_ws(int64_t T, int64_t in, int64_t out, int rank) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  return up((sizeof(float) + sizeof(__half)) * (size_t)T * rank) + up(sizeof(int) * (size_t)((T + 127) / 128) * 129) +
         up(sizeof(__half) * (size_t)in * out);
}

cudaError_t launch_lora_prefill(const LoraArgs &a, int num_sms, cudaStream_t stream) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  uint8_t *ws = reinterpret_cast<uint8_t *>(a.U);
  int *lists = reinterpret_cast<int *>(ws + up((sizeof(float) + sizeof(__half)) * (size_t)a.T * a.rank));
  __half *Wd = reinterpret_cast<__half *>(reinterpret_cast<uint8_t *>(lists) +
                                          up(sizeof(int) * (size_t)((a.T + 127) / 128) * 129));
  const int bm = lora_prefill_bm(a.T, a.out, num_sms);
  const int64_t n_shrink = (a.T + kShT - 1) / kShT, n_lists = (a.T + bm - 1) / bm;
  const int64_t n_deq = ((a.out + kWideOut - 1) / kWideOut) * (a.in / kWideIn);
  // few tokens: as many blocks for each 16 as fill the SMs and as there can be items
  // (785 tokens with nine mixed adapters: 19 us, 31 with one)
  const int64_t most = i64min(kShT, a.adapters) * shrink_passes(a.rank);
  const int shares = (int)i64max(1, i64min(num_sms / n_shrink, most));
  if (n_shrink * shares + n_lists > INT32_MAX || n_deq > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = launch_after(lora_shrink_mma_kernel, n_shrink * shares + n_lists, kShThreads, 0, stream, a, (int)n_shrink, shares, bm,
                               lists);
  if (e == cudaSuccess) e = launch_after(lora_dequant_kernel, n_deq, 256, 0, stream, a, Wd);
  if (e != cudaSuccess) return e;
  return bm == 256 ? launch_product<256, 256>(a, lists, Wd, num_sms, stream)
                   : launch_product<128, 128>(a, lists, Wd, num_sms, stream);
}

AWQ_BOUNDS_READER(bounds_status_prefill)

}  // namespace awq
