// Streaming product of a few fp16 token rows with packed 4-bit weights on the
// warp-level tensor-core instruction: the core of the adapter product for few
// tokens (lora_gemm.cu) and of the mixture-of-experts layer (moe_layer.cu).
//
//   S[t][o] = sum over k in [k0, k1) of x[t][k] (q - z)[k][o] s[k/g][o]
//
// Mathematics.  Within a group the step is common: S = sum_groups s (sum_k
// (q - z) x).  The integers q - z are the A operand: a nibble at bit 0 (bit 4)
// of a 16-bit half, read as fp16, is the subnormal q 2^-24 (q 2^-20), so a code
// needs one AND and no conversion, and subtracting the zero point's subnormal
// is exact.  Products are exact in fp32, the group sums and their scaled total
// are fp32, and no weight is rounded to fp16.
//
// Layout.  m16n8k16: 16 rows = 8 word columns x 2 nibbles (p, p + 4), 8
// columns = 8 tokens.  Lane (g, q) reads word column g of input rows 2q, 2q + 1,
// 2q + 8, 2q + 9 of a 16-row step: four words give, after one byte permute per
// pair, a mask and a subtraction, the A fragments of four MMAs (p = 0..3), 64
// outputs per warp.  Words reach shared memory by TMA as boxes of 64 rows x 128
// bytes with the 128-byte swizzle, under which the four rows a quad reads lie in
// different banks.
//
// Eight consumer warps, four to each of a stage's two boxes, and one producer
// warp that issues every copy into a ring of stages; full and empty barriers let the warps
// drift apart by the depth of the ring, and the producer runs ahead into the
// next tile.  What the two boxes are is the mode's choice:
//   kN    the same 64 input rows of two 256-output column blocks;
//   kK    one column block, input rows 64 of two different 128-row halves: the
//         warp halves' sums are added at the end;
//   kTok  one column block, 128 consecutive input rows: every warp works
//         through both boxes for its half of the tokens.
//
// Measured (g = 128, words in shared memory): 207, 252 and 313 cycles for 16 rows x
// 512 outputs by 8 warps with 1, 2 and 3 token tiles, 260 for two such blocks on an
// SM with 1.  The bound is the instructions that make fragments of words (24 of them
// per 4 words and lane, at half rate) and mma.sync (8 cycles each and sub-partition),
// which two warps a sub-partition overlap in part.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "awq_device.cuh"

namespace awq {
namespace w4s {

constexpr int kConsumers = 256;
constexpr int kThreads = kConsumers + 32;      // the producer is warp 8
constexpr int kBoxN = 256;                     // outputs of a box
constexpr int kBoxK = 64;                      // input rows of a box
constexpr uint32_t kBoxBytes = kBoxK * 128;
constexpr uint32_t kSz = 640;                  // a group's 256 steps (fp16) and 32 zero words
constexpr uint32_t kXPitch = kBoxK * 2 + 16;   // bytes between token rows: conflict-free for ldmatrix

enum class Mode { kN, kK, kTok };

__host__ __device__ constexpr uint32_t x_offset() { return 2 * kBoxBytes; }
template <Mode M, int MAXTOK>
__host__ __device__ constexpr uint32_t sz_offset() {
  return x_offset() + (M == Mode::kN ? 1 : 2) * MAXTOK * kXPitch;
}
template <Mode M, int MAXTOK>
__host__ __device__ constexpr uint32_t stage_bytes() {
  return (sz_offset<M, MAXTOK>() + 4 * kSz + 1023) / 1024 * 1024;
}


__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
  const uint32_t n = ok ? 16u : 0u;  // 0: zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// One arrival on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// Whether the phase of `bar` has completed; does not wait.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

__device__ __forceinline__ uint32_t lds32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The barriers of a ring and whether a wait ran out.
template <int STAGES>
struct __align__(16) RingBars {
  uint64_t full[STAGES], empty[STAGES];
  int abort;
};

template <int STAGES>
__device__ __forceinline__ void ring_init(RingBars<STAGES> *b) {  // one thread
  for (int s = 0; s < STAGES; ++s) {
    mbar_init(&b->full[s], 1 + 32);  // the words' byte count, the producer's lanes
    mbar_init(&b->empty[s], kConsumers / 32);
  }
  b->abort = 0;
  fence_mbar_init();
}

// Bounded wait, uniform over the warp; false when it ran out here or elsewhere
// in the block (max_polls x 64 ns, as mbar_wait_long).
template <int STAGES>
__device__ __forceinline__ bool ring_wait(RingBars<STAGES> *b, uint64_t *bar, uint32_t parity, uint32_t max_polls,
                                          DevStatus *st, uint32_t site) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  if (!ok) ok = mbar_wait_long(bar, parity, max_polls, &b->abort);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) {
    if (!*reinterpret_cast<volatile int *>(&b->abort)) dev_fail(st, kDevTimeout, site);
    *reinterpret_cast<volatile int *>(&b->abort) = 1;
  }
  return false;
}

// Where a warp role stands in the ring; both roles count the same stages.
struct RingPos {
  uint32_t slot = 0, phase = 0, count = 0;
  template <int STAGES>
  __device__ __forceinline__ void next() {
    ++count;
    if (++slot == STAGES) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// After a wait ran out: waits (bounded) for the producer's own copies in flight.
template <int STAGES>
__device__ __forceinline__ void ring_drain(RingBars<STAGES> *b, const RingPos &pos) {
  for (uint32_t j = 1; j <= STAGES && j <= pos.count; ++j) {
    const uint32_t i = pos.count - j;
    (void)mbar_wait_bounded(&b->full[i % STAGES], (i / STAGES) & 1u, 1u << 20, nullptr);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One packed matrix [.., in, out]: its words' tensor map with the first row, and
// the first word column and the end of the columns of either box.
struct Weights {
  const CUtensorMap *map;
  int row0;  // row of the map that is input row 0
  const int32_t *qzeros;
  const __half *scales;
  int64_t words;  // out / 8
  int in;         // input rows
  int shift;      // log2 of the group size
  int col0, end0, col1, end1;
};

// First input row of box b of stage s of a range that starts at k0.  In mode
// kK a super-chunk of 256 rows is two stages, so that a group of 128 stays
// with one warp half.
template <Mode M>
__device__ __forceinline__ int box_row(int k0, int s, int b) {
  return M == Mode::kN ? k0 + s * 64
         : M == Mode::kK ? k0 + (s >> 1) * 256 + b * 128 + (s & 1) * 64
                         : k0 + s * 128 + b * 64;
}
template <Mode M>
__device__ __forceinline__ int num_stages(int rows) {  // rows a multiple of 64
  if (M == Mode::kN) return rows / 64;
  if (M == Mode::kTok) return (rows + 127) / 128;
  const int rem = rows % 256;
  return rows / 256 * 2 + (rem == 0 ? 0 : rem == 64 ? 1 : 2);
}

// ---------------------------------------------------------------- producer
// The words come by TMA, one instruction a box; token rows, steps and zero
// words by the lanes' 16-byte cp.async: bulk copies of a token row's 128 bytes
// held the copy engine up (16 rows: 1.3 us a stage).
template <Mode M, int MAXTOK>
struct Producer {
  static constexpr int kX = (MAXTOK + 3) / 4;  // token rows of a lane
  int n, shift, row0, x0, x1;                   // x0, x1: the boxes' columns in the words' tensor map
#ifdef AWQ_DEBUG_BOUNDS
  int in;
#endif
  const CUtensorMap *map;
  // this lane's chunk of either box's steps, and (lanes 0..7, 8..15) of their zero
  // words, in group 0; bytes between groups
  const char *sc[2], *zp;
  uint32_t sc_row, zp_row, zp_at;
  bool sc_ok[2], zp_ok, box1;
  const char *x[kX];  // 16-byte chunk lane % 8 of rows lane / 8 + 4 j

  __device__ __forceinline__ explicit Producer(const Weights &w) {
    const int lane = threadIdx.x & 31;
    map = w.map;
    row0 = w.row0;
    shift = w.shift;
#ifdef AWQ_DEBUG_BOUNDS
    in = w.in;
#endif
    x0 = w.col0 * 2;
    x1 = w.col1 * 2;
    box1 = w.col1 < w.end1;
    sc_row = (uint32_t)w.words * 16u;
    zp_row = (uint32_t)w.words * 4u;
    sc_ok[0] = w.col0 + lane < w.end0;
    sc_ok[1] = w.col1 + lane < w.end1;
    sc[0] = reinterpret_cast<const char *>(w.scales) + (sc_ok[0] ? (w.col0 + lane) * 16ll : 0ll);
    sc[1] = reinterpret_cast<const char *>(w.scales) + (sc_ok[1] ? (w.col1 + lane) * 16ll : 0ll);
    const int zc = (lane < 8 ? w.col0 : w.col1) + 4 * (lane & 7);
    zp_ok = zc < (lane < 8 ? w.end0 : w.end1);
    zp = reinterpret_cast<const char *>(w.qzeros) + (zp_ok ? zc * 4ll : 0ll);
    zp_at = sz_offset<M, MAXTOK>() + (lane < 8 ? 0u : 2 * kSz) + 512u + (lane & 7) * 16u;
  }

  template <class RowOf>
  __device__ __forceinline__ void rows(const __half *base, int64_t ld, int64_t rows, int count, RowOf row) {
    const int lane = threadIdx.x & 31;
    n = count;
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      const int t = (lane >> 3) + 4 * j;
      const int64_t r = t < n ? row(t) : 0;
      x[j] = reinterpret_cast<const char *>(base + (AWQ_IN_BOUNDS(r >= 0 && r < rows, 0xB090u) ? r * ld : 0) + (lane & 7) * 8);
    }
  }

  // Words, steps and zero words of stage s (and the stage's byte count).
  __device__ __forceinline__ void issue_words(uint32_t st, uint64_t *bar, int k0, int k1, int s) const {
    const int lane = threadIdx.x & 31;
    const int kb0 = box_row<M>(k0, s, 0), kb1 = box_row<M>(k0, s, 1);
    const bool ok1 = kb1 < k1 && box1;  // kb0 is in the range: a stage has its first box
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, ok1 ? 2 * kBoxBytes : kBoxBytes);
      tma_load_2d_at(st, map, bar, x0, row0 + kb0);
      if (ok1) tma_load_2d_at(st + kBoxBytes, map, bar, x1, row0 + kb1);
    }
    __syncwarp();
    const uint32_t d = st + sz_offset<M, MAXTOK>() + lane * 16;
    const bool first0 = shift != 7 || !(kb0 & 64), first1 = ok1 && (shift != 7 || !(kb1 & 64));
    // a group of 128 comes with its first box
    const uint32_t g0 = (uint32_t)kb0 >> shift, g1 = (uint32_t)kb1 >> shift;
    if (!AWQ_IN_BOUNDS(kb0 + kBoxK <= in && (!ok1 || kb1 + kBoxK <= in), 0xB091u)) return;
    if (first0) cp16(d, sc[0] + (uint64_t)g0 * sc_row, sc_ok[0]);
    if (first1) cp16(d + 2 * kSz, sc[1] + (uint64_t)g1 * sc_row, sc_ok[1]);
    if (lane < 16 && (lane < 8 ? first0 : first1)) cp16(st + zp_at, zp + (uint64_t)(lane < 8 ? g0 : g1) * zp_row, zp_ok);
    if (shift == 5) {  // and the second groups of 32
      cp16(d + kSz, sc[0] + (uint64_t)(g0 + 1) * sc_row, sc_ok[0]);
      if (ok1) cp16(d + 3 * kSz, sc[1] + (uint64_t)(g1 + 1) * sc_row, sc_ok[1]);
      if (lane < 16 && (lane < 8 || ok1))
        cp16(st + zp_at + kSz, zp + (uint64_t)((lane < 8 ? g0 : g1) + 1) * zp_row, zp_ok);
    }
  }

  // Token rows of stage s, and the lanes' arrivals.
  __device__ __forceinline__ void issue_rows(uint32_t st, uint64_t *bar, int k0, int k1, int s) const {
    const int lane = threadIdx.x & 31;
    const uint32_t d = st + x_offset() + (lane >> 3) * kXPitch + (lane & 7) * 16;
    const int kb0 = box_row<M>(k0, s, 0), kb1 = box_row<M>(k0, s, 1);
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      if ((lane >> 3) + 4 * j >= n) break;
      cp16(d + 4 * j * kXPitch, x[j] + 2 * kb0, true);
      if (M != Mode::kN && kb1 < k1) cp16(d + (MAXTOK + 4 * j) * kXPitch, x[j] + 2 * kb1, true);
    }
    cp_arrive(bar);
  }

  // Rows [k0, k1).  skip: stages whose words were issued ahead.  A wait that
  // runs out ends the ring's work on both sides (ring_wait); what follows then
  // computes on what there is, and the status says so.
  template <int STAGES>
  __device__ __forceinline__ void run(RingPos &pos, uint32_t ring, RingBars<STAGES> *bars, int k0, int k1,
                                      uint32_t max_polls, DevStatus *st, int skip = 0) const {
    const int ns = num_stages<M>(k1 - k0);
    for (int s = 0; s < ns; ++s) {
      const uint32_t at = ring + pos.slot * stage_bytes<M, MAXTOK>();
      if (s >= skip) {
        if (!ring_wait(bars, &bars->empty[pos.slot], pos.phase ^ 1u, max_polls, st, 0xE20u)) return;
        issue_words(at, &bars->full[pos.slot], k0, k1, s);
      }
      issue_rows(at, &bars->full[pos.slot], k0, k1, s);
      pos.next<STAGES>();
    }
  }
};

// ---------------------------------------------------------------- consumers
// Accumulators of one warp: 64 outputs x 8 NT tokens.  A group's zero points are
// subtracted from the codes (16 packed subtractions a step).  Taking off z sum_k x at the
// group's end instead costs one more MMA a step and is 2 to 4 % faster for one token tile
// with groups of 128 (10.1 against 9.7 us for 1 token), but gives NaN for every weight
// where x is infinite.
template <int NT>
struct Acc {
  float out[4][NT][4];  // totals: [p][token tile][c], 2^-24 (p even) or 2^-20 (p odd) of the sum
  float grp[4][NT][4];  // this group's sum, in the same units
  uint32_t zp[8];       // the group's zero points as subnormal pairs
  uint4 sc;             // the group's steps (8 fp16)
};

template <int NT>
__device__ __forceinline__ void acc_zero(Acc<NT> &a) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) a.out[p][n][c] = a.grp[p][n][c] = 0.0f;
}

template <int NT>
__device__ __forceinline__ void open_group(Acc<NT> &a, const uint8_t *sz, int wcol) {
  a.sc = *reinterpret_cast<const uint4 *>(sz + wcol * 16);
  const uint32_t zw = lds32(sz + 512 + wcol * 4);
  uint32_t lo = __byte_perm(zw, zw, 0x1010), hi = __byte_perm(zw, zw, 0x3232);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t m = (p & 1) ? 0x00F000F0u : 0x000F000Fu;
    if (p == 2) {
      lo >>= 8;
      hi >>= 8;
    }
    a.zp[p] = lo & m;
    a.zp[p + 4] = hi & m;
  }
}

// Closes a group: out += s (sum (q - z) x), then clears the group's sums.
template <int NT>
__device__ __forceinline__ void close_group(Acc<NT> &a) {
  const uint32_t sh[4] = {a.sc.x, a.sc.y, a.sc.z, a.sc.w};
#pragma unroll
  for (int o = 0; o < 8; ++o) {
    const __half2 s2 = *reinterpret_cast<const __half2 *>(&sh[o >> 1]);
    const float s = __half2float((o & 1) ? __high2half(s2) : __low2half(s2));
    const int p = o & 3, h = o >> 2;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 2 * h; c < 2 * h + 2; ++c) {
        a.out[p][n][c] = fmaf(s, a.grp[p][n][c], a.out[p][n][c]);
        a.grp[p][n][c] = 0.0f;
      }
  }
}

// Words and token fragments of two 16-row steps: the one at work and the next.
template <int NT>
struct Frags {
  static constexpr int kB = (NT + 1) / 2;
  uint32_t w[2][4], b[2][kB][4];
};

// The words (this lane's rows 2q, 2q + 1, 2q + 8, 2q + 9) and token fragments of step
// ks of a box; w0 / w1: the word addresses of rows 2q and 2q + 1; xa: the ldmatrix
// address.  One token tile takes the fragments of two steps at once.
template <int NT>
__device__ __forceinline__ void load_step(Frags<NT> &f, const uint8_t *w0, const uint8_t *w1, uint32_t xa, int ks) {
  uint32_t(&d)[4] = f.w[ks & 1];
  d[0] = lds32(w0 + ks * 2048);
  d[1] = lds32(w1 + ks * 2048);
  d[2] = lds32(w0 + ks * 2048 + 1024);
  d[3] = lds32(w1 + ks * 2048 + 1024);
  if (NT == 1) {
    if (!(ks & 1)) ldsm4(f.b[ks >> 1][0], xa + (ks >> 1) * 64);
  } else {
#pragma unroll
    for (int n = 0; n < Frags<NT>::kB; ++n) ldsm4(f.b[ks & 1][n], xa + n * 16 * kXPitch + ks * 32);
  }
}

// One box: four 16-row steps, each step's words and fragments loaded one step
// ahead.  Its first step is loaded already; next() loads the first step of the box
// that follows, while this one's last step is at work.
template <int NT, int SHIFT, class Next>
__device__ __forceinline__ void box(Acc<NT> &a, Frags<NT> &f, const uint8_t *w0, const uint8_t *w1, uint32_t xa,
                                    const uint8_t *sz, int wcol, bool upper, Next next) {
  if (!(SHIFT == 7 && upper)) open_group<NT>(a, sz, wcol);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const uint32_t(&c)[4] = f.w[ks & 1];
    uint32_t v[4] = {__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[0], c[1], 0x7632),
                     __byte_perm(c[2], c[3], 0x5410), __byte_perm(c[2], c[3], 0x7632)};
    if (ks < 3)
      load_step<NT>(f, w0, w1, xa, ks + 1);
    else
      next();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t m = (p & 1) ? 0x00F000F0u : 0x000F000Fu;
      if (p == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] >>= 8;
      }
      const uint32_t a0 = sub2(v[0] & m, a.zp[p]), a1 = sub2(v[1] & m, a.zp[p + 4]);
      const uint32_t a2 = sub2(v[2] & m, a.zp[p]), a3 = sub2(v[3] & m, a.zp[p + 4]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t b0 = NT == 1 ? f.b[ks >> 1][0][2 * (ks & 1)] : f.b[ks & 1][n / 2][2 * (n & 1)];
        const uint32_t b1 = NT == 1 ? f.b[ks >> 1][0][2 * (ks & 1) + 1] : f.b[ks & 1][n / 2][2 * (n & 1) + 1];
        mma16816(a.grp[p][n], a0, a1, a2, a3, b0, b1);
      }
    }
    if (ks == 1 && SHIFT == 5) {
      close_group<NT>(a);
      open_group<NT>(a, sz + kSz, wcol);
    }
  }
  if (SHIFT != 7 || upper) close_group<NT>(a);
}

// The consumers' side of a product over rows [k0, k1) (multiples of 64; of 128
// when g = 128).
template <Mode M, int NT, int MAXTOK, int STAGES, int SHIFT>
__device__ __forceinline__ void consume(Acc<NT> &a, RingPos &pos, uint8_t *ring, RingBars<STAGES> *bars, int k0, int k1,
                                        bool box1, uint32_t max_polls, DevStatus *st) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = warp & 3, half = warp >> 2, g = lane >> 2, q = lane & 3;
  const int wcol = nw * 8 + g, chunk = wcol >> 2;
  const uint32_t o0 = (2 * q) * 128 + ((uint32_t)(chunk ^ (2 * q)) << 4) + (wcol & 3) * 4;
  const uint32_t o1 = (2 * q + 1) * 128 + ((uint32_t)(chunk ^ (2 * q + 1)) << 4) + (wcol & 3) * 4;
  // ldmatrix: for one token tile the four 8-column blocks of 32 input rows, else
  // (token tile, 8-column block) pairs of 16 input rows
  const uint32_t xl = NT == 1 ? (lane & 7) * kXPitch + (lane >> 3) * 16
                              : ((lane >> 4) * 8 + (lane & 7)) * kXPitch + ((lane >> 3) & 1) * 16;
  const uint32_t xt = M == Mode::kTok ? half * NT * 8 * kXPitch : 0;
  acc_zero<NT>(a);
  // This warp's boxes; in modes kN and kK one of each stage, but for the last stages
  // of a range that end before its half.
  const int ns = num_stages<M>(k1 - k0), rows = k1 - k0, rem = rows % 256;
  const int boxes = M == Mode::kN     ? (half == 0 || box1 ? ns : 0)
                    : M == Mode::kTok ? rows / 64
                    : half == 0       ? rows / 256 * 2 + min(rem / 64, 2)
                                      : rows / 256 * 2 + (rem == 192);
  Frags<NT> f;
  const uint32_t w_at = M == Mode::kTok ? 0 : half * kBoxBytes;
  const uint32_t x_at = x_offset() + (M == Mode::kK ? half * MAXTOK * kXPitch : 0) + xl + xt;
  const uint32_t sz_at = sz_offset<M, MAXTOK>() + (M == Mode::kTok ? 0 : half * 2 * kSz);
  const auto load = [&](int b, int ks) {
    const uint8_t *sp = ring + pos.slot * stage_bytes<M, MAXTOK>();
    load_step<NT>(f, sp + w_at + b * kBoxBytes + o0, sp + w_at + b * kBoxBytes + o1,
                  smem_u32(sp) + x_at + b * MAXTOK * kXPitch, ks);
  };
  bool ready = false, ok = true;
  // A group of 128 is two boxes, one after the other (their count is even)
  constexpr int kUnroll = SHIFT == 5 || NT == 4 ? 1 : 2;
#pragma unroll kUnroll
  for (int i = 0; i < boxes; ++i) {
    const int b = M == Mode::kTok ? i & 1 : 0;  // box of the stage
    // The first step was loaded while the box before was at work, and counts if the
    // stage had landed.  There is no branch but this one: instructions of two boxes
    // do not overlap across branches
    if (!__all_sync(0xffffffffu, ready)) {
      ok = ring_wait(bars, &bars->full[pos.slot], pos.phase, max_polls, st, 0xE21u);
      if (!ok) break;
      load(b, 0);
    }
    const bool leaves = M != Mode::kTok || b == 1 || i == boxes - 1;
    RingPos nx = pos;
    nx.next<STAGES>();
    ready = !leaves || mbar_test(&bars->full[nx.slot], nx.phase);
    const uint8_t *sp = ring + pos.slot * stage_bytes<M, MAXTOK>();
    box<NT, SHIFT>(a, f, sp + w_at + b * kBoxBytes + o0, sp + w_at + b * kBoxBytes + o1,
                   smem_u32(sp) + x_at + b * MAXTOK * kXPitch, sp + sz_at + b * 2 * kSz, wcol, (i & 1) != 0, [&] {
                     __syncwarp();  // every load from the box has been issued
                     if (leaves && lane == 0) mbar_arrive(&bars->empty[pos.slot]);
                     if (leaves) pos = nx;
                     load(M == Mode::kTok && !leaves ? 1 : 0, 0);
                   });
  }
  for (int s = M == Mode::kTok ? ns : boxes; ok && s < ns; ++s) {
    ok = ring_wait(bars, &bars->full[pos.slot], pos.phase, max_polls, st, 0xE21u);
    if (ok && lane == 0) mbar_arrive(&bars->empty[pos.slot]);
    pos.next<STAGES>();
  }
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) a.out[p][n][c] *= (p & 1) ? 1048576.0f : 16777216.0f;
}

// A lane's 8 consecutive outputs of token column 8 n + 2 q + e.
template <int NT>
__device__ __forceinline__ void outputs8(const Acc<NT> &a, int n, int e, float (&v)[8]) {
#pragma unroll
  for (int o = 0; o < 8; ++o) v[o] = a.out[o & 3][n][e + 2 * (o >> 2)];
}

// The block's sums of a 256-output tile into shared memory, red[token][kRedPitch];
// the consumers may read them after the barrier at the end.
constexpr int kRedPitch = kBoxN + 1;
template <Mode M, int NT>
__device__ __forceinline__ void store_sums(const Acc<NT> &a, float *red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = warp & 3, half = warp >> 2, g = lane >> 2, q = lane & 3;
  const int t0 = M == Mode::kTok ? half * NT * 8 : 0;
  float *d0 = red + (t0 + 2 * q) * kRedPitch + (nw * 8 + g) * 8;
  auto each = [&](bool add) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float *d = d0 + (n * 8 + (c & 1)) * kRedPitch + p + 4 * (c >> 1);
          *d = add ? *d + a.out[p][n][c] : a.out[p][n][c];
        }
  };
  if (M != Mode::kK) {
    each(false);
  } else {  // the two K halves, in a fixed order
    if (half == 0) each(false);
    consumer_sync();
    if (half == 1) each(true);
  }
  consumer_sync();
}

}  // namespace w4s
}  // namespace awq
