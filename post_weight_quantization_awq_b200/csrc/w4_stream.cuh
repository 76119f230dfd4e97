// Streaming product of a few fp16 token rows with packed 4-bit weights on the
// warp-level tensor-core instruction: the core of the adapter product for few
// tokens (lora_gemm.cu) and of the mixture-of-experts layer (moe_layer.cu).
//
//   S[t][o] = sum over k in [k0, k1) of x[t][k] (q - z)[k][o] s[k/g][o]
//
// Mathematics.  Within a group the step is common, so
//   S = sum_groups s (sum_k q x - z sum_k x):
// the codes themselves are the A operand.  A nibble at bit 0 (bit 4) of a
// 16-bit half, read as fp16, is the subnormal q 2^-24 (q 2^-20), exactly, so
// a code needs one AND and no conversion; sum_k x comes from one more MMA
// whose A operand is 2^-24 everywhere.  Products are exact in fp32, the group
// sums and their scaled total are fp32, and no weight is rounded to fp16.
//
// Layout.  m16n8k16: 16 rows = 8 word columns x 2 nibbles (p, p + 4), 16
// k = 4 consecutive input rows for each of the 4 lanes of a quad, 8 columns =
// 8 tokens.  Lane (g, q) holds word column g and input rows 4q..4q+3 of a
// 16-row step: four words give, after one byte permute per pair and mask, the
// A fragments of four MMAs (p = 0..3), 64 outputs per warp.  The order of k
// inside a step is free as long as A and B agree; 4q..4q+3 makes the B
// fragment of a token one 64-bit shared load.
//
// A block of 8 warps covers 256 outputs (4 warps) and either two K halves or
// two token halves (2 warps); a stage of the cp.async ring is 2 pieces of 64
// input rows x 128 bytes of words, the same rows of X, and the groups' steps
// and zero words.  The words' 16-byte chunks are XOR-swizzled by the row so
// that the four rows a quad reads fall in different banks.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "awq_device.cuh"

namespace awq {
namespace w4s {

constexpr int kThreads = 256;
constexpr int kTileN = 256;                    // outputs per block
constexpr int kPiece = 64;                     // input rows per piece
constexpr uint32_t kPieceW = kPiece * 128;     // bytes of words of a piece
constexpr uint32_t kSz = 640;                  // 256 steps (fp16) + 32 zero words
constexpr uint32_t kXPitch = kPiece * 2 + 32;  // bytes between token rows of a piece

__host__ __device__ constexpr uint32_t stage_bytes(int max_tok) {
  return 2 * kPieceW + 2 * (uint32_t)max_tok * kXPitch + 4 * kSz;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t n) {  // n = 0: zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ int group_shift(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint2 lds64(const uint8_t *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ uint4 lds128(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// One packed matrix [in, out]: two column bases in words (the tile's first and
// second 128 outputs) and the first word past each half's columns.
struct Weights {
  const int32_t *qweight, *qzeros;
  const __half *scales;
  int64_t words;  // out / 8
  int group_shift;  // log2 of the group size
  int64_t col0, end0, col1, end1;
};

// Tokens of a product: row t is base + row(t) * ld.
struct Rows {
  const __half *base;
  int64_t ld;
  const int *index;  // shared memory, or NULL: row t itself
  int n;
};

// How the block's second warp axis is used.
enum class Split { kK, kTok };

// First input row of piece p of stage s of a range that starts at k0.  With
// the K split a super-chunk of 256 rows is two stages: warp half p takes rows
// 128 p .. 128 p + 127 of it, 64 in each stage, so that a group of 128 stays
// with one warp.
template <Split SP>
__device__ __forceinline__ int piece_row(int k0, int s, int p) {
  return SP == Split::kK ? k0 + (s >> 1) * 256 + p * 128 + (s & 1) * 64 : k0 + s * 128 + p * 64;
}
template <Split SP>
__device__ __forceinline__ int num_stages(int rows) {  // rows a multiple of 64
  if (SP == Split::kTok) return (rows + 127) / 128;
  const int rem = rows % 256;
  return rows / 256 * 2 + (rem == 0 ? 0 : rem == 64 ? 1 : 2);
}

// This thread's copies of a stage, their addresses worked out once per product:
// rows r and r + 32 of one 16-byte word chunk of both pieces, up to NX chunks
// of X, and one chunk of the groups' steps or zero words.
template <Split SP, int MAXTOK>
struct Loader {
  static constexpr int NX = (16 * MAXTOK + kThreads - 1) / kThreads;
  const char *w;   // row r of the matrix
  int64_t wrow;    // bytes of a row of words
  uint32_t wdst, wn;
  const char *x[NX];  // NULL: nothing to copy
  const char *sz;     // group 0's chunk
  int64_t szrow;
  uint32_t szdst, szn;
  int role, shift;  // role: -1, or piece * 2 + group of the piece

  __device__ __forceinline__ void init(const Weights &m, const Rows &rows) {
    const int tid = threadIdx.x;
    shift = m.group_shift;
    {
      const int r = tid >> 3, c = tid & 7;
      const int64_t col = (c < 4 ? m.col0 : m.col1) + 4 * (c & 3);
      const bool ok = col < (c < 4 ? m.end0 : m.end1);
      wrow = m.words * 4;
      w = reinterpret_cast<const char *>(m.qweight + (ok ? col : 0)) + r * wrow;
      wdst = r * 128 + ((uint32_t)(c ^ (((r >> 2) & 3) << 1)) << 4);
      wn = ok ? 16u : 0u;  // 0: the chunk is zero-filled, nothing is read
    }
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const int i = tid + j * kThreads, c = i & 7, pt = i >> 3, t = pt % MAXTOK;
      x[j] = nullptr;
      if (pt < 2 * MAXTOK && t < rows.n) {
        const int64_t row = rows.index ? rows.index[t] : t;
        x[j] = reinterpret_cast<const char *>(rows.base + row * rows.ld + c * 8);
      }
    }
    role = tid / 40;  // a piece has one group, two when g = 32
    const int e = tid - role * 40;
    if (role >= 4 || (shift != 5 && (role & 1))) {
      role = -1;
      return;
    }
    const int ch = e < 32 ? e >> 2 : e - 32;  // the 16-byte word chunk it belongs to
    const int64_t col = (ch < 4 ? m.col0 : m.col1) + 4 * (ch & 3) + (e < 32 ? e & 3 : 0);
    const bool ok = col < (ch < 4 ? m.end0 : m.end1);
    szrow = e < 32 ? m.words * 16 : m.words * 4;
    sz = e < 32 ? reinterpret_cast<const char *>(m.scales + (ok ? col : 0) * 8)
                : reinterpret_cast<const char *>(m.qzeros + (ok ? col : 0));
    szdst = 2 * kPieceW + 2 * MAXTOK * kXPitch + role * kSz + (e < 32 ? e * 16 : 512 + (e - 32) * 16);
    szn = ok ? 16u : 0u;
  }

  // Copies of stage s of the range [k0, k1) into shared memory at `st` (not
  // committed).  A piece outside the range is skipped: nobody reads it.
  __device__ __forceinline__ void issue(uint32_t st, int k0, int k1, int s) const {
    const int tid = threadIdx.x;
    const int kb0 = piece_row<SP>(k0, s, 0), kb1 = piece_row<SP>(k0, s, 1);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int kb = p ? kb1 : kb0;
      if (kb >= k1) continue;
      const char *src = w + (int64_t)kb * wrow;
      cp16(st + p * kPieceW + wdst, src, wn);
      cp16(st + p * kPieceW + wdst + 32 * 128, src + 32 * wrow, wn);  // row r + 32: the same swizzle
    }
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const int i = tid + j * kThreads, pt = i >> 3;
      const int kb = pt < MAXTOK ? kb0 : kb1;
      if (x[j] && kb < k1) cp16(st + 2 * kPieceW + pt * kXPitch + (i & 7) * 16, x[j] + 2 * kb, 16u);
    }
    if (role >= 0) {
      const int kb = (role & 2) ? kb1 : kb0;
      // a group of 128 is closed by its second piece, which alone brings it
      if (kb < k1 && (shift != 7 || (kb & 64)))
        cp16(st + szdst, sz + (int64_t)((kb + 32 * (role & 1)) >> shift) * szrow, szn);
    }
  }
};

// Accumulators of one warp: 64 outputs x 8 NT tokens.
template <int NT>
struct Acc {
  float out[4][NT][4];  // scaled totals: [p][token tile][c]
  float grp[4][NT][4];  // this group's sum of q x 2^-24 (p even), 2^-20 (p odd)
  float sx[NT][4];      // this group's sum of x 2^-24
};

template <int NT>
__device__ __forceinline__ void acc_zero(Acc<NT> &a) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) a.out[p][n][c] = a.grp[p][n][c] = 0.0f;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) a.sx[n][c] = 0.0f;
}

// Closes a group: out += s (sum q x - z sum x), then clears the group's sums.
template <int NT>
__device__ __forceinline__ void flush_group(Acc<NT> &a, const uint8_t *sz, int wcol) {
  const uint4 sv = lds128(sz + wcol * 16);
  const uint32_t zw = lds32(sz + 512 + wcol * 4);
  const uint32_t sh[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // output p (rows g), output p + 4 (rows g + 8)
      const int o = p + 4 * h;
      const __half2 s2 = *reinterpret_cast<const __half2 *>(&sh[o >> 1]);
      const float s = __half2float((o & 1) ? __high2half(s2) : __low2half(s2));
      const float sq = s * ((p & 1) ? 1048576.0f : 16777216.0f);                         // 2^20 or 2^24
      const float szx = -s * 16777216.0f * (float)((zw >> (4 * o)) & 15u);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * h + e;
          a.out[p][n][c] = fmaf(sq, a.grp[p][n][c], fmaf(szx, a.sx[n][e], a.out[p][n][c]));
          a.grp[p][n][c] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) a.sx[n][c] = 0.0f;
}

// One 64-row piece: four 16-row steps.  `wb` / `xb`: this lane's word and X
// addresses in the piece.
template <int NT>
__device__ __forceinline__ void piece(Acc<NT> &a, const uint8_t *wb, const uint8_t *xb, const uint8_t *sz,
                                      int wcol, int shift, bool close128) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lds32(wb + (ks * 16 + i) * 128);
    uint2 b[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) b[n] = lds64(xb + n * 8 * kXPitch + ks * 32);
    uint32_t v[4] = {__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                     __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632)};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t m = (p & 1) ? 0x00F000F0u : 0x000F000Fu;
      if (p == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] >>= 8;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma16816(a.grp[p][n], v[0] & m, v[1] & m, v[2] & m, v[3] & m, b[n].x, b[n].y);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      mma16816(a.sx[n], 0x00010001u, 0x00010001u, 0x00010001u, 0x00010001u, b[n].x, b[n].y);
    if (shift == 5 && (ks & 1)) flush_group<NT>(a, sz + (ks >> 1) * kSz, wcol);
  }
  if (shift == 6 || (shift == 7 && close128)) flush_group<NT>(a, sz, wcol);
}

// The product of the block over rows [k0, k1) of its tile (k0 and k1
// multiples of 64; of 128 when g = 128).  Uses the ring at `ring` (STAGES x
// stage_bytes(MAXTOK)), which is free again on return for every thread.
template <int NT, Split SP, int MAXTOK, int STAGES>
__device__ __forceinline__ void product(Acc<NT> &a, uint8_t *ring, const Weights &w, const Rows &x, int k0,
                                        int k1) {
  constexpr uint32_t kStage = stage_bytes(MAXTOK);
  const uint32_t ring_u = smem_u32(ring);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = warp & 3, half = warp >> 2, g = lane >> 2, q = lane & 3;
  const int wcol = nw * 8 + g;
  const int ns = num_stages<SP>(k1 - k0);
  Loader<SP, MAXTOK> ld;
  ld.init(w, x);
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (s < ns) ld.issue(ring_u + s * kStage, k0, k1, s);
    cp_commit();
  }
  acc_zero<NT>(a);
  const uint32_t wlane = (uint32_t)(4 * q) * 128 + ((uint32_t)((wcol >> 2) ^ (q << 1)) << 4) + (wcol & 3) * 4;
  const uint32_t xlane = (uint32_t)g * kXPitch + q * 8 + (SP == Split::kTok ? half * NT * 8 * kXPitch : 0);
  uint32_t slot = 0, next = (STAGES - 1) * kStage;
  for (int s = 0; s < ns; ++s) {
    cp_wait<STAGES - 2>();
    __syncthreads();  // stage s has landed for all, and the slot of s - 1 is free
    if (s + STAGES - 1 < ns) ld.issue(ring_u + next, k0, k1, s + STAGES - 1);
    cp_commit();
    const uint8_t *st = ring + slot;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (SP == Split::kK && p != half) continue;
      const int kb = piece_row<SP>(k0, s, p);
      if (kb < k1)
        piece<NT>(a, st + p * kPieceW + wlane, st + 2 * kPieceW + p * MAXTOK * kXPitch + xlane,
                  st + 2 * kPieceW + 2 * MAXTOK * kXPitch + p * 2 * kSz, wcol, w.group_shift, (kb & 64) != 0);
    }
    next = slot;
    slot = slot + kStage == STAGES * kStage ? 0 : slot + kStage;
  }
  cp_wait<0>();
  __syncthreads();
}

// The block's sums into shared memory, red[token][kRedPitch]: output o of the
// tile at column o.  Every thread may read them on return.
constexpr int kRedPitch = 257;
template <int NT, Split SP>
__device__ __forceinline__ void store_sums(const Acc<NT> &a, float *red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = warp & 3, half = warp >> 2, g = lane >> 2, q = lane & 3;
  const int t0 = SP == Split::kTok ? half * NT * 8 : 0;
  auto each = [&](bool add) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float *d = red + (t0 + n * 8 + 2 * q + (c & 1)) * kRedPitch + (nw * 8 + g) * 8 + p + 4 * (c >> 1);
          *d = add ? *d + a.out[p][n][c] : a.out[p][n][c];
        }
  };
  if (SP == Split::kTok) {
    each(false);
  } else {  // the two K halves, in a fixed order
    if (half == 0) each(false);
    __syncthreads();
    if (half == 1) each(true);
  }
  __syncthreads();
}

}  // namespace w4s
}  // namespace awq
