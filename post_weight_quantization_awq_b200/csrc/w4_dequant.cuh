// Dequantising packed 4-bit words to fp16 weights RN16((q - z) scale): shared by
// the W4A16 product (w4a16_gemm.cu) and the adapter product for many tokens
// (lora_prefill.cu).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "awq_device.cuh"

namespace awq {
namespace {

// fp16 pairs {1024 + nibble p, 1024 + nibble p + 4}, p = 0..3, of a word
__device__ __forceinline__ void nib_pairs(uint32_t w, __half2 (&h)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t bits = ((w >> (4 * p)) & 0x000F000Fu) | 0x64006400u;
    h[p] = *reinterpret_cast<const __half2 *>(&bits);
  }
}

// scales of outputs (p, p + 4), p = 0..3, from 8 consecutive fp16 scales
__device__ __forceinline__ void scale_pairs(uint4 sc, __half2 (&h)[4]) {
  const uint32_t lo[2] = {sc.x, sc.y}, hi[2] = {sc.z, sc.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    // half p of the first four, half p of the last four
    const uint32_t a = lo[p >> 1], b = hi[p >> 1];
    const uint32_t bits = __byte_perm(a, b, (p & 1) ? 0x7632u : 0x5410u);
    h[p] = *reinterpret_cast<const __half2 *>(&bits);
  }
}

// 8 weights RN16((q - z) * scale) of one word in the order 0,4,1,5,2,6,3,7;
// (1024 + q) - (1024 + z) is exact
__device__ __forceinline__ uint4 dequant_word(uint32_t w, const __half2 (&zp)[4], const __half2 (&sp)[4]) {
  __half2 qp[4];
  nib_pairs(w, qp);
  uint32_t o[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const __half2 r = __hmul2(__hsub2(qp[p], zp[p]), sp[p]);
    o[p] = *reinterpret_cast<const uint32_t *>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A tile of kDeqIn inputs x kDeqOut outputs, as a block of 256 threads turns it
// from packed words (input-major) into output-major rows of Wd [out, in] through
// shared memory, so both the word loads and the 16-byte row stores are
// contiguous.
constexpr int kDeqIn = 128, kDeqOut = 64;

__device__ __forceinline__ void dequant_tile(__half *tile, const int32_t *__restrict__ qweight,
                                             const int32_t *__restrict__ qzeros, const __half *__restrict__ scales,
                                             int64_t in, int64_t out, int group, int64_t o0, int64_t j0,
                                             __half *__restrict__ Wd) {
  constexpr int TJ = kDeqIn, TO = kDeqOut, WPR = TO / 8;  // inputs, outputs, words per input row
  // [output][input] with the 16-byte chunks of row r XOR-swizzled by r / 8, so
  // that the 2-byte writes of one warp (8 word columns, i.e. rows 8 apart)
  // fall in different banks and the 16-byte row reads stay aligned
  const int64_t words = out / 8;
  // a thread converts the words of two consecutive input rows of one word
  // column (one group: group % 32 == 0) and writes each output's two weights
  // as one half2
#pragma unroll
  for (int i = 0; i < TJ * WPR / 512; ++i) {
    const int w = threadIdx.x + 256 * i;
    const int jp = w / WPR, ow = w % WPR;  // input row pair of the tile, word column
    const int jj = 2 * jp;
    const int64_t j = j0 + jj, wc = o0 / 8 + ow;
    uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
    if (j < in && wc < words) {  // in % 64 == 0: rows j and j + 1 are both in
      const int64_t gi = j / group;
      __half2 zp[4], sp[4];
      nib_pairs((uint32_t)__ldg(qzeros + gi * words + wc), zp);
      scale_pairs(__ldg(reinterpret_cast<const uint4 *>(scales + gi * out + 8 * wc)), sp);
      const int32_t *qp = qweight + j * words + wc;
      v0 = dequant_word((uint32_t)__ldg(qp), zp, sp);
      v1 = dequant_word((uint32_t)__ldg(qp + words), zp, sp);
    }
    // v0 / v1 hold outputs 0,4,1,5,2,6,3,7 of the word in rows jj / jj + 1
    const uint32_t h0[4] = {v0.x, v0.y, v0.z, v0.w}, h1[4] = {v1.x, v1.y, v1.z, v1.w};
    const int col = (((jj >> 3) ^ ow) << 3) | (jj & 7);  // rows 8 ow .. 8 ow + 7 share the swizzle
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      // output p: low halves of row jj and row jj + 1; output p + 4: the high halves
      const uint32_t lo = __byte_perm(h0[p], h1[p], 0x5410u), hi = __byte_perm(h0[p], h1[p], 0x7632u);
      *reinterpret_cast<uint32_t *>(tile + (8 * ow + p) * TJ + col) = lo;
      *reinterpret_cast<uint32_t *>(tile + (8 * ow + p + 4) * TJ + col) = hi;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TO * (TJ / 8) / 256; ++i) {
    const int c = threadIdx.x + 256 * i;
    const int oo = c / (TJ / 8), jc = c % (TJ / 8);  // output row, 8-input chunk
    const int64_t o = o0 + oo, j = j0 + 8 * jc;
    if (o < out && j < in)  // in % 64 == 0: a chunk is whole
      *reinterpret_cast<uint4 *>(Wd + o * in + j) =
          *reinterpret_cast<const uint4 *>(tile + oo * TJ + 8 * (jc ^ (oo >> 3)));
  }
}

// The same weights with 256-output tiles of 64 inputs (the adapter product's; w4a16_gemm.cu's
// dequantise-once form has the tiles above): 128 bytes of a row of words and of a
// row of weights at a time, which HBM reads and writes faster than 32 bytes.  The
// 16-byte chunks of an output's 64 weights are XOR-swizzled by its word column, and
// the 4-byte pairs inside a chunk by the column's upper bits, so that a warp's
// writes (32 word columns, one input pair) fall in different banks.  Loads pass by L1: the
// kernel may start before the one that precedes it has ended (serve_launch.h).
constexpr int kWideIn = 64, kWideOut = 256;

__device__ __forceinline__ void dequant_wide(__half *tile, const int32_t *__restrict__ qweight,
                                             const int32_t *__restrict__ qzeros, const __half *__restrict__ scales,
                                             int64_t in, int64_t out, int group, int64_t o0, int64_t j0,
                                             __half *__restrict__ Wd) {
  const int64_t words = out / 8;
  const int ow = threadIdx.x & 31, jw = threadIdx.x >> 5;  // word column; inputs 8 jw .. 8 jw + 7 (one group)
  const int64_t wc = o0 / 8 + ow, j = j0 + 8 * jw;
  uint32_t wv[8];
  __half2 zp[4], sp[4];
  const bool ok = wc < words && j < in && AWQ_IN_BOUNDS(j + 8 <= in, 0xB0C1u);  // in % 64 == 0
  if (ok) {
    const int64_t gi = j / group;
#pragma unroll
    for (int r = 0; r < 8; ++r) wv[r] = (uint32_t)__ldcg(qweight + (j + r) * words + wc);
    nib_pairs((uint32_t)__ldcg(qzeros + gi * words + wc), zp);
    scale_pairs(__ldcg(reinterpret_cast<const uint4 *>(scales + gi * out + 8 * wc)), sp);
    uint32_t *t = reinterpret_cast<uint32_t *>(tile) + 8 * ow * (kWideIn / 2) + ((jw ^ (ow & 7)) << 2);
#pragma unroll
    for (int r = 0; r < 8; r += 2) {
      const uint4 v0 = dequant_word(wv[r], zp, sp), v1 = dequant_word(wv[r + 1], zp, sp);
      const uint32_t h0[4] = {v0.x, v0.y, v0.z, v0.w}, h1[4] = {v1.x, v1.y, v1.z, v1.w};
      const int at = (r >> 1) ^ (ow >> 3);
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // output p: low halves of the two rows; p + 4: the high halves
        t[p * (kWideIn / 2) + at] = __byte_perm(h0[p], h1[p], 0x5410u);
        t[(p + 4) * (kWideIn / 2) + at] = __byte_perm(h0[p], h1[p], 0x7632u);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWideOut * (kWideIn / 8) / 256; ++i) {
    const int c = threadIdx.x + 256 * i, oo = c >> 3, jc = c & 7;  // output, 8-input chunk
    const int64_t o = o0 + oo, jj = j0 + 8 * jc;
    if (o >= out || jj >= in || !AWQ_IN_BOUNDS(jj + 8 <= in, 0xB0C0u)) continue;
    const uint4 v = *reinterpret_cast<const uint4 *>(tile + oo * kWideIn + 8 * (jc ^ ((oo >> 3) & 7)));
    const int x = oo >> 6;  // undo the pairs' swizzle: pair i lies at i ^ x
    const uint32_t a = (x & 1) ? v.y : v.x, b = (x & 1) ? v.x : v.y, e = (x & 1) ? v.w : v.z, f = (x & 1) ? v.z : v.w;
    *reinterpret_cast<uint4 *>(Wd + o * in + jj) = (x & 2) ? make_uint4(e, f, a, b) : make_uint4(a, b, e, f);
  }
}

}  // namespace
}  // namespace awq
