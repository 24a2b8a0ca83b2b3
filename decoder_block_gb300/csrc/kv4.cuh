// Rows of keys and values held in 4 bits, a scale for 16 of them (llama_ops.h describes
// the blocks): sizes, reading and writing.
//
// The scale's byte is the top of an fp32 or bf16 number -- three bits of mantissa under
// an exponent that starts at -20 -- so that it turns into one with an add and a shift,
// reaches from 2^-20 to 3840 without a factor per tensor, and a code times it has seven
// significant bits: bf16 holds every value exactly.  Equal steps lose less of such blocks than
// fp4's do (normal values: an error of 0.0929 of their RMS, for 0.0942 with a scale that is exactly
// a sixth of the largest and 0.1004 with one of these).  The smallest scale that reaches the
// largest value is found without trying: the best of it and the next four smaller ones, which cut
// the largest off, would lose 0.0828.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "paged.cuh"

namespace llama {

constexpr int KV4_BLOCK = 16;                  // elements of a scale
constexpr int KV4_SCALE_BASE = (127 - 20) << 3;  // a scale byte plus this: sign, exponent and three bits of an fp32
constexpr float KV4_LEVELS = 7.0f;             // codes stored are 8 - 7 .. 8 + 7
constexpr float KV4_MOST = 7.0f * 3840.0f;

__host__ __device__ constexpr int kv4_code_bytes(int D) { return D / 2; }
__host__ __device__ constexpr int kv4_scale_bytes(int D) { return D / KV4_BLOCK; }
__host__ __device__ constexpr int kv4_block_bytes(int page_size, int D) {
  return page_size * (kv4_code_bytes(D) + kv4_scale_bytes(D));
}

// Where a row of a page lies.
struct Kv4Row {
  const uint8_t *codes = nullptr;  // null: zeros
  const uint8_t *scales = nullptr;
  __device__ __forceinline__ bool operator!=(decltype(nullptr)) const { return codes != nullptr; }
};
__device__ __forceinline__ long long kv4_block_at(const PagedView &pv, int page, int g, int D) {
  return page * pv.page_stride + (long long)g * kv4_block_bytes(1 << pv.page_log2, D);
}
__device__ __forceinline__ Kv4Row kv4_row(const uint8_t *pool, const PagedView &pv, int page, int g, int D, int slot) {
  Kv4Row r;
  const uint8_t *block = pool + kv4_block_at(pv, page, g, D);
  r.codes = block + slot * kv4_code_bytes(D);
  r.scales = block + (kv4_code_bytes(D) << pv.page_log2) + slot * kv4_scale_bytes(D);
  return r;
}

__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __uint_as_float((byte + KV4_SCALE_BASE) << 20); }
// The scale twice, as bf16, from two bytes (low half: `a`).
__device__ __forceinline__ uint32_t kv4_scale2(uint32_t a, uint32_t b) {
  return ((a + KV4_SCALE_BASE) << 4) | ((b + KV4_SCALE_BASE) << 20);
}

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// (x & mask) | set in one instruction (the compiler makes two of it, for it has room for one
// constant in each).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t set) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "r"(mask), "r"(set));
  return d;
}
// A code n in the mantissa of 16.0 or 128.0 reads as 16 + n (bits 3 to 6 of a bf16) or 128 + n
// (bits 0 to 3); times s and less 24 s or 136 s, in one rounding that has nothing to round,
// it is (n - 8) s.  (24 s and 136 s are bf16 too: s is 8 to 15 times a power of two, and
// 17 * 15 = 255.)  The codes in the lowest bits need no shift.
struct Kv4Scale {
  uint32_t s, b24, b136;
};
// From a byte for each half.
__device__ __forceinline__ Kv4Scale kv4_scales(uint32_t lo, uint32_t hi) {
  Kv4Scale r;
  r.s = kv4_scale2(lo, hi);
  r.b24 = bf16x2_mul(r.s, 0xc1c0c1c0u);
  r.b136 = bf16x2_mul(r.s, 0xc308c308u);
  return r;
}
// A byte for both.
__device__ __forceinline__ Kv4Scale kv4_scales(uint32_t byte) {
  Kv4Scale r;
  r.s = byte * 0x00100010u + KV4_SCALE_BASE * 0x00100010u;
  r.b24 = bf16x2_mul(r.s, 0xc1c0c1c0u);
  r.b136 = bf16x2_mul(r.s, 0xc308c308u);
  return r;
}
// Codes in bits 4 j .. and 4 j + 16 .. of a word (elements 2 j and 2 j + 1 of its eight).
template <int J>
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, const Kv4Scale &k) {
  if constexpr (J == 0) return bf16x2_fma(and_or(w, 0x000f000fu, 0x43004300u), k.s, k.b136);
  return bf16x2_fma(and_or(w >> (J == 0 ? 0 : 4 * J - 3), 0x00780078u, 0x41804180u), k.s, k.b24);
}
// Eight elements as bf16.
__device__ __forceinline__ uint4 kv4_eight(uint32_t w, const Kv4Scale &k) {
  return make_uint4(kv4_pair<0>(w, k), kv4_pair<1>(w, k), kv4_pair<2>(w, k), kv4_pair<3>(w, k));
}

// Half of every value is an fp16 (a multiple of 2^-24, at most 15360), and so is all that
// comes on the way there: 16 + n (bits 6 to 9 of 16.0) times s / 2, less 12 s.  Values that
// are to be weighted are taken so, where the weights can be fp16 too.
struct Kv4Half {
  uint32_t s, b;
};
__device__ __forceinline__ Kv4Half kv4_halves(uint32_t lo, uint32_t hi) {
  const float a = __uint_as_float((lo + KV4_SCALE_BASE - 8) << 20), b = __uint_as_float((hi + KV4_SCALE_BASE - 8) << 20);
  Kv4Half r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r.s) : "f"(b), "f"(a));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r.b) : "r"(r.s), "r"(0xce00ce00u));  // -24
  return r;
}
template <int J>
__device__ __forceinline__ uint32_t kv4_half_pair(uint32_t w, const Kv4Half &k) {
  const uint32_t at = J == 0 ? w << 6 : J == 1 ? w << 2 : J == 2 ? w >> 2 : w >> 6;
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(and_or(at, 0x03c003c0u, 0x4c004c00u)), "r"(k.s), "r"(k.b));
  return d;
}
__device__ __forceinline__ uint4 kv4_half_eight(uint32_t w, const Kv4Half &k) {
  return make_uint4(kv4_half_pair<0>(w, k), kv4_half_pair<1>(w, k), kv4_half_pair<2>(w, k), kv4_half_pair<3>(w, k));
}

// Four elements 4 (c % 2) .. of eight as fp32.
__device__ __forceinline__ float4 kv4_four(uint32_t w, int half, float scale) {
  w >>= 8 * half;
  return make_float4((float)((int)(w & 15) - 8) * scale, (float)((int)(w >> 16 & 15) - 8) * scale,
                     (float)((int)(w >> 4 & 15) - 8) * scale, (float)((int)(w >> 20 & 15) - 8) * scale);
}

__device__ __forceinline__ float max_nan_abs(float a, float b, float c) {  // of magnitudes; NaN when one is
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// A block of 16 values: its scale byte and codes (two words).  `bad` is set for a NaN, which is
// stored as 0, or a magnitude beyond KV4_MOST, stored as that.
//
// A code is x / s rounded, ties to even.  With y = 1 / s rounded, q = x y is off by 2^-23; the
// remainder x - s q is exact in one fma (s has four bits), and q + (x - s q) y then differs
// from x / s by 2^-46 before it is rounded.  That is as good as the quotient itself: x / s is
// halfway between two whole numbers, which are fp32 numbers, or away from there by more
// than its rounding (by 2^-23 / 1.875 of itself at least, as x and s times a half are fp32).
// The sum with 1.5 * 2^23 + 8 rounds it and has the code in its lowest bits; multiplied by
// powers of two the codes add up in their places, and what the sums' upper bits add is known.
__device__ __forceinline__ uint32_t kv4_quantise(float (&x)[KV4_BLOCK], uint32_t (&words)[2], bool &bad) {
  float most = 0.f;
#pragma unroll
  for (int e = 0; e < KV4_BLOCK; e += 2) most = max_nan_abs(most, x[e], x[e + 1]);
  if (!(most <= KV4_MOST)) {
    bad = true;
    most = 0.f;
#pragma unroll
    for (int e = 0; e < KV4_BLOCK; ++e) {
      x[e] = x[e] != x[e] ? 0.f : fminf(fmaxf(x[e], -KV4_MOST), KV4_MOST);
      most = fmaxf(most, fabsf(x[e]));
    }
  }
  // the smallest three-bit mantissa at or above most / 7: round the fp32's bits up
  const int up = (int)((__float_as_uint(__fdiv_rn(most, KV4_LEVELS)) + 0xfffffu) >> 20) - KV4_SCALE_BASE;
  const uint32_t byte = (uint32_t)min(max(up, 0), 255);
  const float s = kv4_scale(byte), y = __frcp_rn(s);
  constexpr float SUM = 12582912.f + 8.f;      // 1.5 * 2^23 + 8
  constexpr uint32_t UPPER = 0x4b400000u;      // its bits without the 8
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0u - UPPER * 0x11111111u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = x[8 * h + e], q = v * y;
      const float n = fmaf(fmaf(-s, q, v), y, q) + SUM;
      w += __float_as_uint(n) << (4 * (e / 2) + 16 * (e % 2));
    }
    words[h] = w;
  }
  return byte;
}

}  // namespace llama
