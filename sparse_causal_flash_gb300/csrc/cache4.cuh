// The 4-bit row format of the paged cache (scfa.h, "Paged key/value cache held
// in 4 bits"), shared by the kernels that write, read and attend over it.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace scfa {

constexpr int kC4Tile = 16;  // tokens per tile

// Byte offsets inside one tile of one head, D channels.
template <int D>
struct C4 {
  static constexpr int kG = D / 32;                 // groups per row
  static constexpr int kKCodes = 0;                 // [16][4][G] words
  static constexpr int kVCodes = kC4Tile * D / 2;   // [2][8][4][2][G] half words
  static constexpr int kKScales = 2 * kVCodes;      // [16][G] bytes
  static constexpr int kVScales = kKScales + kC4Tile * kG;
  static constexpr int kTileBytes = kVScales + kC4Tile * kG;
  static_assert(kTileBytes == kC4Tile * (D + D / 16), "4.25 bits per value");
  // the row of token t (0..15): its K words start here, word (j, g) at + (j * G + g) * 4
  __host__ __device__ static constexpr int k_row(int t) { return kKCodes + t * (D / 2); }
  // V half words of token t, channel quad r: G consecutive half words
  __host__ __device__ static constexpr int v_piece(int t, int r) {
    return kVCodes + (t >> 3) * 4 * D + r * 16 * kG + ((t >> 1) & 3) * 4 * kG + (t & 1) * 2 * kG;
  }
};

// first byte of the tile that holds slot `at` (place inside its page) of `head`
__device__ __forceinline__ long long c4_tile_base(long long page, int Hkv, int head, int page_size, int at,
                                                  int tile_bytes) {
  return ((page * Hkv + head) * (page_size / kC4Tile) + at / kC4Tile) * tile_bytes;
}

// scale byte -> its value times 2^(shift - 112) for an exponent offset `shift`
// (112: the value itself). Every byte is a finite positive number.
__device__ __forceinline__ float c4_scale(uint32_t b, uint32_t shift = 112u) {
  return __uint_as_float((b << 20) + (shift << 23));
}

// Scale byte of a group with largest magnitude a (a NaN has been left out of
// a). a / 7 must be the correctly rounded quotient: bf16 and fp16 inputs then
// round to four bits exactly as the real quotient does (a = 7 t for a tie t
// divides exactly, any other quotient is at least 2^-15 of itself away).
__device__ __forceinline__ uint32_t c4_scale_byte(float a) {
  const float t = fminf(fmaxf(__fdiv_rn(a, 7.f), 0x1p-15f), 9216.f);
  uint32_t u = __float_as_uint(t);
  u += 0x7FFFFu + ((u >> 20) & 1u);
  return (u >> 20) - (112u << 3);
}

// code + 8 of x under scale s: x / s to nearest even, within -7..7. The
// quotient is correctly rounded, so a tie (x = (k + 1/2) s, exact) stays one.
__device__ __forceinline__ uint32_t c4_code(float x, float s) {
  x = x == x ? x : 0.f;
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x, s)), -7.f), 7.f)) + 8);
}

template <bool F16>
__device__ __forceinline__ float2 c4_unpack(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t c4_pack(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

inline bool c4_page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

}  // namespace scfa
