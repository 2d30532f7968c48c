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
// a): a / 7 rounded to four significant bits, ties to even. The product with
// 1 / 7 is within 2^-23 of the quotient; rounding it to 17 bits first brings
// a tie (a = 7 t) back to t exactly and can not make one, since any other
// quotient of a bf16 or fp16 number is 2^-11 of itself or more away from a tie.
__device__ __forceinline__ uint32_t c4_scale_byte(float a) {
  const float t = fminf(fmaxf(a * (1.f / 7.f), 0x1p-15f), 9216.f);
  uint32_t u = (__float_as_uint(t) + 0x40u) & ~0x7Fu;
  u += 0x7FFFFu + ((u >> 20) & 1u);
  return (u >> 20) - (112u << 3);
}

// Code + 8 of x under the scale whose reciprocal is inv: x / s to nearest
// even. fma(x, 1 / s, 384) rounds the quotient to a multiple of 2^-15,
// which restores a tie (x = (k + 1/2) s) and makes none: any other quotient of
// a bf16 or fp16 number by a scale is 2^-13 or more away from one, the product
// within 2^-20 of it. Adding 1.5 2^23 + 8 - 384 then rounds to a whole number,
// ties to even in the low bits. A magnitude of at most 64512 is below 7.5 s, so no
// code leaves -7..7.
__device__ __forceinline__ float c4_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}
__device__ __forceinline__ uint32_t c4_code(float x, float inv) {  // 0x4B400000 + code + 8
  return __float_as_uint(fmaf(x, inv, 384.f) + (12582912.f + 8.f - 384.f));
}
// for what is not finite or above 64512: NaN is 0, magnitudes are cut
__device__ __forceinline__ float c4_cut(float x) { return x == x ? fminf(fmaxf(x, -64512.f), 64512.f) : 0.f; }

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

// Tokens that a request's row of the block table may stand for: positions, rounded up to whole units of 128, stay ints.
constexpr long long kC4MostTokens = (1ll << 31) - 256;

inline bool c4_page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

// Rows [N][H] of D channels to write that certainly share elements: a stride shorter than a row, or two equal ones.
inline bool c4_rows_overlap(long long token, long long head, int N, int H, int D) {
  return (N > 1 && token < D && token > -D) || (H > 1 && head < D && head > -D) || (N > 1 && H > 1 && token == head);
}

// Let the kernel launched behind this one start its CTAs as these leave; it
// waits with grid_wait() before it reads what this one writes.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch behind a kernel that calls grid_release(); the launched one calls grid_wait().
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kern)(Params...), dim3 grid, int threads, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace scfa
