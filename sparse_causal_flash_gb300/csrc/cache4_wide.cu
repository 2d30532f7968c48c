// Attention over the paged 4-bit cache for many query rows of a request (a
// prompt chunk, a handful of drafted tokens): tcgen05 tiles.
//
// The kernel of cache4_attn.cu holds O in registers: 16 rows are what fits, and
// every further 16 would unpack the cached codes again. Here a unit of 128
// tokens is unpacked once for up to 128 rows, into fp16 tiles in shared memory
// (c s is exact in fp16), and S = Q K^T and O += P V run on tcgen05:
//   warp 0       copies the pages of the next units into a ring of raw stages;
//   warps 2-9    unpack the keys of a stage into one of two tiles (128-byte
//                swizzle), and at an item's first unit put its queries, brought
//                to a largest magnitude in [2^13, 2^14), into TMEM;
//   warps 10-17  unpack the values;
//   warps 1, 22  issue the MMAs of the scores and of the values; both A
//                operands, Q and P, are read from TMEM, so that only B takes
//                shared-memory bandwidth;
//   warps 18-21  softmax, thread = row = TMEM lane; P (fp16, weights times 2^7)
//                overwrites the scores it came from.
// With few rows the 128 lanes hold the same RP = 32 or 64 rows several times,
// and each copy weighs its own part of every unit's tokens (its other weights
// are zero): the softmax of 32 rows then takes a quarter of the time, and the
// copies, which keep their own maximum and sum, meet once per item.
// At 128 channels a unit takes an SM some 2,300 cycles with 32 rows and 3,100
// with 128; the tensor cores are 45% and 30% busy, the issue slots 64% and 59%.
// The MMAs alone, with nothing else running, take 1,300 cycles (80 each, 64 at
// the peak rate). With 32 rows the unpacking warps work for
// 1,800 of a unit's cycles, with 128 the softmax warps for 2,500; eight of those
// instead of four take as long each (141 us instead of 142 in all), and so do
// loads of 16 scores under the work on the 16 before (144). Code size counts: see
// the loops that are not unrolled.
// Two chunks of 500 tokens over 4,000 to 8,000 (96 GFLOP): 136 us and 8 us for
// the join, 650 TFLOP/s, 33% of the measured matrix product; 32 requests with
// drafts of 1 to 7 tokens (276 MB): 145 and 4 us (pages elsewhere: up to 158).
#include <type_traits>

#include "cache4_attn.cuh"

namespace scfa {
namespace {

constexpr int kDqWarps = 16;  // the first eight unpack K, the others V
constexpr int kWideThreads = 32 * (2 + kDqWarps + 4 + 1);
constexpr int kWideStages = 3;
constexpr int kDescs = 16;  // more than the units between the copies and the softmax
constexpr uint32_t kSub = 16384;  // one [128][64] fp16 tile
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColQ2 = 64;  // TMEM columns (S and Q twice)

template <int D>
struct WideSmem {
  uint8_t k[2][D / 64][kSub];
  uint8_t v[2][D / 64][kSub];
  uint8_t raw[kWideStages][kChTiles * C4<D>::kTileBytes];
  float merge[4 * 32 * 32];
  float ml[128][2];
  float factor[4][128];  // by item
  int seen[4][128];
  C4Stage stage[kDescs];
  uint64_t raw_full[kWideStages], raw_empty[kWideStages], desc_full[kDescs];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], q_ready[4];
  // (P and its MMA have two barriers each: the softmax may be a unit ahead of
  // the MMAs, and a single barrier's parity can not tell phases two apart)
  uint64_t p_full[2], pv_done[2], o_empty, group, drain[2];
  C4SpanSmem<kWideThreads> span;
  uint32_t tmem_base;
  int abort_flag;
};


// true in one lane of the warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// kind::f16 with fp16 operands, fp32 accumulators
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int D, bool F16, int RP>
__global__ void __launch_bounds__(kWideThreads, 1) cache4_wide_kernel(C4AttnArgs a) {
  using L = C4<D>;
  constexpr int G = L::kG, S = kWideStages, REP = 128 / RP, KEYS = 128 / REP;
  extern __shared__ uint8_t smem_raw[];
  WideSmem<D>& sm = *reinterpret_cast<WideSmem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  C4Desc* const desc = a.desc + blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], kDqWarps);
    }
    for (int s = 0; s < kDescs; ++s) mbar_init(&sm.desc_full[s], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], 8);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 8);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sm.q_ready[i], 8);
    mbar_init(&sm.o_empty, 4);
    mbar_init(&sm.group, 4);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    fence_mbar_init();
    sm.abort_flag = 0;
    desc->err = SCFA_OK;
    desc->parts = 0;
  }
  grid_release();
  C4Span span;
  if (!c4_span<RP, kWideThreads>(a, sm.span, span)) return;  // (the whole CTA)
  const int n_units = span.units;
  if (warp == 1) tmem_alloc(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, 0), idesc_o = idesc_f16_f32(128, D, 1);
  constexpr uint64_t kBuf16 = (D / 64) * kSub >> 4;
  const uint64_t kdesc = smem_desc_sw128(smem_u32(sm.k[0][0]), 16, 1024);
  const uint64_t vdesc = smem_desc_sw128(smem_u32(sm.v[0][0]), kSub, 1024);
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  volatile int* const abort_flag = &sm.abort_flag;
  int* const err = &desc->err;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    C4Walk<RP> walk;
    walk.begin(a, span, lane);
    C4Pages pages(a);
    int issued = 0;
    for (int u = 0; u < n_units; ++u) {
      const int s = u % S;
      if (u >= S && !wait_all(&sm.raw_empty[s], ((u / S) & 1) ^ 1, abort_flag, err)) break;
      const uint32_t mask = pages.look_up(a, walk, lane, err);
      const bool go = !(a.stall && u == 0);
      if (go) pages.template copy<D>(a, walk, lane, sm.raw[s], &sm.raw_full[s]);
      __syncwarp();
      if (lane == 0) {
        C4Stage d;
        walk.describe(span, u, desc, d);
        d.tiles = static_cast<int>(mask);
        sm.stage[u % kDescs] = d;
        mbar_arrive(&sm.desc_full[u % kDescs]);
        if (go) mbar_arrive_expect_tx(&sm.raw_full[s], __popc(mask) * L::kTileBytes);
      }
      __syncwarp();
      issued = u + 1;
      walk.next(a, u + 1 < n_units);
    }
    // copies in flight land before the shared memory goes
    for (int u = max(0, issued - S); u < issued; ++u)
      if (!(a.stall && u == 0)) mbar_wait_drain(&sm.raw_full[u % S], (u / S) & 1, err);
  } else if (warp == 1) {
    // ------------------------------------------------------------ score MMAs
    // Issuing an MMA takes longer than the MMA: two warps share them. Operand
    // places are constants of the unit's and the item's parity (the whole of
    // TMEM is this CTA's, so its columns begin at 0), and the warps stay
    // together but for the elected lane, so that descriptors are uniform.
    // The loops are not unrolled: the roles of a scheduler share its
    // instruction cache, and fetching code is what most of their waits were.
    int items = 0;
    auto scores = [&](auto unit, auto item) {
      constexpr int I = decltype(unit)::value, Q = decltype(item)::value;
      if (elect_one()) {
        const uint64_t b = kdesc + I * kBuf16;
#pragma unroll 1
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ts(kColS + I * 128, kColQ + Q * kColQ2 + kk * 8, b + kstep_off16(kk, kSub), idesc_s, kk > 0);
        tc_commit(&sm.s_full[I]);
        tc_commit(&sm.k_empty[I]);
      }
      __syncwarp();
    };
    for (int u = 0; u < n_units; ++u) {
      const int i = u & 1;
      if (!wait_all(&sm.desc_full[u % kDescs], (u / kDescs) & 1, abort_flag, err)) break;
      if (sm.stage[u % kDescs].flags & kFirst) ++items;
      // P of u - 2 lies where these scores go
      if (u > 1 && !wait_all(&sm.pv_done[i], ((u - 2) >> 1) & 1, abort_flag, err)) break;
      if (!wait_all(&sm.k_full[i], (u >> 1) & 1, abort_flag, err)) break;
      tc_fence_after();
      if (items & 1) {
        if (i) scores(c1, c0);
        else scores(c0, c0);
      } else {
        if (i) scores(c1, c1);
        else scores(c0, c1);
      }
    }
    if (elect_one()) tc_commit(&sm.drain[0]);
    __syncwarp();
    mbar_wait_drain(&sm.drain[0], 0, err);
  } else if (warp == 22) {
    // ------------------------------------------------------------ value MMAs
    int items = 0;
    auto values = [&](auto unit, uint32_t accumulate) {
      constexpr int I = decltype(unit)::value;
      if (elect_one()) {
        const uint64_t b = vdesc + I * kBuf16;
#pragma unroll 1
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(kColO, kColS + I * 128 + kk * 8, b + static_cast<uint64_t>(kk * 128), idesc_o,
                      kk > 0 ? 1u : accumulate);
        tc_commit(&sm.pv_done[I]);
        tc_commit(&sm.v_empty[I]);
      }
      __syncwarp();
    };
    for (int u = 0; u < n_units; ++u) {
      const int i = u & 1;
      if (!wait_all(&sm.desc_full[u % kDescs], (u / kDescs) & 1, abort_flag, err)) break;
      const bool first = sm.stage[u % kDescs].flags & kFirst;
      if (first && !wait_all(&sm.o_empty, (items++ & 1) ^ 1, abort_flag, err)) break;
      if (!wait_all(&sm.v_full[i], (u >> 1) & 1, abort_flag, err)) break;
      if (!wait_all(&sm.p_full[i], (u >> 1) & 1, abort_flag, err)) break;
      tc_fence_after();
      if (i) values(c1, first ? 0u : 1u);
      else values(c0, first ? 0u : 1u);
    }
    if (elect_one()) tc_commit(&sm.drain[1]);
    __syncwarp();
    mbar_wait_drain(&sm.drain[1], 0, err);
  } else if (warp < 2 + kDqWarps) {
    // ------------------------------------------------------------ unpacking, queries
    const int dw = (warp - 2) & 7, quad = warp & 3, dt = dw * 32 + lane;
    const bool keys = warp < 10;
    const uint32_t k128 = a.k128, magic = a.magic;
    int items = 0;
    for (int u = 0; u < n_units; ++u) {
      const int s = u % S, i = u & 1;
      if (!wait_all(&sm.raw_full[s], (u / S) & 1, abort_flag, err)) break;
      const C4Stage d = sm.stage[u % kDescs];
      const uint8_t* raw = sm.raw[s];
      if (keys) {
        if (!wait_all(&sm.k_empty[i], ((u >> 1) & 1) ^ 1, abort_flag, err)) break;
        if (d.flags & kFirst) {
          // Two warps per TMEM lane quarter, each half of the channels. Q has two
          // places: the scores of the item before last are done, they came two
          // units ago. What the softmax reads has four: it is past the unit four
          // before this one, whose P had to be used up for the scores two before.
          // (those MMAs read the place that is written here: the wait for their commit orders it with this fence)
          tc_fence_after();
          const int ib = items++ & 3, half = dw >> 2;
          const int row = d.row0 + (quad * 32) % RP + lane;
          const bool in = row < d.rows;
          const int tok = in ? row / a.G : 0;
          const uint4* qp = reinterpret_cast<const uint4*>(a.q + (d.tok0 + tok) * a.qt +
                                                           (d.head * a.G + (in ? row - tok * a.G : 0)) * a.qh);
          float mx = 0.f;
          if (in) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = qp[c];
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float2 f = c4_unpack<F16>(x[y]);
                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
          }
          const uint32_t ex = min(253u, 267u - (__float_as_uint(mx) >> 23));
          // an infinity spoils its row whatever the signs of the codes it meets: all of the row becomes NaN (a NaN does so
          // by itself)
          const float up = __uint_as_float(mx < INFINITY ? ex << 23 : 0x7FC00000u);
          uint32_t reg[D / 4];
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint4 v = in ? qp[half * (D / 16) + c] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 f = c4_unpack<F16>(x[y]);
              reg[4 * c + y] = c4_pack<true>(f.x * up, f.y * up);
            }
          }
          const uint32_t col =
              tmem + (static_cast<uint32_t>(quad * 32) << 16) + kColQ + (ib & 1) * kColQ2 + half * (D / 4);
          if constexpr (D == 128) tmem_st32(col, reg);
          else tmem_st16(col, reg);
          if (half == 0) {
            sm.factor[ib][quad * 32 + lane] = fmaxf(a.factor * __uint_as_float((254u - ex) << 23), 0x1p-126f);
            sm.seen[ib][quad * 32 + lane] = in ? a.vis[d.tok0 + tok] : INT_MAX;
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.q_ready[ib]);
        }
        // K: lane = (key, j), the 8 channels 32 g + 8 j of every group
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int key = (dt >> 2) + 64 * x, j = dt & 3, tile = key >> 4, t = key & 15;
          const uint8_t* p = raw + tile * L::kTileBytes;
          uint32_t w[G], sb;
          if (G == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + L::k_row(t) + j * 16);
            w[0] = v.x, w[1] = v.y, w[G - 2] = v.z, w[G - 1] = v.w;
            sb = *reinterpret_cast<const uint32_t*>(p + L::kKScales + t * 4);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p + L::k_row(t) + j * 8);
            w[0] = v.x, w[1] = v.y;
            sb = *reinterpret_cast<const uint16_t*>(p + L::kKScales + t * 2);
          }
          // what is not a visible row may hold scales that are infinite in fp16
          if (!(d.tiles >> tile & 1) || d.base + key >= d.seen) sb = 0;
          const bool odd = key & 1;  // odd keys take the groups of a pair the other way round: no bank twice
          uint8_t* const row = &sm.k[i][0][0] + key * 128;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t word = odd ? w[g ^ 1] : w[g];
            const uint32_t sel = odd ? (0x4040u | (g ^ 1) | (g ^ 1) << 8) : (0x4040u | g | g << 8);
            const uint32_t sc = __byte_perm(sb, 0u, sel) * k128 + 0x04000400u;
            const int chunk = ((odd ? (g ^ 1) : g) & 1) * 4 + j;
            *reinterpret_cast<uint4*>(row + (g >> 1) * kSub + ((chunk ^ (key & 7)) << 4)) = c4_unpack8(word, sc, magic);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.k_full[i]);
          mbar_arrive(&sm.raw_empty[s]);
        }
      } else {
        // V: lane = (key, r). A 64-column half holds groups 2 x and 2 x + 1, column 8 r + 2 i + b = channel
        // 32 (2 x + b) + 4 r + i
        if (!wait_all(&sm.v_empty[i], ((u >> 1) & 1) ^ 1, abort_flag, err)) break;
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          const int item = dw + 8 * x, key = (item >> 1) * 8 + (lane & 7), r = (item & 1) * 4 + (lane >> 3);
          const int tile = key >> 4, t = key & 15;
          const uint8_t* p = raw + tile * L::kTileBytes;
          uint32_t w[G / 2], sb;
          if (G == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + L::v_piece(t, r));
            w[0] = v.x, w[G / 2 - 1] = v.y;
            sb = *reinterpret_cast<const uint32_t*>(p + L::kVScales + t * 4);
          } else {
            w[0] = *reinterpret_cast<const uint32_t*>(p + L::v_piece(t, r));
            sb = *reinterpret_cast<const uint16_t*>(p + L::kVScales + t * 2);
          }
          if (!(d.tiles >> tile & 1) || d.base + key >= d.seen) sb = 0;
          uint8_t* const row = &sm.v[i][0][0] + key * 128 + ((r ^ (key & 7)) << 4);
#pragma unroll
          for (int y = 0; y < G / 2; ++y) {
            const uint32_t sc = __byte_perm(sb, 0u, y ? 0x4342 : 0x4140) * k128 + 0x04000400u;
            *reinterpret_cast<uint4*>(row + y * kSub) = c4_unpack8(w[y], sc, magic);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.v_full[i]);
          mbar_arrive(&sm.raw_empty[s]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, rep = quad * 32 / RP, key_lo = rep * KEYS;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t key_tiles = ((1u << (KEYS / 16)) - 1u) << (key_lo / 16);
    float m = kNoMax, l = 0.f, f = 0.f;
    int row_seen = 0, items = 0, syncs = 0;
    auto group_sync = [&]() -> bool {  // the four warps, bounded
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.group);
      return wait_all(&sm.group, syncs++ & 1, abort_flag, err);
    };
    bool ok = true;
    for (int u = 0; ok && u < n_units; ++u) {
      const int i = u & 1;
      if (!wait_all(&sm.desc_full[u % kDescs], (u / kDescs) & 1, abort_flag, err)) break;
      const C4Stage d = sm.stage[u % kDescs];
      const bool first = d.flags & kFirst;
      if (first) {
        const int ib = items & 3;
        if (!wait_all(&sm.q_ready[ib], (items >> 2) & 1, abort_flag, err)) break;
        ++items;
        f = sm.factor[ib][quad * 32 + lane];
        row_seen = sm.seen[ib][quad * 32 + lane];
        m = kNoMax;
        l = 0.f;
      }
      if (!wait_all(&sm.s_full[i], (u >> 1) & 1, abort_flag, err)) break;
      tc_fence_after();
      const uint32_t sc = lanes + kColS + i * 128;
      const int key0 = d.base + key_lo;
      const bool edge = (static_cast<uint32_t>(d.tiles) & key_tiles) != key_tiles ||
                        __any_sync(0xffffffffu, key0 + KEYS > row_seen);
      uint32_t x[32];
      auto load = [&](int c) {
        tmem_ld32(sc + key_lo + 32 * c, x);
        tmem_wait_ld();
        tmem_ld_fence(x);
      };
      // scores out of sight to -inf, in TMEM: the loops below stay short
#pragma unroll 1
      for (int c = edge ? 0 : KEYS / 32; c < KEYS / 32; ++c) {
        load(c);
        const int n = min(max(row_seen - (key0 + 32 * c), 0), 32);
        const uint32_t tt = static_cast<uint32_t>(d.tiles) >> ((key_lo + 32 * c) / 16);
        const uint32_t bits =
            (n == 32 ? 0xFFFFFFFFu : (1u << n) - 1u) & ((tt & 1 ? 0xFFFFu : 0u) | (tt & 2 ? 0xFFFF0000u : 0u));
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!(bits >> e & 1)) x[e] = 0xFF800000u;
        tmem_st32(sc + key_lo + 32 * c, x);
        tmem_wait_st();
      }
      float mx = -INFINITY, mx2 = -INFINITY, l2 = 0.f;
#pragma unroll 1
      for (int c = 0; c < KEYS / 32; ++c) {
        load(c);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          mx = max3f(mx, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          mx2 = max3f(mx2, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
        }
      }
      mx = fmaxf(mx, mx2);
      // the reference moves only when a weight would exceed 2^15
      mx = __fmul_rn(mx, f);
      if (__any_sync(0xffffffffu, __fsub_rn(mx, m) > 15.f)) {
        const float mn = fmaxf(m, mx - 7.f), fix = ex2_approx(m - mn);
        m = mn;
        l *= fix;
        if (!first) {
          if (!wait_all(&sm.pv_done[i ^ 1], ((u - 1) >> 1) & 1, abort_flag, err)) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(lanes + kColO + 32 * c, o);
            tmem_wait_ld();
            tmem_ld_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fix);
            tmem_st32(lanes + kColO + 32 * c, o);
          }
          tmem_wait_st();
          if (KEYS == 32) load(0);
        }
      }
      const uint64_t mm = f2(-m, -m);
#pragma unroll 1
      for (int c = 0; c < KEYS / 32; ++c) {
        if (KEYS > 32) load(c);
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          // (two multiplications that are rounded, one packed subtraction; packed both gave infinities for far scores, as
          // one rounding for both would)
          float y0, y1;
          f2_split(add2(f2(__fmul_rn(__uint_as_float(x[e]), f), __fmul_rn(__uint_as_float(x[e + 1]), f)), mm), y0, y1);
          const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
          l += p0;
          l2 += p1;
          p[e / 2] = c4_pack<true>(p0, p1);
        }
        // P of keys 32 c.. lies over scores that have been read
        tmem_st16(sc + (key_lo + 32 * c) / 2, p);
      }
      l += l2;
      if (REP > 1) {  // the other copies' tokens weigh nothing here
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 32 < key_lo || c * 32 >= key_lo + KEYS) tmem_st16(sc + 16 * c, z);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[i]);

      if (d.flags & kLast) {
        if (!wait_all(&sm.pv_done[i], (u >> 1) & 1, abort_flag, err)) break;
        tc_fence_after();
        const bool tail = d.flags & kOpenStart, open = d.flags & kOpenEnd;
        const int row = (quad * 32) % RP + lane, grow = d.row0 + row;
        const bool in = grow < d.rows;
        float mt = m, lt = l, weight = 1.f;
        if (REP > 1) {
          sm.ml[quad * 32 + lane][0] = m;
          sm.ml[quad * 32 + lane][1] = l;
          if (!(ok = group_sync())) break;
          lt = 0.f;
#pragma unroll
          for (int y = 0; y < REP; ++y) mt = fmaxf(mt, sm.ml[y * RP + row][0]);
#pragma unroll
          for (int y = 0; y < REP; ++y) lt = fmaf(sm.ml[y * RP + row][1], ex2_approx(sm.ml[y * RP + row][0] - mt), lt);
          weight = ex2_approx(m - mt);
        }
        const float inv = lt != 0.f ? 1.f / lt : 0.f;
        const int tok = d.tok0 + (in ? grow / a.G : 0), head = d.head * a.G + (in ? grow % a.G : 0);
        const long long at = (static_cast<long long>(blockIdx.x) * 2 + (tail ? 0 : 1)) * RP + row;
        uint16_t* const op = a.o + tok * a.ot + head * a.oh;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(lanes + kColO + 32 * c, o);
          tmem_wait_ld();
          tmem_ld_fence(o);
          // columns 8 r + 2 i + b of half c >> 1: channels 32 (2 (c >> 1) + b) + 16 (c & 1) + 4 r + i
          const int ch0 = 64 * (c >> 1) + 16 * (c & 1);
          if (REP == 1) {
            if (in) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[8 * (e >> 2) + 2 * (e & 3) + b]);
                if (!tail && !open) {
                  uint32_t z[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) z[e] = c4_pack<F16>(v[2 * e] * inv, v[2 * e + 1] * inv);
                  *reinterpret_cast<uint4*>(op + ch0 + 32 * b) = make_uint4(z[0], z[1], z[2], z[3]);
                  *reinterpret_cast<uint4*>(op + ch0 + 32 * b + 8) = make_uint4(z[4], z[5], z[6], z[7]);
                } else {
#pragma unroll
                  for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4*>(a.part + at * D + ch0 + 32 * b + e) =
                        make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
              }
            }
          } else {
            // the copies of a row add up: each takes its share of the 32 columns
#pragma unroll
            for (int e = 0; e < 32; ++e) sm.merge[(quad * 32 + e) * 32 + lane] = __uint_as_float(o[e]) * weight;
            if (!(ok = group_sync())) break;
            constexpr int SH = 32 / REP;  // columns: SH / 8 values of r
#pragma unroll
            for (int z = 0; z < SH / 8; ++z) {
              const int r = rep * (SH / 8) + z;
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                v[e] = 0.f;
#pragma unroll
                for (int y = 0; y < REP; ++y)
                  v[e] += sm.merge[(((quad * 32) % RP / 32 + y * (RP / 32)) * 32 + 8 * r + e) * 32 + lane];
              }
              if (in) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const int ch = ch0 + 32 * b + 4 * r;
                  if (!tail && !open)
                    *reinterpret_cast<uint2*>(op + ch) = make_uint2(c4_pack<F16>(v[b] * inv, v[2 + b] * inv),
                                                                    c4_pack<F16>(v[4 + b] * inv, v[6 + b] * inv));
                  else
                    *reinterpret_cast<float4*>(a.part + at * D + ch) = make_float4(v[b], v[2 + b], v[4 + b], v[6 + b]);
                }
              }
            }
            if (!(ok = group_sync())) break;
          }
        }
        if (!ok) break;
        if (in && rep == 0) {
          if (!tail && !open) {
            a.lse[static_cast<long long>(tok) * a.Hq + head] =
                lt != 0.f ? (mt + log2f(lt)) * 0.69314718055994531f : -INFINITY;
          } else {
            a.ml[2 * at] = mt;
            a.ml[2 * at + 1] = lt;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, bool F16, int RP>
cudaError_t launch(int grid, const C4AttnArgs& a, cudaStream_t st) {
  return launch_and_join<D, F16, RP>(cache4_wide_kernel<D, F16, RP>, grid, kWideThreads, sizeof(WideSmem<D>) + 1024, a,
                                     st);
}

template <int D, bool F16>
cudaError_t launch_rp(int rp, int grid, const C4AttnArgs& a, cudaStream_t st) {
  return rp == 32   ? launch<D, F16, 32>(grid, a, st)
         : rp == 64 ? launch<D, F16, 64>(grid, a, st)
                    : launch<D, F16, 128>(grid, a, st);
}

}  // namespace

cudaError_t launch_cache4_wide(int D, bool f16, int rp, int grid, const C4AttnArgs& a, cudaStream_t st) {
  if (D == 64) return f16 ? launch_rp<64, true>(rp, grid, a, st) : launch_rp<64, false>(rp, grid, a, st);
  return f16 ? launch_rp<128, true>(rp, grid, a, st) : launch_rp<128, false>(rp, grid, a, st);
}

}  // namespace scfa
