// Attention of new tokens over the paged 4-bit cache.
//
// One pass over the cached tokens with the running maximum and sum of the
// softmax. An item is up to 8 * NT query rows (token, head) of one request
// that share a key head; its tokens are walked in chunks of 128, and the
// chunks of all items, in one long line, are cut into equal pieces, one per
// CTA of a grid that fills the GPU: a ragged batch and one long request are
// spread alike. An item that falls into several pieces leaves partial rows
// (O, m, l in fp32), which a second kernel joins in a fixed order, so results
// do not depend on scheduling.
//
// A CTA is a producer warp, which walks the block table and copies whole
// tiles of the pages into a ring of shared-memory stages, and four warps that
// each take two 16-token tiles of every chunk with their own m, l and O (they
// meet once per item). The cached codes are the A operands: S^T = K Q^T and
// O^T = V^T P^T with 16 keys or channels by 8 query rows by 16, so up to 8
// rows cost what one does, and the page layout is the operand layout: no
// shuffle between the copy and the MMA. The matrix instructions are the
// warp-level ones: they are 20% busy here.
//   Both operands are fp16, whatever the rows' type. Unpacking bounds the
//   kernel: per eight codes one shift and four AND(-OR)s on the ALU, the rest,
//   for V an addition and a multiplication a pair, on the FMA pipe, both at half
//   rate. Of the 2.9 (128 channels) or 3.8 (64) lane operations a value takes in
//   all, some 1.7 unpack it; over the whole of the two cases below the issue
//   slots are 51% and 67% busy, the ALU 39% and 51%.
//   One request of 131,072 tokens, 8 key heads of 128 channels, 4 query heads
//   each (143 MB): 37 us, 3.9 TB/s, 57% of the copy rate, some 5 us of it before
//   the first unit's data; the join 7 us more. 61 ragged requests, 12 heads of 64
//   channels (408 MB): 123 us, 3.3 TB/s. 8 requests of up to 512: 6 + 4 us.
//   K: the bits of c + 8 are read as a subnormal, (c + 8) 2^-24 (2^-20 for
//      the upper half of a byte, whose query channels are divided by 16); the
//      offset comes off as -8 sum(q), with the group's scale, in fp32. A query
//      row is brought to a largest magnitude in [2^13, 2^14) by a power of two.
//      It is then exact in fp16 down to 2^-23 of that magnitude if it was fp16
//      (2^-26 if bf16), what is smaller within 2^-34 of it; the channels that
//      are not divided by 16 have four bits more.
//   V: codes become c s in fp16 (exact: seven significant bits below 2^16).
//      P is held times 2^7 in fp16, so weights down to 2^-32 of the largest
//      count; each is rounded once (2^-11 of itself), as 16-bit operands ask,
//      while their sum takes them in 32 bits.
#include <cmath>

#include "cache4_attn.cuh"

namespace scfa {
namespace {

constexpr int kWarps = 4;  // compute warps
constexpr int kTpw = kChTiles / kWarps;
constexpr int kThreads = 32 * (kWarps + 1);

// The query rows of an item, as the producer leaves them: B operands of the
// score MMAs, and per row what turns sums into scores.
template <int D, int NT>
struct C4Queries {
  uint4 frag[NT][D / 32][32];
  float offset[NT][D / 32][8];  // -8 2^-24 sum(q) per group
  float factor[8 * NT];         // score in log2 units = sum * factor
  int seen[8 * NT];             // tokens that the row sees
  int all_see[4];               // [0]: tokens that every row sees
};

template <int D, int NT>
struct C4Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = kChTiles * C4<D>::kTileBytes;
  static constexpr int kCtas = NT == 1 ? (D == 128 ? 3 : 4) : 2;  // per SM
  static constexpr int kStages = NT == 1 ? (D == 128 ? 3 : 4) : (D == 128 ? 4 : 6);
  static constexpr size_t kPartBytes = sizeof(float) * kWarps * kRows * D;
  static constexpr size_t kSmem =
      static_cast<size_t>(kStages) * (kStageBytes + sizeof(C4Queries<D, NT>)) + kPartBytes;
};

// Place of four channels of a row in the warps' partial O: chunks are swapped
// by row so that a warp's stores (two rows per lane quad) meet no bank twice.
template <int D>
__device__ __forceinline__ int c4_part_at(int row, int chunk) {
  return row * D + (chunk ^ (row & 6)) * 4;
}

// d = a b + c, 16 x 8 x 16
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                        float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// transpose of an 8 x 8 matrix of 16-bit values, one row per four lanes
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The query rows from row0 on of key head h, by one warp: lane (r8, j) takes
// channels 32 g + 8 j + 0..7 of row r8, the B operand's place of them. Their
// loads come first, the pages' copies next, the work on them last.
template <int D, int NT>
struct C4Raw {
  uint4 v[NT][D / 32];
  int seen[NT];
};
template <int D, int NT>
__device__ __forceinline__ void c4_load_queries(const C4AttnArgs& a, const C4Req& q, int row0, int h, int lane,
                                                C4Raw<D, NT>& x) {
  const int r8 = lane >> 2, j = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + nt * 8 + r8, tok = row / a.G;
    const bool in = row < q.rows;
    const uint16_t* p = a.q + (q.tok0 + tok) * a.qt + (h * a.G + row - tok * a.G) * a.qh + 8 * j;
#pragma unroll
    for (int g = 0; g < D / 32; ++g)
      x.v[nt][g] = in ? *reinterpret_cast<const uint4*>(p + 32 * g) : make_uint4(0u, 0u, 0u, 0u);
    x.seen[nt] = in ? a.vis[q.tok0 + tok] : INT_MAX;
  }
}
template <int D, bool F16, int NT>
__device__ __forceinline__ void c4_queries(const C4AttnArgs& a, const C4Raw<D, NT>& x, int lane, C4Queries<D, NT>& s) {
  constexpr int G = D / 32;
  const int r8 = lane >> 2, j = lane & 3;
  auto& v = x.v;
  auto& seen = x.seen;
  int all = INT_MAX;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mx = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t in4[4] = {v[nt][g].x, v[nt][g].y, v[nt][g].z, v[nt][g].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float2 f = c4_unpack<F16>(in4[y]);
        mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // exponent of the power of two that brings the row to [2^13, 2^14)
    const uint32_t ex = min(253u, 267u - (__float_as_uint(mx) >> 23));
    const float up = __uint_as_float(ex << 23);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t in4[4] = {v[nt][g].x, v[nt][g].y, v[nt][g].z, v[nt][g].w};
      uint32_t hq[4];
      float sum = 0.f;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float2 f = c4_unpack<F16>(in4[y]);
        const float k = (y & 1) ? up * 0.0625f : up;
        hq[y] = c4_pack<true>(f.x * k, f.y * k);
        sum += f.x * up + f.y * up;
      }
      s.frag[nt][g][lane] = make_uint4(hq[0], hq[1], hq[2], hq[3]);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (j == 0) s.offset[nt][g][r8] = sum * (-8.f * 0x1p-24f);
    }
    if (j == 0) {
      // times 2^(24 + 127 - ex), in two steps so that no product between leaves fp32
      const int e = 24 + 127 - static_cast<int>(ex), e1 = e >> 1;
      const float half = __uint_as_float(static_cast<uint32_t>(127 + e1) << 23);
      const float rest = __uint_as_float(static_cast<uint32_t>(127 + e - e1) << 23);
      s.factor[nt * 8 + r8] = fmaxf(a.factor * half * rest, 0x1p-126f);
      s.seen[nt * 8 + r8] = seen[nt];
    }
    all = min(all, seen[nt]);
  }
  all = __reduce_min_sync(0xffffffffu, all);
  if (lane == 0) s.all_see[0] = all;
}

template <int D, bool F16, int NT>
__global__ void __launch_bounds__(kThreads, C4Cfg<D, NT>::kCtas) cache4_attn_kernel(C4AttnArgs a) {
  using L = C4<D>;
  using C = C4Cfg<D, NT>;
  constexpr int G = L::kG, ROWS = C::kRows, S = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[S], empty[S], mfull, mempty;
  __shared__ C4Stage stage[S];
  __shared__ float s_ml[kWarps][ROWS][2];
  __shared__ C4SpanSmem<kThreads> s_span;
  __shared__ volatile int abort_flag;
  C4Queries<D, NT>* const s_q = reinterpret_cast<C4Queries<D, NT>*>(smem + static_cast<size_t>(S) * C::kStageBytes);
  float* const s_part = reinterpret_cast<float*>(s_q + S);

  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  C4Desc* const desc = a.desc + blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    mbar_init(&mfull, kWarps);
    mbar_init(&mempty, kWarps);
    fence_mbar_init();
    abort_flag = 0;
    desc->err = SCFA_OK;
    desc->parts = 0;
  }

  grid_release();
  C4Span span;
  if (!c4_span<ROWS, kThreads>(a, s_span, span)) return;  // (the whole CTA)
  __syncthreads();
  const int n_units = span.units;

  if (w == kWarps) {
    // ================================================= producer
    C4Walk<ROWS> walk;
    walk.begin(a, span, lane);
    C4Pages pages(a);
    int issued = 0, qslot = -1;
    for (int u = 0; u < n_units; ++u) {
      const int s = u % S;
      if (u >= S && !wait_all(&empty[s], ((u / S) & 1) ^ 1, &abort_flag, &desc->err)) break;
      const bool first = walk.ch == 0 || u == 0;
      C4Raw<D, NT> raw;
      if (first) c4_load_queries<D, NT>(a, walk.q, walk.b * ROWS, walk.h, lane, raw);
      const uint32_t mask = pages.look_up(a, walk, lane, &desc->err);
      const bool go = !(a.stall && u == 0);
      if (go) pages.copy<D>(a, walk, lane, smem + static_cast<size_t>(s) * C::kStageBytes, &full[s]);
      if (first) {
        // at most S items have units in the ring, so the slot of the item S before is free
        if (++qslot == S) qslot = 0;
        c4_queries<D, F16, NT>(a, raw, lane, s_q[qslot]);
      }
      __syncwarp();
      if (lane == 0) {
        C4Stage d;
        walk.describe(span, u, desc, d);
        d.tiles = static_cast<int>(mask);
        d.qslot = qslot;
        stage[s] = d;
        // (the copies may have landed already: the phase ends with this arrival and all bytes)
        if (go) mbar_arrive_expect_tx(&full[s], __popc(mask) * L::kTileBytes);
      }
      __syncwarp();
      issued = u + 1;
      walk.next(a, u + 1 < n_units);
    }
    // copies in flight land before the shared memory goes
    for (int u = max(0, issued - S); u < issued; ++u)
      if (!(a.stall && u == 0)) mbar_wait_drain(&full[u % S], (u / S) & 1, &desc->err);
    return;
  }

  // =================================================== compute warps
  const int r8 = lane >> 2, j = lane & 3;
  const uint32_t k16 = a.k16, k128 = a.k128, magic = a.magic;
  float O[NT][G][2][4];
  float factor[NT][2];
  float m[NT][2], l[NT][2];  // reference of the weights (a running maximum - 7), and their sum
  int items = 0;
  for (int u = 0; u < n_units; ++u) {
    const int s = u % S;
    if (!wait_all(&full[s], (u / S) & 1, &abort_flag, &desc->err)) return;
    const C4Stage d = stage[s];
    const C4Queries<D, NT>& qs = s_q[d.qslot];
    if (d.flags & kFirst) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int y = 0; y < 4; ++y) O[nt][g][0][y] = O[nt][g][1][y] = 0.f;
        const float2 f = *reinterpret_cast<const float2*>(&qs.factor[nt * 8 + 2 * j]);
        factor[nt][0] = f.x, factor[nt][1] = f.y;
        m[nt][0] = m[nt][1] = kNoMax;
        l[nt][0] = l[nt][1] = 0.f;
      }
    }
    const int t0 = w * kTpw;
    const uint32_t there = static_cast<uint32_t>(d.tiles) >> t0 & ((1u << kTpw) - 1u);
    if (there != 0) {
      const uint8_t* tile0 = smem + static_cast<size_t>(s) * C::kStageBytes + t0 * L::kTileBytes;
      float x[kTpw][NT][4];
      // ---- scores
      uint32_t kw[kTpw][2][G], ks[kTpw][2];
#pragma unroll
      for (int i = 0; i < kTpw; ++i) {
        const uint8_t* tile = tile0 + i * L::kTileBytes;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint8_t* p = tile + L::k_row(r8 + 8 * y) + j * 4 * G;
          if (G == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            kw[i][y][0] = v.x, kw[i][y][1] = v.y, kw[i][y][G - 2] = v.z, kw[i][y][G - 1] = v.w;
            ks[i][y] = *reinterpret_cast<const uint32_t*>(tile + L::kKScales + (r8 + 8 * y) * G);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            kw[i][y][0] = v.x, kw[i][y][1] = v.y;
            ks[i][y] = *reinterpret_cast<const uint16_t*>(tile + L::kKScales + (r8 + 8 * y) * G);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[i][nt][0] = x[i][nt][1] = x[i][nt][2] = x[i][nt][3] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint4 qv[NT];
        float2 x0[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          qv[nt] = qs.frag[nt][g][lane];
          x0[nt] = *reinterpret_cast<const float2*>(&qs.offset[nt][g][2 * j]);
        }
#pragma unroll
        for (int i = 0; i < kTpw; ++i) {
          uint32_t A[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t lo = kw[i][y][g], hi = lo >> 8;
            A[0][y] = lo & 0x000F000Fu, A[0][y + 2] = lo & 0x00F000F0u;
            A[1][y] = hi & 0x000F000Fu, A[1][y + 2] = hi & 0x00F000F0u;
          }
          // scale = (b << 20) + (112 << 23), from the byte at bits 16-23
          const float s0 = __uint_as_float(__byte_perm(ks[i][0], 0u, 0x4044 | g << 8) * k16 + (112u << 23));
          const float s1 = __uint_as_float(__byte_perm(ks[i][1], 0u, 0x4044 | g << 8) * k16 + (112u << 23));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma_f16(acc, A[0], qv[nt].x, qv[nt].y, 0.f, 0.f, 0.f, 0.f);
            mma_f16(acc, A[1], qv[nt].z, qv[nt].w, acc[0], acc[1], acc[2], acc[3]);
            x[i][nt][0] = fmaf(acc[0] + x0[nt].x, s0, x[i][nt][0]);
            x[i][nt][1] = fmaf(acc[1] + x0[nt].y, s0, x[i][nt][1]);
            x[i][nt][2] = fmaf(acc[2] + x0[nt].x, s1, x[i][nt][2]);
            x[i][nt][3] = fmaf(acc[3] + x0[nt].y, s1, x[i][nt][3]);
          }
        }
      }
      const int key0 = d.base + t0 * kC4Tile;
      if (there != (1u << kTpw) - 1u || key0 + kTpw * kC4Tile > qs.all_see[0]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int2 seen = *reinterpret_cast<const int2*>(&qs.seen[nt * 8 + 2 * j]);
#pragma unroll
          for (int i = 0; i < kTpw; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(there >> i & 1) || key0 + i * kC4Tile + r8 + 8 * (e >> 1) >= ((e & 1) ? seen.y : seen.x))
                x[i][nt][e] = -INFINITY;
        }
      }
      // ---- softmax: the reference moves only when a weight would exceed 2^15
      uint32_t P[kTpw][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        bool over = false;
#pragma unroll
        for (int i = 0; i < kTpw; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[i][nt][e] = __fmul_rn(x[i][nt][e], factor[nt][e & 1]);  // in log2 units
            over |= __fsub_rn(x[i][nt][e], m[nt][e & 1]) > 15.f;
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < kTpw; ++i) mx = fmaxf(mx, fmaxf(x[i][nt][c], x[i][nt][c + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(m[nt][c], mx - 7.f);
            const float f = ex2_approx(m[nt][c] - mx);
            m[nt][c] = mx;
            l[nt][c] *= f;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int t = 0; t < 2; ++t) O[nt][g][t][c] *= f, O[nt][g][t][c + 2] *= f;
          }
        }
#pragma unroll
        for (int i = 0; i < kTpw; ++i) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = ex2_approx(__fsub_rn(x[i][nt][e], m[nt][e & 1]));
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          P[i][nt][0] = transpose8(c4_pack<true>(p[0], p[1]));
          P[i][nt][1] = transpose8(c4_pack<true>(p[2], p[3]));
        }
      }
      // ---- values
#pragma unroll
      for (int i = 0; i < kTpw; ++i) {
        const uint8_t* tile = tile0 + i * L::kTileBytes;
        uint32_t vw[2][2][G / 2];  // [keys 0-7 / 8-15][key 2 j + ..][groups 2 y, 2 y + 1]
        uint32_t vs[2][2];         // scale bytes of those keys
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint8_t* p = tile + L::kVCodes + y * 4 * D + r8 * 16 * G + j * 4 * G;
          const uint8_t* q = tile + L::kVScales + (8 * y + 2 * j) * G;
          if (G == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            vw[y][0][0] = v.x, vw[y][0][G / 2 - 1] = v.y, vw[y][1][0] = v.z, vw[y][1][G / 2 - 1] = v.w;
            const uint2 f = *reinterpret_cast<const uint2*>(q);
            vs[y][0] = f.x, vs[y][1] = f.y;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            vw[y][0][0] = v.x, vw[y][1][0] = v.y;
            const uint32_t f = *reinterpret_cast<const uint32_t*>(q);
            vs[y][0] = f & 0xFFFFu, vs[y][1] = f >> 16;
          }
        }
        // scale bytes behind the last visible token are not a row's: they could
        // be infinite in fp16
        if (there != (1u << kTpw) - 1u || key0 + kTpw * kC4Tile > d.seen) {
          const int n = there >> i & 1 ? d.seen - key0 - i * kC4Tile : 0;
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              if (8 * y + 2 * j + b >= n) vs[y][b] = 0;
        }
        uint32_t sb[2][2][2];  // [y][group parity][key]: two scale bytes, in bits 0-7 and 16-23
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            sb[y][0][b] = vs[y][b] & 0x00FF00FFu;
            sb[y][1][b] = __byte_perm(vs[y][b], 0u, 0x4341);
          }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          uint32_t A[2][4];  // channels 4 r + 2 t, + 1 of two m16 tiles
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t lo = __byte_perm(vw[y][0][g / 2], vw[y][1][g / 2], (g & 1) ? 0x7632 : 0x5410);
            // the two keys' scales times 2: fp16 bits (b << 7) + (1 << 10), normal for every byte of a row
            const uint32_t sc =
                __byte_perm(sb[y][g & 1][0], sb[y][g & 1][1], g < 2 ? 0x5410 : 0x7632) * k128 + 0x04000400u;
            const uint4 v = c4_unpack8(lo, sc, magic);
            A[0][2 * y] = v.x, A[0][2 * y + 1] = v.y;
            A[1][2 * y] = v.z, A[1][2 * y + 1] = v.w;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              float(&z)[4] = O[nt][g][t];
              mma_f16(z, A[t], P[i][nt][0], P[i][nt][1], z[0], z[1], z[2], z[3]);
            }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    if (d.flags & kLast) {
      // ---- the four warps' rows become one
      if (items > 0 && !wait_all(&mempty, (items - 1) & 1, &abort_flag, &desc->err)) return;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float z = l[nt][c];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
          const int row = nt * 8 + 2 * j + c;
          if (r8 == 0) s_ml[w][row][0] = m[nt][c], s_ml[w][row][1] = z;
#pragma unroll
          for (int g = 0; g < G; ++g)
            *reinterpret_cast<float4*>(s_part + c4_part_at<D>(w * ROWS + row, 8 * g + r8)) =
                make_float4(O[nt][g][0][c], O[nt][g][0][c + 2], O[nt][g][1][c], O[nt][g][1][c + 2]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&mfull);
      if (!wait_all(&mfull, items & 1, &abort_flag, &desc->err)) return;
      constexpr int CPT = D / 16;  // channels per thread
      const int ch0 = (tid & 15) * CPT;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + (tid >> 4), grow = d.row0 + row;
        if (grow < d.rows) {
          float mt = s_ml[0][row][0];
#pragma unroll
          for (int i = 1; i < kWarps; ++i) mt = fmaxf(mt, s_ml[i][row][0]);
          float lt = 0.f, o[CPT];
#pragma unroll
          for (int e = 0; e < CPT; ++e) o[e] = 0.f;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            const float f = ex2_approx(s_ml[i][row][0] - mt);
            lt = fmaf(s_ml[i][row][1], f, lt);
#pragma unroll
            for (int e = 0; e < CPT; e += 4) {
              const float4 v = *reinterpret_cast<const float4*>(s_part + c4_part_at<D>(i * ROWS + row, (ch0 + e) / 4));
              o[e] = fmaf(v.x, f, o[e]), o[e + 1] = fmaf(v.y, f, o[e + 1]);
              o[e + 2] = fmaf(v.z, f, o[e + 2]), o[e + 3] = fmaf(v.w, f, o[e + 3]);
            }
          }
          const bool tail = d.flags & kOpenStart, open = d.flags & kOpenEnd;
          if (!tail && !open) {
            const int tok = d.tok0 + grow / a.G, head = d.head * a.G + grow % a.G;
            const float inv = lt != 0.f ? 1.f / lt : 0.f;
            uint32_t z[CPT / 2];
#pragma unroll
            for (int e = 0; e < CPT; e += 2) z[e / 2] = c4_pack<F16>(o[e] * inv, o[e + 1] * inv);
            uint16_t* op = a.o + tok * a.ot + head * a.oh + ch0;
            if (CPT == 8) *reinterpret_cast<uint4*>(op) = make_uint4(z[0], z[1], z[CPT / 2 - 2], z[CPT / 2 - 1]);
            else *reinterpret_cast<uint2*>(op) = make_uint2(z[0], z[1]);
            if ((tid & 15) == 0)
              a.lse[static_cast<long long>(tok) * a.Hq + head] =
                  lt != 0.f ? (mt + log2f(lt)) * 0.69314718055994531f : -INFINITY;
          } else {
            const long long at = (static_cast<long long>(blockIdx.x) * 2 + (tail ? 0 : 1)) * ROWS + row;
#pragma unroll
            for (int e = 0; e < CPT; e += 4)
              *reinterpret_cast<float4*>(a.part + at * D + ch0 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            if ((tid & 15) == 0) a.ml[2 * at] = mt, a.ml[2 * at + 1] = lt;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&mempty);
      ++items;
    }
  }
}

// Query rows of an item, from the average request's: up to 16 with the
// warp-level kernel, more in blocks of 32, 64 or 128 on tcgen05. Requests of
// several tokens are ragged and may have twice the average, so they leave the
// warp-level kernel at 8 (32 requests with drafts of 1 to 7 tokens, groups of 4,
// 128 channels: 149 us with blocks of 32, 204 us with blocks of 16).
// One size serves the whole call, and N and R, which the host knows, count
// padding and requests without a new token too. So a call that mixes a long
// prompt with many idle or single-token requests gets blocks that fit neither:
// right, but slower than the two kinds in calls of their own.
int c4_rows(int N, int R, int G) {
  const long long tokens = (static_cast<long long>(N) + R - 1) / R, rows = tokens * G;
  return rows <= 8 ? 8 : rows <= 16 && tokens == 1 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}
int c4_ctas(int rows, int D, int sms) { return (rows == 8 ? (D == 128 ? 3 : 4) : rows == 16 ? 2 : 1) * sms; }

struct C4Ws {
  size_t desc = 0, ml = 0, part = 0, total = 0;
};
// One size for every N and R, so that a workspace serves smaller steps too.
C4Ws c4_ws(int D, int sms) {
  C4Ws w;
  size_t n = 0, rows = 0;
  for (int x = 8; x <= 128; x *= 2) {
    const size_t c = c4_ctas(x, D, sms);
    n = c > n ? c : n;
    rows = c * 2 * x > rows ? c * 2 * x : rows;
  }
  w.desc = sizeof(WsHeader);
  w.ml = align_up(w.desc + n * sizeof(C4Desc), 256);
  w.part = align_up(w.ml + rows * 2 * sizeof(float), 256);
  w.total = align_up(w.part + rows * D * sizeof(float), 256);
  return w;
}

template <int D, bool F16, int NT>
cudaError_t launch(int grid, const C4AttnArgs& a, cudaStream_t st) {
  using C = C4Cfg<D, NT>;
  return launch_and_join<D, F16, C::kRows>(cache4_attn_kernel<D, F16, NT>, grid, kThreads, C::kSmem, a, st);
}

template <int D, bool F16>
cudaError_t launch_rows(int rows, int grid, const C4AttnArgs& a, cudaStream_t st) {
  return rows == 8 ? launch<D, F16, 1>(grid, a, st) : launch<D, F16, 2>(grid, a, st);
}

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" {

size_t scfa_cache4_attn_workspace_size(int N, int R, int Hq, int Hkv, int D) {
  if (N < 1 || R < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return c4_ws(D, num_sms()).total;
}

scfa_status scfa_cache4_attn(const uint16_t* q, long long q_token, long long q_head, const uint8_t* cache,
                             int page_size, int n_pages, const int32_t* table, int max_pages,
                             const int32_t* q_start, const int32_t* vis, int N, int R, int Hq, int Hkv, int D,
                             float scale, int dtype, uint16_t* o, long long o_token, long long o_head, float* lse,
                             void* ws, size_t ws_bytes, unsigned flags, void* stream) {
  if (!q || !cache || !table || !q_start || !vis || !o || !lse || !ws) return SCFA_ERR_INVALID;
  if (N < 1 || R < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || n_pages < 1 || max_pages < 1) return SCFA_ERR_INVALID;
  const float factor = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // to log2 units
  if (!(scale > 0.f && factor < INFINITY)) return SCFA_ERR_INVALID;
  if (dtype != SCFA_DTYPE_BF16 && dtype != SCFA_DTYPE_F16) return SCFA_ERR_UNSUPPORTED;
  if ((D != 64 && D != 128) || !c4_page_size_ok(page_size)) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(n_pages) * page_size >= (1ll << 31) ||
      static_cast<long long>(max_pages) * page_size > kC4MostTokens ||
      static_cast<long long>(N) * Hq >= (1ll << 31) - 256)
    return SCFA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(q), static_cast<const void*>(cache), static_cast<const void*>(o)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SCFA_ERR_INVALID;
  if ((q_token | q_head | o_token | o_head) & 7) return SCFA_ERR_INVALID;
  if (c4_rows_overlap(o_token, o_head, N, Hq, D)) return SCFA_ERR_INVALID;
  const int G = Hq / Hkv, rows = c4_rows(N, R, G), sms = num_sms(), grid = c4_ctas(rows, D, sms);
  const C4Ws w = c4_ws(D, sms);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < w.total) return SCFA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = dtype == SCFA_DTYPE_F16;
  char* p = static_cast<char*>(ws);
  C4AttnArgs a = {};
  a.q = q, a.qt = q_token, a.qh = q_head;
  a.cache = cache, a.page_size = page_size, a.n_pages = n_pages;
  while ((1 << a.log_ps) < page_size) ++a.log_ps;
  a.table = table, a.max_pages = max_pages, a.q_start = q_start, a.vis = vis;
  a.N = N, a.R = R, a.Hq = Hq, a.Hkv = Hkv, a.G = G;
  a.factor = factor;
  a.o = o, a.ot = o_token, a.oh = o_head, a.lse = lse;
  a.status = reinterpret_cast<int*>(p);
  a.desc = reinterpret_cast<C4Desc*>(p + w.desc);
  a.ml = reinterpret_cast<float*>(p + w.ml);
  a.part = reinterpret_cast<float*>(p + w.part);
  a.stall = (flags & SCFA_FLAG_DEBUG_STALL) ? 1 : 0;
  a.k16 = 16u, a.k128 = 128u, a.magic = 0x60006000u;
  const cudaError_t e =
      rows > 16 ? launch_cache4_wide(D, f16, rows, grid, a, st)
      : D == 64 ? (f16 ? launch_rows<64, true>(rows, grid, a, st) : launch_rows<64, false>(rows, grid, a, st))
                : (f16 ? launch_rows<128, true>(rows, grid, a, st) : launch_rows<128, false>(rows, grid, a, st));
  if (e != cudaSuccess) return SCFA_ERR_CUDA;
  if ((flags & SCFA_FLAG_DEBUG_SYNC) && cudaStreamSynchronize(st) != cudaSuccess) return SCFA_ERR_CUDA;
  return SCFA_OK;
}

}  // extern "C"
