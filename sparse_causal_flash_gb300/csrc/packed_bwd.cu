// Attention over packed sequences with shared key heads, backward: dQ, dK and dV from dO.
//
// With P = 2^(s scale log2(e) - lse log2(e)) recomputed from q, k and the forward's lse, delta = rowsum(dO * O),
// dP = dO V^T and dS = P (dP - delta):  dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Three kernels. `packed_stats_kernel` writes -lse log2(e) and -delta of every query row, in rows of query tiles. `packed_dq_kernel` holds a query tile and walks its key tiles (S, dP, dQ: three products a tile);
// `packed_dkv_kernel` holds a key tile and walks the query tiles of all its heads (S^T, dP^T, dV, dK: four). Seven
// products a tile pair where one kernel for all would do five, and no sums in memory: such a kernel has to add its dQ
// tiles into fp32 rows across CTAs (64 KB per tile pair through L2, in an order that changes from run to run, with a
// pass to clear and one to convert), which held the one-kernel backward of the tile-list attention to 820-870 TFLOP/s at
// 128 channels. Here the gradients of heads that share a key head are summed in TMEM and every result is the same bits on
// every run.
//
// P, dS are fp32 up to one rounding to the rows' type for the products that take them; every sum is fp32; scale comes in
// at the end. Rows that lie behind a sequence's last in a tile are masked (bits, so NaN stays out), those among the 16
// rows of the last MMA step zeroed in shared memory where they are summed over.
//
// Both kernels: one CTA per SM, pieces of work from a counter, longest first; warp 0 copies (TMA), warp 1 issues the
// MMAs, warp 2 prepares the scales of dS for fp16, warps 4-7 and 8-11 take 64 columns each of a 128 x 128 tile (thread =
// TMEM lane; with 32 columns a thread in 16 warps the kernels issue a third more instructions: dQ took 539 us instead of
// 460). What chunks of cut pieces leave is joined by a kernel behind both, in the order of the chunks.
//
// Bounded at D = 128 by the tensor cores (79 and 85% busy), at D = 64 by latency inside the softmax. Measured in a graph, one
// call after another: 1,063 us for 8192 tokens of 32 heads over 8 of 128 channels (1,290 TFLOP/s of useful work; dQ 462, dK
// and dV 611, statistics 26 alone), 1,376 us for 16384 of 16 heads over 4 of 64 (1,000). Called on inputs that change from
// call to call the first takes 1,190 us (1,150), under the power cap.
#include <climits>
#include <type_traits>

#include "packed.cuh"

namespace scfa {
namespace {

constexpr int kThreads = 384;
constexpr int kRegsFew = 72, kRegsMany = 216;  // 128 x 72 + 256 x 216 = 384 x 168, what a CTA starts with
constexpr int kSoftWarps = 8;                  // two warpgroups, 64 columns of a tile each
constexpr int kSlots = 3;                      // items known ahead

struct PBwdParams {
  const char* plan;
  long long plan_bytes;
  int N, M, Hq, Hkv, G, tpt;
  float scale, scale_log2;
  const uint16_t *o, *dO, *v;
  long long ot, oh, dot, doh, vt, vh;
  const float* lse;
  uint16_t *dq, *dk, *dv;
  long long dqt, dqh, dkt, dkh, dvt, dvh;
  float* stats;             // [2][tiles][Hkv][128] and, for fp16, lengths of rows
  long long stats_bytes;    // room for them
  int* counter;
  float *part, *part_q;     // chunks' shares of dV and dK, and of dQ
  int stall;
  int* status;
};

__device__ __forceinline__ int bwd_plan_status(const PBwdParams& p) {
  const PackHeader* h = reinterpret_cast<const PackHeader*>(p.plan);
  const int s = pack_plan_status(h, p.plan_bytes, p.N, p.M, p.Hq, p.Hkv);
  if (s != SCFA_OK) return s;
  return pack_stats_bytes(h->n_qtiles, p.M, h->R, p.Hkv) > p.stats_bytes ? SCFA_ERR_WORKSPACE : SCFA_OK;
}

// ------------------------------------------------------------------ fp16: what P and dS are held times
// A weight over n flat keys is 1 / n and dS = P (dP - delta) may be any size, while fp16 has normal numbers from 2^-14 to
// 2^16 only: as they are, weights over 16,384 keys and dS of a dO of 0.001 over 2,000 lose their digits, and a dO of
// thousands leaves infinities. So for fp16 P is held times 2^10 (normal from 2^-24 up; it is at most 1, and room for 2^6
// is left to an lse that is far from zero), and dS times 2^k, with 2^12 <= 2^k |dO| |V| <= 2^13 for the query's own row and
// the longest V row that its piece of work meets (dQ), or for the longest rows of dO and V that meet in a piece (dK, dV).
// |dP - delta| <= 2 |dO| |V|, so dS stays below 2^14, and is normal down to 2^-26 |dO| |V|. Both are powers of two and
// taken out again in fp32. The statistics kernel finds the lengths, squared: of each row of dO, of the longest of eight, and
// of the longest of 16 rows of V. What is not finite counts as nothing there, and spoils what
// it meets in any case. It costs 5 us on the statistics' 14 and 2-3% of the other kernels for 9 texts of 101 to 3501 tokens,
// 12 heads over 4 of 64 channels (233 us in a graph, 219 unscaled), and 1% of all for 8192 tokens, 32 over 8 of 128.
constexpr int kPUp = 10, kDsUp = 13;
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }
// k of the squared lengths a (dO), b (V), each 0 or 2^-48 to 2^39
__device__ __forceinline__ int ds_up(float a, float b) {
  const int e = (__float_as_int(a * b) >> 23) - 127;  // |dO| |V| < 2^((e + 1) / 2)
  return kDsUp - ((e + 2) >> 1);
}
__device__ __forceinline__ float finite_or_zero(float x) { return x < INFINITY ? x : 0.f; }
// The largest of n groups of PER numbers (none negative), group i at base + i * stride; by a whole warp.
template <int PER>
__device__ __forceinline__ float warp_largest(const float* base, long long stride, int n, int lane) {
  constexpr int L = PER / 4;
  float m = 0.f;
  for (int i0 = lane; i0 < n * L; i0 += 4 * 32) {
    float4 x[4];  // (all on their way at once; the last one again where there is none)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(i0 + 32 * j, n * L - 1);
      x[j] = __ldcg(reinterpret_cast<const float4*>(base + (i / L) * stride) + i % L);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) m = pack_max3(m, pack_max3(x[j].x, x[j].y, x[j].z), x[j].w);
  }
  return __int_as_float(static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
}

// ------------------------------------------------------------------ row statistics
// A warp takes eight rows of a tile at a time, a 16-byte piece of O and dO per lane and row, all on their way at once.
// Bounded by HBM: both are read once (26 us for 8192 tokens of 32 heads of 128 channels, 5.2 TB/s).
template <int D, bool F16>
__global__ void __launch_bounds__(256, D == 64 ? 6 : 4) packed_stats_kernel(const __grid_constant__ PBwdParams p) {
  constexpr int L = D / 8, RW = 32 / L, kRows = 8, kSteps = kRows / RW;
  const PackHeader* h = reinterpret_cast<const PackHeader*>(p.plan);
  const int status = bwd_plan_status(p);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = status, p.counter[0] = p.counter[1] = 0;  // for the kernels behind
  if (status != SCFA_OK) return;
  const int4* const tiles = reinterpret_cast<const int4*>(p.plan + h->qtiles);
  const int lane = threadIdx.x & 31, ch = lane % L;
  // (32 bits hold it: each is 64 bytes of the workspace)
  const uint32_t units = static_cast<uint32_t>(h->n_qtiles) * p.Hkv * (kTile / kRows), step = gridDim.x * (blockDim.x / 32);
  const long long n = static_cast<long long>(units) * kRows;
  for (uint32_t unit = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); unit < units; unit += step) {
    const uint32_t pair = unit / (kTile / kRows), tile = pair / p.Hkv;
    const int head = static_cast<int>(pair - tile * p.Hkv);
    const int4 t = __ldg(tiles + tile);
    uint4 a[kSteps], b[kSteps];
    float lse[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = static_cast<int>(unit % (kTile / kRows)) * kRows + i * RW + lane / L;
      const int tok = row / p.G, qh = head * p.G + row - tok * p.G;
      const bool live = tok < t.y;
      a[i] = b[i] = make_uint4(0, 0, 0, 0), lse[i] = -INFINITY;
      if (live) {
        a[i] = *reinterpret_cast<const uint4*>(p.o + static_cast<long long>(t.x + tok) * p.ot + qh * p.oh + ch * 8);
        b[i] = *reinterpret_cast<const uint4*>(p.dO + static_cast<long long>(t.x + tok) * p.dot + qh * p.doh + ch * 8);
        lse[i] = p.lse[static_cast<long long>(t.x + tok) * p.Hq + qh];
      }
    }
    float longest = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t aw[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bw[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
      float s = 0.f, sq = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = c4_unpack<F16>(aw[k]), y = c4_unpack<F16>(bw[k]);
        s = fmaf(x.x, y.x, fmaf(x.y, y.y, s));
        if (F16) sq = fmaf(y.x, y.x, fmaf(y.y, y.y, sq));
      }
#pragma unroll
      for (int o = L / 2; o; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (F16) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      }
      if (F16) sq = lse[i] == -INFINITY ? 0.f : finite_or_zero(sq), longest = fmaxf(longest, sq);
      if (ch == 0) {
        const long long at = static_cast<long long>(unit) * kRows + i * RW + lane / L;
        // a row that sees nothing, or is none, weighs nothing: P = 2^(-inf)
        p.stats[at] = lse[i] == -INFINITY ? -INFINITY : F16 ? fmaf(-lse[i], kPackLog2e, static_cast<float>(kPUp)) : -(lse[i] * kPackLog2e);
        p.stats[n + at] = lse[i] == -INFINITY ? 0.f : -s;
        if (F16) p.stats[2 * n + at] = sq;
      }
    }
    if (F16) {
#pragma unroll
      for (int o = L; o < 32; o <<= 1) longest = fmaxf(longest, __shfl_xor_sync(0xffffffffu, longest, o));
      if (lane == 0) p.stats[3 * n + unit] = longest;
    }
  }
  if (F16) {  // 16 rows of a key tile of V a warp at a time
    constexpr int kVRows = kTile / kVUnits, kVSteps = kVRows / RW;
    const PackEntry* const tiles_v = reinterpret_cast<const PackEntry*>(p.plan + h->entries[kListDkv]);
    float* const big_v = p.stats + 3 * n + units;
    const long long n_v = static_cast<long long>(h->n_entries[kListDkv]) * p.Hkv * kVUnits;
    // (counted from the grid's middle: in small calls by CTAs that have nothing to do above and run at the same time)
    for (long long x = ((blockIdx.x + gridDim.x / 2) % gridDim.x) * (blockDim.x / 32) + (threadIdx.x >> 5); x < n_v; x += step) {
      const int piece = static_cast<int>(x % kVUnits);
      const uint32_t pair = static_cast<uint32_t>(x / kVUnits);  // (entries x heads: below 2^31)
      const PackEntry& e = tiles_v[pair / p.Hkv];
      const int head = static_cast<int>(pair % p.Hkv), n_tok = __ldg(&e.n_tok), k0 = __ldg(&e.k0), diag = __ldg(&e.diag);
      if (__ldg(&e.chunk) != 0) continue;  // (the first chunk does it)
      uint4 a[kVSteps];
#pragma unroll
      for (int i = 0; i < kVSteps; ++i) {
        const int row = piece * kVRows + i * RW + lane / L;
        a[i] = row < n_tok ? *reinterpret_cast<const uint4*>(p.v + static_cast<long long>(k0 + row) * p.vt + head * p.vh + ch * 8) : make_uint4(0, 0, 0, 0);
      }
      float longest = 0.f;
#pragma unroll
      for (int i = 0; i < kVSteps; ++i) {
        const uint32_t aw[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 y = c4_unpack<F16>(aw[k]);
          sq = fmaf(y.x, y.x, fmaf(y.y, y.y, sq));
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        longest = fmaxf(longest, finite_or_zero(sq));
      }
#pragma unroll
      for (int o = L; o < 32; o <<= 1) longest = fmaxf(longest, __shfl_xor_sync(0xffffffffu, longest, o));
      if (lane == 0) big_v[(pack_key_tile(k0 - diag, __ldg(&e.seq), diag / kTile) * p.Hkv + head) * kVUnits + piece] = longest;
    }
  }
  grid_release();
}

// ------------------------------------------------------------------ dQ
// TMEM: S [0,128), dP [128,256), dQ [256,256+D), two buffers of dS at 384 and 448. Products in the order
// dP(j+1) S(j+1) dQ(j): dP of a tile is in registers while its S runs, and there are two products' time to make dS from
// them. V comes first so that K_j, which stays until dQ(j), is needed again late: at D = 128 shared memory holds three K
// tiles, and a fourth product's time for loading the next is what L2 needs.
template <int D>
struct __align__(1024) DqSmem {
  static constexpr int kSubs = D / 64, kQs = D == 64 ? 2 : 1, kKs = D == 64 ? 4 : 3, kVs = D == 64 ? 4 : 2;
  uint8_t q[kQs][kSubs][kPackSub];
  uint8_t dO[kQs][kSubs][kPackSub];
  uint8_t k[kKs][kSubs][kPackSub];
  uint8_t v[kVs][kSubs][kPackSub];
  PackEntry item[kSlots];
  uint64_t q_full[kQs], q_empty[kQs], k_full[kKs], k_empty[kKs], v_full[kVs], v_empty[kVs];
  uint64_t s_full, s_free, dp_full, dp_free, ds_full[2], ds_free[2], dq_full, dq_empty, tail, drain;
  uint64_t item_full[kSlots], item_empty[kSlots], v_known[kSlots];
  float v_longest[kSlots];  // fp16: squared length of the longest V row that the item meets
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
packed_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                 const __grid_constant__ PBwdParams p) {
  using Sm = DqSmem<D>;
  constexpr int kSubs = Sm::kSubs, kQs = Sm::kQs, kKs = Sm::kKs, kVs = Sm::kVs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Nothing here needs the dK / dV kernel: these CTAs come as its CTAs leave, and fill its last round. They end behind it,
  // so that what follows this kernel follows both. What is needed is the statistics kernel's: the dK / dV kernel has waited
  // for its end, and so for its writes in L2, before any of these CTAs could start. A kernel in between promises nothing
  // about L1, so all that comes from there is read past it (__ldcg, and an atomic for the counter).
  grid_release();
  if (bwd_plan_status(p) != SCFA_OK) {  // (the first kernel has said so)
    grid_wait();
    return;
  }
  if (smem_u32(smem_raw) & 1023u) {  // the swizzled tiles need this; all shared memory there is leaves no room to move
    if (threadIdx.x == 0) raise_status(p.status, SCFA_ERR_UNSUPPORTED);
    grid_wait();
    return;
  }
  const PackHeader* const h = reinterpret_cast<const PackHeader*>(p.plan);
  const int window = h->window, n_work = h->n_entries[kListDq] * p.Hkv, used = p.G * p.tpt;
  const long long n_stats = static_cast<long long>(h->n_qtiles) * p.Hkv * kTile;
  PackWork work;
  if (warp == 0) work.first(reinterpret_cast<const PackEntry*>(p.plan + h->entries[kListDq]), n_work, p.Hkv, lane);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQs; ++s) mbar_init(&sm.q_full[s], 1), mbar_init(&sm.q_empty[s], 1);
    for (int s = 0; s < kKs; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], 1);
    for (int s = 0; s < kVs; ++s) mbar_init(&sm.v_full[s], 1), mbar_init(&sm.v_empty[s], 1);
    mbar_init(&sm.s_full, 1), mbar_init(&sm.s_free, kSoftWarps), mbar_init(&sm.ds_full[0], kSoftWarps);
    mbar_init(&sm.ds_full[1], kSoftWarps), mbar_init(&sm.dp_full, 1), mbar_init(&sm.dp_free, kSoftWarps);
    mbar_init(&sm.ds_free[0], 1), mbar_init(&sm.ds_free[1], 1);
    mbar_init(&sm.dq_full, 1), mbar_init(&sm.dq_empty, kSoftWarps), mbar_init(&sm.tail, 1), mbar_init(&sm.drain, 1);
    for (int s = 0; s < kSlots; ++s)
      mbar_init(&sm.item_full[s], 1), mbar_init(&sm.item_empty[s], 1 + kSoftWarps + (F16 ? 1 : 0)), mbar_init(&sm.v_known[s], 1);
    sm.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_v), tma_prefetch_desc(&tm_do);
  }
  if (used < kTile) {  // rows that no copy writes: zero for good
    for (int s = 0; s < kQs; ++s) {
      zero_tile_rows(sm.q[s][0], kSubs, used, kTile, threadIdx.x, kThreads);
      zero_tile_rows(sm.dO[s][0], kSubs, used, kTile, threadIdx.x, kThreads);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* const abort_flag = &sm.abort_flag;

  if (warp < 4) {
    regs_release<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      int q_it = 0, k_it = 0, v_it = 0, tails = 0, unmarked = -1;  // unmarked: K tile whose zeros an abort kept from being written
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % kSlots;
        ok = warp_wait(&sm.item_empty[slot], ((it / kSlots) & 1) ^ 1, abort_flag, p.status);
        if (!ok || !work.publish(&sm.item[slot], &sm.item_full[slot], lane)) break;
        const PackEntry& e = sm.item[slot];
        const int head = e.head, a = e.a, b = e.b;
        if (a == b) {
          work.next(p.counter, lane);
          continue;
        }
        if (p.stall && k_it == 0) break;  // debug stall: no load ever arrives
        {
          const int s = q_it % kQs;
          ok = warp_wait(&sm.q_empty[s], ((q_it / kQs) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.q_full[s], 2 * D * used * 2);
            for (int sub = 0; sub < kSubs; ++sub) {
              tma_load_3d(sm.q[s][sub], &tm_q, &sm.q_full[s], sub * 64, head * p.G, e.q0);
              tma_load_3d(sm.dO[s][sub], &tm_do, &sm.q_full[s], sub * 64, head * p.G, e.q0);
            }
          }
          ++q_it;
        }
        for (int j = a; j < b && ok; ++j) {
          const int valid = e.m - j * kTile;
          const bool cut = valid < kTile && (valid & 15) != 0;
          const int s = k_it % kKs, vs = v_it % kVs;
          ok = warp_wait(&sm.v_empty[vs], ((v_it / kVs) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.v_full[vs], D * kTile * 2);
            for (int sub = 0; sub < kSubs; ++sub) tma_load_3d(sm.v[vs][sub], &tm_v, &sm.v_full[vs], sub * 64, head, e.k0 + j * kTile);
          }
          ++v_it;
          ok = warp_wait(&sm.k_empty[s], ((k_it / kKs) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          if (lane == 0) {
            uint64_t* const kb = cut ? &sm.tail : &sm.k_full[s];
            mbar_arrive_expect_tx(kb, D * kTile * 2);
            for (int sub = 0; sub < kSubs; ++sub) tma_load_3d(sm.k[s][sub], &tm_k, kb, sub * 64, head, e.k0 + j * kTile);
          }
          ++k_it;
          if (cut) {
            ok = warp_wait(&sm.tail, tails & 1, abort_flag, p.status);
            ++tails;
            if (!ok) {
              unmarked = k_it - 1;
              break;
            }
            zero_tile_rows(sm.k[s][0], kSubs, valid, (valid + 15) & ~15, lane, 32);
            fence_proxy_async_smem();
            warp_arrive(&sm.k_full[s]);
          }
          if (j == a) work.next(p.counter, lane);  // (under the loads)
        }
      }
      if (lane == 0) {
        // every copy issued has landed before the CTA exits, also after an abort
        if (tails > 0) mbar_wait_drain(&sm.tail, (tails - 1) & 1, p.status);
        for (int d = 1; d <= kKs && d <= k_it; ++d)
          if (k_it - d != unmarked) mbar_wait_drain(&sm.k_full[(k_it - d) % kKs], ((k_it - d) / kKs) & 1, p.status);
        for (int d = 1; d <= kVs && d <= v_it; ++d) mbar_wait_drain(&sm.v_full[(v_it - d) % kVs], ((v_it - d) / kVs) & 1, p.status);
        for (int d = 1; d <= kQs && d <= q_it; ++d) mbar_wait_drain(&sm.q_full[(q_it - d) % kQs], ((q_it - d) / kQs) & 1, p.status);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t idesc_s = pack_idesc<F16>(kTile, kTile, 0, 0), idesc_q = pack_idesc<F16>(kTile, D, 0, 1);
        constexpr uint32_t kTile16 = (kSubs * kPackSub) >> 4;
        const uint32_t qd = desc_low(smem_u32(sm.q[0][0]), 16), dod = desc_low(smem_u32(sm.dO[0][0]), 16);
        const uint32_t kd = desc_low(smem_u32(sm.k[0][0]), 16), vd = desc_low(smem_u32(sm.v[0][0]), 16);
        const uint32_t kn = desc_low(smem_u32(sm.k[0][0]), kPackSub);
        int q_it = 0, kv = 0, n_q = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
          const int slot = it % kSlots;
          if (!mbar_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
          if (sm.item[slot].head < 0) break;
          const int a = sm.item[slot].a, b = sm.item[slot].b, m_keys = sm.item[slot].m;
          if (a < b) {
            const int qs = q_it % kQs;
            auto do_s = [&](int i) -> bool {  // S of key tile number i
              const int s = i % kKs;
              if (i > 0 && !mbar_wait(&sm.s_free, (i - 1) & 1, abort_flag, p.status)) return false;
              if (!mbar_wait(&sm.k_full[s], (i / kKs) & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              mma_ss_steps<0, D / 16>(tmem, qd + qs * kTile16, kd + s * kTile16, idesc_s, false);
              tc_commit(&sm.s_full);
              return true;
            };
            auto do_dp = [&](int i) -> bool {
              const int s = i % kVs;
              if (i > 0 && !mbar_wait(&sm.dp_free, (i - 1) & 1, abort_flag, p.status)) return false;
              if (!mbar_wait(&sm.v_full[s], (i / kVs) & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              mma_ss_steps<0, D / 16>(tmem + 128, dod + qs * kTile16, vd + s * kTile16, idesc_s, false);
              tc_commit(&sm.dp_full);
              tc_commit(&sm.v_empty[s]);
              return true;
            };
            auto do_dq = [&](int i, int j) -> bool {
              if (j == a && !mbar_wait(&sm.dq_empty, (n_q & 1) ^ 1, abort_flag, p.status)) return false;
              if (!mbar_wait(&sm.ds_full[i & 1], (i >> 1) & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              const uint32_t ds = tmem + 384u + 64u * (i & 1), bk = kn + (i % kKs) * kTile16;
              const int steps = min(kTile / 16, (m_keys - j * kTile + 15) >> 4);
              if (steps == 8) mma_ts_steps<0, 8>(tmem + 256, ds, bk, idesc_q, j > a, 8);
              else mma_ts_steps<0, 8>(tmem + 256, ds, bk, idesc_q, j > a, steps);
              tc_commit(&sm.k_empty[i % kKs]);
              tc_commit(&sm.ds_free[i & 1]);
              return true;
            };
            ok = mbar_wait(&sm.q_full[qs], (q_it / kQs) & 1, abort_flag, p.status) && do_dp(kv) && do_s(kv);
            for (int j = a; j < b && ok; ++j, ++kv) {
              if (j + 1 < b) ok = do_dp(kv + 1) && do_s(kv + 1);
              else tc_commit(&sm.q_empty[qs]);
              if (ok) ok = do_dq(kv, j);
            }
            if (!ok) break;
            tc_commit(&sm.dq_full);
            ++n_q, ++q_it;
          }
          mbar_arrive(&sm.item_empty[slot]);
        }
        tc_commit(&sm.drain);
        mbar_wait_drain(&sm.drain, 0, p.status);
      }
    } else if (F16 && warp == 2) {
      // ---------------------------------------------------------- the longest V rows, ahead of the softmax
      const float* const big_v = p.stats + 3 * n_stats + n_stats / (kTile / kDoUnits);
      for (int it = 0;; ++it) {
        const int slot = it % kSlots;
        if (!warp_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
        const PackEntry& e = sm.item[slot];
        if (e.head < 0) break;
        const float v2 = warp_largest<kVUnits>(big_v + (pack_key_tile(e.k0, e.seq, e.a) * p.Hkv + e.head) * kVUnits,
                                               static_cast<long long>(p.Hkv) * kVUnits, e.b - e.a, lane);
        if (lane == 0) sm.v_longest[slot] = v2;
        warp_arrive(&sm.v_known[slot]);
        warp_arrive(&sm.item_empty[slot]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_take<kRegsMany>();
    const int wg = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane, col0 = wg * 64;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int r_tok = r / p.G;
    int n = 0, n_q = 0;
    for (int it = 0;; ++it) {
      const int slot = it % kSlots;
      if (!warp_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
      const PackEntry& e = sm.item[slot];
      const int head = e.head;
      if (head < 0) break;
      const int a = e.a, b = e.b, first = e.diag, n_tok = e.n_tok;
      const bool valid = r_tok < n_tok;
      const int hi = valid ? first + r_tok : -1;
      const long long at = (static_cast<long long>(e.tile0) * p.Hkv + head) * kTile + r;
      float nl = __ldcg(p.stats + at), down = 1.f;
      const float nd = __ldcg(p.stats + n_stats + at);
      if (F16) {  // dS is held times 2^k = 1 / down: a row's own, in its exponent, from which P's 2^10 is taken again
        const float o2 = __ldcg(p.stats + 2 * n_stats + at);
        if (!warp_wait(&sm.v_known[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
        const int k = ds_up(o2, sm.v_longest[slot]);
        nl += static_cast<float>(k - kPUp), down = pow2(-k);
      }
      auto tile = [&](auto may_mask, bool masked, int j) -> bool {
        uint32_t sr[64], dr[64];
        if (!warp_wait(&sm.dp_full, n & 1, abort_flag, p.status)) return false;
        tc_fence_after();
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) tmem_ld32(lanes + 128 + col0 + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&dr[cc * 32]));
        tmem_wait_ld();
        tmem_ld_fence(dr);
        tc_fence_before();
        warp_arrive(&sm.dp_free);
        if (!warp_wait(&sm.s_full, n & 1, abort_flag, p.status)) return false;
        tc_fence_after();
        uint32_t pk[32];
        auto weigh = [&](int from, int to) {
          const uint64_t sl2 = f2(p.scale_log2, p.scale_log2), nl2 = f2(nl, nl), nd2 = f2(nd, nd);
#pragma unroll
          for (int c = from; c < to; c += 2) {
            float x0, x1;
            f2_split(fma2(f2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl2, nl2), x0, x1);
            x0 = ex2_approx(x0), x1 = ex2_approx(x1);
            f2_split(mul2(f2(x0, x1), add2(f2(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1])), nd2)), x0, x1);
            pk[c >> 1] = c4_pack<F16>(x0, x1);
          }
        };
        uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
        uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
        tmem_ld32(lanes + col0, s0);
        if (D == 64) {  // the other half of S comes under the first half's exponentials (651 -> 605 us at 16384 tokens, 16 heads
          tmem_wait_ld();  // over 4; at D = 128, where the MMAs wait for these columns, 447 -> 467 us at 8192, 32 over 8)
          tmem_ld_fence(s0);
          tmem_ld32(lanes + col0 + 32, s1);
          weigh(0, 32);
          tmem_wait_ld();
          tmem_ld_fence(s1);
          tc_fence_before();
          warp_arrive(&sm.s_free);
          weigh(32, 64);
        } else {
          tmem_ld32(lanes + col0 + 32, s1);
          tmem_wait_ld();
          tmem_ld_fence(sr);
          tc_fence_before();
          warp_arrive(&sm.s_free);
          weigh(0, 64);
        }
        if (decltype(may_mask)::value && masked) {  // columns lo .. lim are seen
          const int lim = hi - j * kTile - col0, lo = window ? lim - window + 1 : 0;
          const uint32_t bits[2] = {bit_range(lo, lim + 1), bit_range(lo - 32, lim + 1 - 32)};
#pragma unroll
          for (int c = 0; c < 64; c += 2) pk[c >> 1] &= bit_pair(bits[c >> 5], c & 31);
        }
        if (n > 1) {  // dQ two tiles back has read this buffer
          if (!warp_wait(&sm.ds_free[n & 1], ((n >> 1) - 1) & 1, abort_flag, p.status)) return false;
          tc_fence_after();
        }
        tmem_st32(lanes + 384u + 64u * (n & 1) + wg * 32, pk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&sm.ds_full[n & 1]);  // (two: at D = 64 a warp may be a whole tile ahead of another)
        ++n;
        return true;
      };
      // tiles [plain, masked) are seen whole by every row, as in the forward
      const int plain = window ? min(b, max(a, (first + n_tok - window + kTile - 1) / kTile)) : a;
      const int masked = max(plain, min(b, max(0, first + 1) / kTile));
      bool ok = true;
      if (D == 64) {  // (one copy of the code or two: as in the forward)
        for (int j = a; j < b && ok; ++j) ok = tile(std::true_type{}, j < plain || j >= masked, j);
      } else {
        int j = a;
        for (int part = 0; part < 2 && ok; ++part) {
          const int stop = part ? b : plain;
          for (; j < stop && ok; ++j) ok = tile(std::true_type{}, true, j);
          if (part == 0)
            for (; j < masked && ok; ++j) ok = tile(std::false_type{}, false, j);
        }
      }
      if (!ok) break;
      // this warp's 16 rows of dQ
      const int row = quarter * 32 + wg * 16 + (lane >> 2);
      const uint32_t from = lanes + 256 + (static_cast<uint32_t>(wg * 16) << 16);
      if (a < b) {
        if (!warp_wait(&sm.dq_full, n_q & 1, abort_flag, p.status)) break;
        tc_fence_after();
        ++n_q;
      }
      // (16 rows a warp: all columns at once; in quad_blocks' loop the kernel took 464 us instead of 453, 8192 tokens, 32
      // heads over 8 of 128 channels)
      uint32_t acc[D / 32][16];
      quad_part<D>(from, a < b, acc);
      if (a < b) {
        tc_fence_before();
        warp_arrive(&sm.dq_empty);
      }
      float f[2] = {1.f, 1.f};
      if (F16) {
#pragma unroll
        for (int u = 0; u < 2; ++u) f[u] = __shfl_sync(0xffffffffu, down, (row + 8 * u) & 31);
      }
      if (e.slot >= 0) {  // this chunk's share, for the join behind this kernel
        float* const mine = p.part_q + (static_cast<long long>(e.slot + e.chunk) * p.Hkv + head) * kTile * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) leave_part<D, F16>(mine + c, acc[c / 32], row, f);
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tk = (row + 8 * u) / p.G, qh = head * p.G + row + 8 * u - tk * p.G;
          uint16_t* const to = p.dq + static_cast<long long>(e.q0 + tk) * p.dqt + qh * p.dqh;
#pragma unroll
          for (int c = 0; c < D; c += 32) quad_store<F16>(to + c, tk < n_tok, acc[c / 32], u, p.scale * f[u]);
        }
      }
      warp_arrive(&sm.item_empty[slot]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  grid_wait();
}

// ------------------------------------------------------------------ dK and dV
// Eight MMA steps of 16 queries whose A lies four steps (32 columns) to every 64 columns; `steps` of them hold something.
template <int KK>
__device__ __forceinline__ void mma_half_steps(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool add_to, int steps) {
  if constexpr (KK < 8) {
    if (KK < steps) mma_ts_at<(KK >> 2) * 64 + (KK & 3) * 8, KK * 128>(d_tmem, a_tmem, b_low, idesc, KK > 0 || add_to ? 1u : 0u);
    mma_half_steps<KK + 1>(d_tmem, a_tmem, b_low, idesc, add_to, steps);
  }
}

// Tiles are transposed: lanes are keys, columns queries.
// D = 128: scores take turns in two regions of 128 TMEM columns (dV and dK take the rest): S^T(t) in one, and a warpgroup
// writes P^T and dS^T of its 64 queries over its own 64 columns of it; dP^T(t) in the other, free again once it is in
// registers. Products come in the order dP(t) dV(t) S(t+1) dK(t), which gives the softmax two products' time (1,024 cycles)
// for P behind S and for dS behind dP, and the tensor cores work without a pause.
// D = 64: products take half the time, the softmax the same. S^T, dP^T, P^T and dS^T have columns of their own: S(t+1) and
// dP(t+1) run while P(t) and dS(t) are made, in one go, so that exponentials and products share their cycles (made one
// after another the kernel took 904 us instead of 832 at 16384 tokens, 16 heads over 4).
template <int D>
struct __align__(1024) DkvSmem {
  static constexpr int kSubs = D / 64, kQs = D == 64 ? 4 : 3, kOs = D == 64 ? 4 : 2, kKs = D == 64 ? 2 : 1;
  uint8_t k[kKs][kSubs][kPackSub];
  uint8_t v[kKs][kSubs][kPackSub];
  uint8_t q[kQs][kSubs][kPackSub];
  uint8_t dO[kOs][kSubs][kPackSub];
  static constexpr int kStatStages = D == 64 ? 4 : 2;  // (all that fits at D = 128)
  alignas(16) float nl[kStatStages][kTile];
  alignas(16) float nd[kStatStages][kTile];
  PackEntry item[kSlots];
  uint64_t k_full[kKs], k_empty[kKs], q_full[kQs], q_empty[kQs], do_full[kOs], do_empty[kOs];
  uint64_t st_full[kStatStages], st_empty[kStatStages], st_raw[kStatStages];
  uint64_t s_full, s_free, dp_full, dp_free, p_full, ds_full, pd_free, acc_full, acc_empty, tail[2], drain;
  uint64_t item_full[kSlots], item_empty[kSlots], up_known[kSlots];
  int up[kSlots];  // fp16: k of the item
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
packed_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                  const __grid_constant__ PBwdParams p) {
  using Sm = DkvSmem<D>;
  constexpr int kSubs = Sm::kSubs, kQs = Sm::kQs, kOs = Sm::kOs, kKs = Sm::kKs, kStatStages = Sm::kStatStages;
  constexpr bool kOwn = D == 64;
  constexpr uint32_t colDV = 512 - 2 * D, colDK = 512 - D;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();     // the rows' statistics are there,
  grid_release();  // also for the dQ kernel, whose CTAs may come from now on
  if (bwd_plan_status(p) != SCFA_OK) return;  // (the first kernel has said so)
  if (smem_u32(smem_raw) & 1023u) {  // the swizzled tiles need this; all shared memory there is leaves no room to move
    if (threadIdx.x == 0) raise_status(p.status, SCFA_ERR_UNSUPPORTED);
    return;
  }
  const PackHeader* const h = reinterpret_cast<const PackHeader*>(p.plan);
  const int window = h->window, n_work = h->n_entries[kListDkv] * p.Hkv, used = p.G * p.tpt;
  const long long n_stats = static_cast<long long>(h->n_qtiles) * p.Hkv * kTile;
  PackWork work;
  if (warp == 0) work.first(reinterpret_cast<const PackEntry*>(p.plan + h->entries[kListDkv]), n_work, p.Hkv, lane);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKs; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], 1);
    for (int s = 0; s < kQs; ++s) mbar_init(&sm.q_full[s], 1), mbar_init(&sm.q_empty[s], 1);
    for (int s = 0; s < kOs; ++s) mbar_init(&sm.do_full[s], 1), mbar_init(&sm.do_empty[s], 1);
    for (int s = 0; s < kStatStages; ++s) mbar_init(&sm.st_full[s], 1), mbar_init(&sm.st_raw[s], 1), mbar_init(&sm.st_empty[s], kSoftWarps);
    mbar_init(&sm.s_full, 1), mbar_init(&sm.s_free, kSoftWarps), mbar_init(&sm.dp_full, 1), mbar_init(&sm.dp_free, kSoftWarps);
    mbar_init(&sm.p_full, kSoftWarps), mbar_init(&sm.ds_full, kSoftWarps), mbar_init(&sm.pd_free, 1);
    mbar_init(&sm.acc_full, 1), mbar_init(&sm.acc_empty, kSoftWarps);
    mbar_init(&sm.tail[0], 1), mbar_init(&sm.tail[1], 1), mbar_init(&sm.drain, 1);
    for (int s = 0; s < kSlots; ++s)
      mbar_init(&sm.item_full[s], 1), mbar_init(&sm.item_empty[s], 1 + kSoftWarps + (F16 ? 1 : 0)), mbar_init(&sm.up_known[s], 1);
    sm.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_v), tma_prefetch_desc(&tm_do);
  }
  if (used < kTile) {  // rows that no copy writes: zero for good
    for (int s = 0; s < kQs; ++s) zero_tile_rows(sm.q[s][0], kSubs, used, kTile, threadIdx.x, kThreads);
    for (int s = 0; s < kOs; ++s) zero_tile_rows(sm.dO[s][0], kSubs, used, kTile, threadIdx.x, kThreads);
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* const abort_flag = &sm.abort_flag;

  if (warp < 4) {
    regs_release<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      int k_it = 0, q_it = 0, do_it = 0, st_it = 0, tails[2] = {0, 0}, unmarked[2] = {-1, -1};
      uint64_t* const st_land = F16 ? sm.st_raw : sm.st_full;
      bool ok = true;
      // Q or dO tile of query tile i into its ring. Rows behind the sequence's last, up to the last MMA step's end, become
      // zero, and those of queries that see nothing (before the first key): their P and dS are zero, 0 x NaN is not
      auto load = [&](int which, const CUtensorMap* map, uint8_t (*ring)[kSubs][kPackSub], uint64_t* full, uint64_t* empty, int& n, int stages,
                      int head, const PackEntry& e, int i, int blind) -> bool {
        const int s = n % stages, rows = min(p.tpt, e.m - i * p.tpt) * p.G;
        const bool cut = (rows < used && (rows & 15) != 0) || blind > 0;
        if (!warp_wait(&empty[s], ((n / stages) & 1) ^ 1, abort_flag, p.status)) return false;
        if (lane == 0) {
          uint64_t* const bar = cut ? &sm.tail[which] : &full[s];
          mbar_arrive_expect_tx(bar, D * used * 2);
          for (int sub = 0; sub < kSubs; ++sub) tma_load_3d(ring[s][sub], map, bar, sub * 64, head * p.G, e.q0 + i * p.tpt);
        }
        ++n;
        if (cut) {
          const bool got = warp_wait(&sm.tail[which], tails[which] & 1, abort_flag, p.status);
          ++tails[which];
          if (!got) {
            unmarked[which] = n - 1;
            return false;
          }
#pragma unroll 1
          for (int part = 0; part < 2; ++part) zero_tile_rows(ring[s][0], kSubs, part ? 0 : rows, part ? blind : (rows + 15) & ~15, lane, 32);
          fence_proxy_async_smem();
          warp_arrive(&full[s]);
        }
        return true;
      };
      for (int it = 0; ok; ++it) {
        const int slot = it % kSlots;
        ok = warp_wait(&sm.item_empty[slot], ((it / kSlots) & 1) ^ 1, abort_flag, p.status);
        if (!ok || !work.publish(&sm.item[slot], &sm.item_full[slot], lane)) break;
        const PackEntry& e = sm.item[slot];
        const int head = e.head, a = e.a, b = e.b;
        if (a == b) {
          work.next(p.counter, lane);
          continue;
        }
        if (p.stall && k_it == 0) break;  // debug stall: no load ever arrives
        {
          const int s = k_it % kKs;
          ok = warp_wait(&sm.k_empty[s], ((k_it / kKs) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.k_full[s], 2 * D * kTile * 2);
            for (int sub = 0; sub < kSubs; ++sub) {
              tma_load_3d(sm.v[s][sub], &tm_v, &sm.k_full[s], sub * 64, head, e.k0);
              tma_load_3d(sm.k[s][sub], &tm_k, &sm.k_full[s], sub * 64, head, e.k0);
            }
          }
          ++k_it;
        }
        int blind = max(-e.shift - a * p.tpt, 0) * p.G;  // (a piece's first tile alone may have such rows)
        for (int i = a; i < b && ok; ++i, blind = 0) {
          ok = load(0, &tm_q, sm.q, sm.q_full, sm.q_empty, q_it, kQs, head, e, i, blind);
          if (!ok) break;
          ok = load(1, &tm_do, sm.dO, sm.do_full, sm.do_empty, do_it, kOs, head, e, i, blind);
          if (!ok) break;
          const int s = st_it % kStatStages;
          ok = warp_wait(&sm.st_empty[s], ((st_it / kStatStages) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          if (lane == 0) {
            const float* const st = p.stats + (static_cast<long long>(e.tile0 + i) * p.Hkv + head) * kTile;
            mbar_arrive_expect_tx(&st_land[s], 2 * kTile * 4);
            bulk_load(sm.nl[s], st, kTile * 4, &st_land[s]);
            bulk_load(sm.nd[s], st + n_stats, kTile * 4, &st_land[s]);
          }
          ++st_it;
          if (i == a) work.next(p.counter, lane);  // (under the loads)
        }
      }
      if (lane == 0) {
        // every copy issued has landed before the CTA exits, also after an abort
        for (int x = 0; x < 2; ++x)
          if (tails[x] > 0) mbar_wait_drain(&sm.tail[x], (tails[x] - 1) & 1, p.status);
        for (int d = 1; d <= kQs && d <= q_it; ++d)
          if (q_it - d != unmarked[0]) mbar_wait_drain(&sm.q_full[(q_it - d) % kQs], ((q_it - d) / kQs) & 1, p.status);
        for (int d = 1; d <= kOs && d <= do_it; ++d)
          if (do_it - d != unmarked[1]) mbar_wait_drain(&sm.do_full[(do_it - d) % kOs], ((do_it - d) / kOs) & 1, p.status);
        for (int d = 1; d <= kStatStages && d <= st_it; ++d)
          mbar_wait_drain(&st_land[(st_it - d) % kStatStages], ((st_it - d) / kStatStages) & 1, p.status);
        for (int d = 1; d <= kKs && d <= k_it; ++d) mbar_wait_drain(&sm.k_full[(k_it - d) % kKs], ((k_it - d) / kKs) & 1, p.status);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t idesc_s = pack_idesc<F16>(kTile, kTile, 0, 0), idesc_a = pack_idesc<F16>(kTile, D, 0, 1);
        constexpr uint32_t kTile16 = (kSubs * kPackSub) >> 4;
        const uint32_t kd = desc_low(smem_u32(sm.k[0][0]), 16), vd = desc_low(smem_u32(sm.v[0][0]), 16);
        const uint32_t qd = desc_low(smem_u32(sm.q[0][0]), 16), dod = desc_low(smem_u32(sm.dO[0][0]), 16);
        const uint32_t qn = desc_low(smem_u32(sm.q[0][0]), kPackSub), don = desc_low(smem_u32(sm.dO[0][0]), kPackSub);
        int k_it = 0, t = 0, n_acc = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
          const int slot = it % kSlots;
          if (!mbar_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
          if (sm.item[slot].head < 0) break;
          const int a = sm.item[slot].a, b = sm.item[slot].b, m_tok = sm.item[slot].m;
          if (a < b) {
            const int ks = k_it % kKs;
            // t: query tile number over the CTA's whole work
            auto s_at = [&](int n) { return tmem + (kOwn ? 0u : 128u * (n & 1)); };
            auto dp_at = [&](int n) { return tmem + (kOwn ? 128u : 128u * ((n & 1) ^ 1)); };
            auto do_s = [&](int n) -> bool {
              // (own columns: once S and dP of the tile before are in registers. Two regions: where dP of it was)
              if (n > 0 && !mbar_wait(kOwn ? &sm.s_free : &sm.dp_free, (n - 1) & 1, abort_flag, p.status)) return false;
              if (!mbar_wait(&sm.q_full[n % kQs], (n / kQs) & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              mma_ss_steps<0, D / 16>(s_at(n), kd + ks * kTile16, qd + (n % kQs) * kTile16, idesc_s, false);
              if (!kOwn) tc_commit(&sm.s_full);
              return true;
            };
            auto do_dp = [&](int n) -> bool {  // (two regions: P and dS that were there are behind dV and dK issued already)
              if (!mbar_wait(&sm.do_full[n % kOs], (n / kOs) & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              mma_ss_steps<0, D / 16>(dp_at(n), vd + ks * kTile16, dod + (n % kOs) * kTile16, idesc_s, false);
              tc_commit(kOwn ? &sm.s_full : &sm.dp_full);
              return true;
            };
            // dV += P^T dO, dK += dS^T Q
            auto do_dv = [&](int n, int i, int steps) -> bool {
              if (i == a && !mbar_wait(&sm.acc_empty, (n_acc & 1) ^ 1, abort_flag, p.status)) return false;
              if (!mbar_wait(&sm.p_full, n & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              if (kOwn) mma_ts_steps<0, 8>(tmem + colDV, tmem + 256, don + (n % kOs) * kTile16, idesc_a, i > a, steps);
              else mma_half_steps<0>(tmem + colDV, s_at(n), don + (n % kOs) * kTile16, idesc_a, i > a, steps);
              tc_commit(&sm.do_empty[n % kOs]);
              return true;
            };
            auto do_dk = [&](int n, int i, int steps) -> bool {
              if (!kOwn && !mbar_wait(&sm.ds_full, n & 1, abort_flag, p.status)) return false;
              tc_fence_after();
              if (kOwn) mma_ts_steps<0, 8>(tmem + colDK, tmem + 320, qn + (n % kQs) * kTile16, idesc_a, i > a, steps);
              else mma_half_steps<0>(tmem + colDK, s_at(n) + 32, qn + (n % kQs) * kTile16, idesc_a, i > a, steps);
              tc_commit(&sm.q_empty[n % kQs]);
              if (kOwn) tc_commit(&sm.pd_free);
              return true;
            };
            ok = mbar_wait(&sm.k_full[ks], (k_it / kKs) & 1, abort_flag, p.status) && do_s(t);
            if (kOwn) ok = ok && do_dp(t);
            for (int i = a; i < b && ok; ++i, ++t) {
              const bool next = i + 1 < b;
              const int steps = min(kTile / 16, (min(p.tpt, m_tok - i * p.tpt) * p.G + 15) >> 4);
              if (kOwn) {
                if (next) ok = do_s(t + 1) && do_dp(t + 1);
                ok = ok && do_dv(t, i, steps) && do_dk(t, i, steps);
              } else {
                ok = do_dp(t) && do_dv(t, i, steps);
                if (next) ok = ok && do_s(t + 1);
                ok = ok && do_dk(t, i, steps);
              }
            }
            if (!ok) break;
            tc_commit(&sm.acc_full);
            tc_commit(&sm.k_empty[ks]);
            ++n_acc, ++k_it;
          }
          mbar_arrive(&sm.item_empty[slot]);
        }
        tc_commit(&sm.drain);
        mbar_wait_drain(&sm.drain, 0, p.status);
      }
    } else if (F16 && warp == 2) {
      // ---------------------------------------------------------- what dS is held times, and -delta times that, ahead of the
      // softmax (which did both by itself at first: 244 us instead of 219 unscaled for 9 texts of 101 to 3501 tokens, 12 heads
      // over 4 of 64 channels)
      const float* const big_do = p.stats + 3 * n_stats;
      const float* const big_v = big_do + n_stats / (kTile / kDoUnits);
      int t = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % kSlots;
        if (!warp_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
        const PackEntry& e = sm.item[slot];
        if (e.head < 0) break;
        // (a key tile's numbers come together with the first of the queries')
        const float v = __ldcg(big_v + (pack_key_tile(e.k0 - e.diag, e.seq, e.diag / kTile) * p.Hkv + e.head) * kVUnits + lane % kVUnits);
        const float o2 = warp_largest<kDoUnits>(big_do + (static_cast<long long>(e.tile0 + e.a) * p.Hkv + e.head) * kDoUnits,
                                                static_cast<long long>(p.Hkv) * kDoUnits, e.b - e.a, lane);
        const float v2 = __int_as_float(static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(v))));
        const int k = ds_up(o2, v2);
        const float up = pow2(k - kPUp);
        if (lane == 0) sm.up[slot] = k;
        warp_arrive(&sm.up_known[slot]);
        for (int i = e.a; i < e.b && ok; ++i, ++t) {
          const int ss = t % kStatStages;
          ok = warp_wait(&sm.st_raw[ss], (t / kStatStages) & 1, abort_flag, p.status);
          if (!ok) break;
          float4& d = *reinterpret_cast<float4*>(&sm.nd[ss][4 * lane]);
          d.x *= up, d.y *= up, d.z *= up, d.w *= up;
          fence_proxy_async_smem();  // (the next copy writes there)
          warp_arrive(&sm.st_full[ss]);
        }
        warp_arrive(&sm.item_empty[slot]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_take<kRegsMany>();
    const int wg = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane, col0 = wg * 64;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int t = 0, n_acc = 0;
    uint32_t s_col = col0;  // this warpgroup's columns of S (two regions in turn at D = 128)
    for (int it = 0;; ++it) {
      const int slot = it % kSlots;
      if (!warp_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
      const PackEntry& e = sm.item[slot];
      const int head = e.head;
      if (head < 0) break;
      const int a = e.a, b = e.b, n_tok = e.n_tok, key = e.diag + r;
      float up = 1.f, down = 1.f;  // fp16: dS is held times 2^k = 1 / down, P times 2^10
      if (F16) {
        if (!warp_wait(&sm.up_known[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
        const int k = sm.up[slot];
        up = pow2(k - kPUp), down = pow2(-k);
      }
      auto tile = [&](auto may_mask, bool masked, int i) -> bool {
        const int ss = t % kStatStages;
        const uint32_t s_at = lanes + s_col, dp_at = lanes + (s_col ^ 128u);
        // P and dS of the queries that see this thread's key: those of tokens from .. to - 1 of the tile
        auto keep = [&](uint32_t (&w)[32]) {
          const long long ahead = static_cast<long long>(key) - e.shift - static_cast<long long>(i) * p.tpt;
          const long long n_left = min(p.tpt, e.m - i * p.tpt);
          const int from = static_cast<int>(max(0ll, min(n_left, ahead))) * p.G - col0;
          const int to = static_cast<int>(window ? max(0ll, min(n_left, ahead + window)) : n_left) * p.G - col0;
          const uint32_t bits[2] = {bit_range(from, to), bit_range(from - 32, to - 32)};
#pragma unroll
          for (int c = 0; c < 64; c += 2) w[c >> 1] &= bit_pair(bits[c >> 5], c & 31);
        };
        const uint64_t sl2 = f2(p.scale_log2, p.scale_log2), up2 = f2(up, up);
        // dP - delta, for fp16 times up (and so is -delta in nd)
        auto centred = [&](uint32_t x0, uint32_t x1, float d0, float d1) {
          const uint64_t x = f2(__uint_as_float(x0), __uint_as_float(x1)), d = f2(d0, d1);
          return F16 ? fma2(x, up2, d) : add2(x, d);
        };
        if constexpr (kOwn) {
          uint32_t x[64], y[64], ps[32], ds[32];
          if (!warp_wait(&sm.s_full, t & 1, abort_flag, p.status)) return false;
          if (!warp_wait(&sm.st_full[ss], (t / kStatStages) & 1, abort_flag, p.status)) return false;
          tc_fence_after();
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) tmem_ld32(s_at + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[cc * 32]));
          tmem_wait_ld();
          tmem_ld_fence(x);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) tmem_ld32(dp_at + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&y[cc * 32]));
          tmem_wait_ld();
          tmem_ld_fence(y);
          tc_fence_before();
          warp_arrive(&sm.s_free);
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(&sm.nl[ss][col0 + c]), d4 = *reinterpret_cast<const float4*>(&sm.nd[ss][col0 + c]);
            float z[4];
            f2_split(fma2(f2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2, f2(l4.x, l4.y)), z[0], z[1]);
            f2_split(fma2(f2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sl2, f2(l4.z, l4.w)), z[2], z[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = ex2_approx(z[k]);
            ps[c >> 1] = c4_pack<F16>(z[0], z[1]), ps[(c >> 1) + 1] = c4_pack<F16>(z[2], z[3]);
            f2_split(mul2(f2(z[0], z[1]), centred(y[c], y[c + 1], d4.x, d4.y)), z[0], z[1]);
            f2_split(mul2(f2(z[2], z[3]), centred(y[c + 2], y[c + 3], d4.z, d4.w)), z[2], z[3]);
            ds[c >> 1] = c4_pack<F16>(z[0], z[1]), ds[(c >> 1) + 1] = c4_pack<F16>(z[2], z[3]);
          }
          warp_arrive(&sm.st_empty[ss]);
          if (decltype(may_mask)::value && masked) keep(ps), keep(ds);
          if (t > 0) {  // dV, dK of the tile before have read P and dS
            if (!warp_wait(&sm.pd_free, (t - 1) & 1, abort_flag, p.status)) return false;
            tc_fence_after();
          }
          tmem_st32(lanes + 256 + wg * 32, ps);
          tmem_st32(lanes + 320 + wg * 32, ds);
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sm.p_full);
        } else {
          uint32_t x[64], pk[32];
          if (!warp_wait(&sm.s_full, t & 1, abort_flag, p.status)) return false;
          if (!warp_wait(&sm.st_full[ss], (t / kStatStages) & 1, abort_flag, p.status)) return false;
          tc_fence_after();
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) tmem_ld32(s_at + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[cc * 32]));
          tmem_wait_ld();
          tmem_ld_fence(x);
          uint64_t pr[32];  // P, in pairs
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(&sm.nl[ss][col0 + c]);
            float y[4];
            f2_split(fma2(f2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2, f2(l4.x, l4.y)), y[0], y[1]);
            f2_split(fma2(f2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sl2, f2(l4.z, l4.w)), y[2], y[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = ex2_approx(y[k]);
            pr[c >> 1] = f2(y[0], y[1]), pr[(c >> 1) + 1] = f2(y[2], y[3]);
            pk[c >> 1] = c4_pack<F16>(y[0], y[1]), pk[(c >> 1) + 1] = c4_pack<F16>(y[2], y[3]);
          }
          if (decltype(may_mask)::value && masked) keep(pk);
          tmem_st32(s_at, pk);
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sm.p_full);
          if (!warp_wait(&sm.dp_full, t & 1, abort_flag, p.status)) return false;
          tc_fence_after();
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) tmem_ld32(dp_at + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[cc * 32]));
          tmem_wait_ld();
          tmem_ld_fence(x);
          tc_fence_before();
          warp_arrive(&sm.dp_free);
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 d4 = *reinterpret_cast<const float4*>(&sm.nd[ss][col0 + c]);
            float y[4];
            f2_split(mul2(pr[c >> 1], centred(x[c], x[c + 1], d4.x, d4.y)), y[0], y[1]);
            f2_split(mul2(pr[(c >> 1) + 1], centred(x[c + 2], x[c + 3], d4.z, d4.w)), y[2], y[3]);
            pk[c >> 1] = c4_pack<F16>(y[0], y[1]), pk[(c >> 1) + 1] = c4_pack<F16>(y[2], y[3]);
          }
          warp_arrive(&sm.st_empty[ss]);
          if (decltype(may_mask)::value && masked) keep(pk);
          tmem_st32(s_at + 32, pk);
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sm.ds_full);
          s_col ^= 128u;
        }
        ++t;
        return true;
      };
      // Tiles [plain, last) need no mask: whole ones whose first token sees the last key of a whole key tile and whose last
      // token still sees the first
      int plain = b, last = b;
      if (a < b) {
        const long long see = static_cast<long long>(e.diag) + kTile - 1 - e.shift;  // token that sees the last key
        plain = static_cast<int>(min(static_cast<long long>(b), max(static_cast<long long>(a), see <= 0 ? 0 : (see + p.tpt - 1) / p.tpt)));
        last = min(b, e.m / p.tpt);
        if (window) {
          const long long until = static_cast<long long>(e.diag) + window - e.shift;  // the first token that no longer sees the first key
          last = until < p.tpt ? plain : static_cast<int>(min(static_cast<long long>(last), until / p.tpt));
        }
        last = max(last, plain);
      }
      bool ok = true;
      if (D == 64) {
        for (int i = a; i < b && ok; ++i) ok = tile(std::true_type{}, i < plain || i >= last, i);
      } else {
        int i = a;
        for (int part = 0; part < 2 && ok; ++part) {
          const int stop = part ? b : plain;
          for (; i < stop && ok; ++i) ok = tile(std::true_type{}, true, i);
          if (part == 0)
            for (; i < last && ok; ++i) ok = tile(std::false_type{}, false, i);
        }
      }
      if (!ok) break;
      if (a < b) {
        if (!warp_wait(&sm.acc_full, n_acc & 1, abort_flag, p.status)) break;
        tc_fence_after();
        ++n_acc;
      }
      // the first warpgroup writes dV, the second dK, 16 rows of a warp's 32 at a time
      const int row = quarter * 32 + (lane >> 2);
      const uint32_t from = lanes + (wg ? colDK : colDV);
      const float back = !F16 ? 1.f : wg ? down : pow2(-kPUp);
      const float f[2] = {back, back};
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t at = from + (static_cast<uint32_t>(hf * 16) << 16);
        if (e.slot >= 0) {  // this chunk's share, for the join behind these kernels
          float* const mine = p.part + ((static_cast<long long>(e.slot + e.chunk) * p.Hkv + head) * 2 + wg) * kTile * D;
          quad_blocks<D>(at, a < b, [&](int c, const uint32_t(&acc)[16]) { leave_part<D, F16>(mine + c, acc, row + 16 * hf, f); });
          continue;
        }
        uint16_t* to[2];
        bool live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = row + 16 * hf + 8 * u;
          live[u] = c < n_tok;
          to[u] = wg ? p.dk + static_cast<long long>(e.k0 + c) * p.dkt + head * p.dkh
                     : p.dv + static_cast<long long>(e.k0 + c) * p.dvt + head * p.dvh;
        }
        quad_blocks<D>(at, a < b, [&](int c, const uint32_t(&acc)[16]) {
#pragma unroll
          for (int u = 0; u < 2; ++u) quad_store<F16>(to[u] + c, live[u], acc, u, wg ? p.scale * back : back);
        });
      }
      if (a < b) {
        tc_fence_before();
        warp_arrive(&sm.acc_empty);
      }
      warp_arrive(&sm.item_empty[slot]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename Kernel>
cudaError_t launch_one(Kernel kern, size_t smem, bool (&allowed)[64], const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                       const CUtensorMap& dO, const PBwdParams& p, int grid, bool behind, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !allowed[dev]) {  // (setting it twice does no harm)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  return launch_behind_with(kern, dim3(grid), kThreads, smem, behind, st, q, k, v, dO, p);
}

template <int D, bool F16>
cudaError_t launch_bwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO, PBwdParams p, int sms,
                       cudaStream_t st) {
  static bool dq_allowed[64] = {}, dkv_allowed[64] = {};
  constexpr size_t dq_smem = sizeof(DqSmem<D>), dkv_smem = sizeof(DkvSmem<D>);
  static_assert(dq_smem <= 227 * 1024 && dkv_smem <= 227 * 1024, "shared memory per CTA");
  packed_stats_kernel<D, F16><<<8 * sms, 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.M > 0) e = launch_one(packed_dkv_kernel<D, F16>, dkv_smem, dkv_allowed, q, k, v, dO, p, sms, true, st);
  ++p.counter;
  if (e == cudaSuccess && p.N > 0) e = launch_one(packed_dq_kernel<D, F16>, dq_smem, dq_allowed, q, k, v, dO, p, sms, p.M > 0, st);
  return e;
}

bool write_rows_ok(const void* p, long long token, long long head, int n, int H, int D) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15u) && !((token | head) & 7) && !c4_rows_overlap(token, head, n, H, D);
}

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" scfa_status scfa_packed_bwd(const uint16_t* q, long long q_token, long long q_head, const uint16_t* k, long long k_token,
                                       long long k_head, const uint16_t* v, long long v_token, long long v_head, const uint16_t* o,
                                       long long o_token, long long o_head, const float* lse, const uint16_t* dO, long long do_token,
                                       long long do_head, const void* plan, size_t plan_bytes, int N, int M, int Hq, int Hkv, int D,
                                       float scale, int dtype, uint16_t* dq, long long dq_token, long long dq_head, uint16_t* dk,
                                       long long dk_token, long long dk_head, uint16_t* dv, long long dv_token, long long dv_head,
                                       void* ws, size_t ws_bytes, unsigned flags, void* stream) {
  if (!plan || !ws || N < 0 || M < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0) return SCFA_ERR_INVALID;
  const float factor = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // to log2 units
  if (!(scale > 0.f && factor < INFINITY)) return SCFA_ERR_INVALID;
  if ((D != 64 && D != 128) || (dtype != SCFA_DTYPE_BF16 && dtype != SCFA_DTYPE_F16) || Hq / Hkv > kTile) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * Hq >= (1ll << 31) - 256 || static_cast<long long>(M) * Hkv >= (1ll << 31) - 256) return SCFA_ERR_UNSUPPORTED;
  const int sms = num_sms();
  const PackWs w = pack_ws(D, sms);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < w.stats) return SCFA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(plan) & 255u) || plan_bytes < sizeof(PackHeader)) return SCFA_ERR_INVALID;
  if (N > 0 && (!lse || !pack_rows_ok(q, q_token, q_head, N, Hq) || !pack_rows_ok(o, o_token, o_head, N, Hq) ||
                !pack_rows_ok(dO, do_token, do_head, N, Hq) || !write_rows_ok(dq, dq_token, dq_head, N, Hq, D)))
    return SCFA_ERR_INVALID;
  if (M > 0 && (!pack_rows_ok(k, k_token, k_head, M, Hkv) || !pack_rows_ok(v, v_token, v_head, M, Hkv) ||
                !write_rows_ok(dk, dk_token, dk_head, M, Hkv, D) || !write_rows_ok(dv, dv_token, dv_head, M, Hkv, D)))
    return SCFA_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* c = static_cast<char*>(ws);
  if (N == 0 && M == 0) return cudaMemsetAsync(c, 0, w.clear, st) == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
  PBwdParams p = {};
  p.plan = static_cast<const char*>(plan), p.plan_bytes = static_cast<long long>(plan_bytes);
  p.N = N, p.M = M, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.tpt = kTile / p.G, p.scale = scale, p.scale_log2 = factor;
  p.o = o, p.ot = o_token, p.oh = o_head, p.dO = dO, p.dot = do_token, p.doh = do_head, p.lse = lse;
  p.v = v, p.vt = v_token, p.vh = v_head;
  p.dq = dq, p.dqt = dq_token, p.dqh = dq_head, p.dk = dk, p.dkt = dk_token, p.dkh = dk_head, p.dv = dv, p.dvt = dv_token, p.dvh = dv_head;
  p.counter = reinterpret_cast<int*>(c + w.counters);
  p.part = reinterpret_cast<float*>(c + w.part), p.part_q = reinterpret_cast<float*>(c + w.part_q), p.stats = reinterpret_cast<float*>(c + w.stats);
  p.stats_bytes = static_cast<long long>(ws_bytes - w.stats);
  p.stall = (flags & SCFA_FLAG_DEBUG_STALL) ? 1 : 0, p.status = reinterpret_cast<int*>(c);
  const bool f16 = dtype == SCFA_DTYPE_F16;
  CUtensorMap tq = {}, tk = {}, tv = {}, tdo = {};
  if (N > 0 && (!make_tmap_rows(&tq, q, f16, D, Hq, N, q_head, q_token, p.G, p.tpt) ||
                !make_tmap_rows(&tdo, dO, f16, D, Hq, N, do_head, do_token, p.G, p.tpt)))
    return SCFA_ERR_INVALID;
  if (M > 0 && (!make_tmap_rows(&tk, k, f16, D, Hkv, M, k_head, k_token, 1, kTile) ||
                !make_tmap_rows(&tv, v, f16, D, Hkv, M, v_head, v_token, 1, kTile)))
    return SCFA_ERR_INVALID;
  // without queries (or keys) no tile of them is ever copied: any valid map will do
  if (N == 0) tq = tdo = tk;
  if (M == 0) tk = tv = tq;
  const cudaError_t e = D == 64 ? (f16 ? launch_bwd<64, true>(tq, tk, tv, tdo, p, sms, st) : launch_bwd<64, false>(tq, tk, tv, tdo, p, sms, st))
                                : (f16 ? launch_bwd<128, true>(tq, tk, tv, tdo, p, sms, st) : launch_bwd<128, false>(tq, tk, tv, tdo, p, sms, st));
  if (e != cudaSuccess) return SCFA_ERR_CUDA;
  PackJoin j = {};
  j.plan = p.plan, j.plan_bytes = p.plan_bytes, j.N = N, j.M = M, j.Hq = Hq, j.Hkv = Hkv, j.G = p.G, j.tpt = p.tpt;
  j.part = p.part, j.part_q = p.part_q, j.scale = scale, j.status = p.status;
  j.dq = dq, j.dqt = dq_token, j.dqh = dq_head, j.dk = dk, j.dkt = dk_token, j.dkh = dk_head, j.dv = dv, j.dvt = dv_token, j.dvh = dv_head;
  if (pack_may_cut(N, M, p.tpt, true) && launch_pack_join(j, D, f16, true, sms, st) != cudaSuccess) return SCFA_ERR_CUDA;
  if ((flags & SCFA_FLAG_DEBUG_SYNC) && cudaStreamSynchronize(st) != cudaSuccess) return SCFA_ERR_CUDA;
  return SCFA_OK;
}
