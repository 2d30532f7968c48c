// Attention over packed sequences with shared key heads, forward: o = softmax(scale q K^T) V and the log-sum-exp of each
// query row, over the keys that its token sees (causal, the last query at the last key; optionally the last `window`).
//
// One pass over the keys with a running reference m and sum l per row: P = 2^(s scale log2(e) - m), O += P V, and when a
// row's maximum outgrows m by more than 8 (log2 units) O and l are brought to the new one. O / l and m + log2(l) at the
// end. S, O, m and l are fp32; P is rounded once to the rows' type for its product with V (the tensor cores take 16-bit
// operands), at most 2^8 by the rule above.
//
// One CTA per SM, work from a counter, longest first. A work item is two tiles of query rows of one key head that share
// each K and V tile. Roles:
//   warp 0        producer: TMA of the item's two Q tiles and of K_j, V_j into rings
//   warp 1 (2)    MMA issuers: S = Q K^T, then O += P V with P read from TMEM, in two halves of the keys
//   warps 4-7, 8-11  softmax of tile 0 and 1: thread = row = TMEM lane; a row's 128 scores stay in its registers (216 of
//                 them; the first four warps give up what they do not need)
// TMEM: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 behind it. At D = 128 that is all of it and P_g takes the first
// half of S_g; at D = 64 P_g has columns of its own and S of the next key tile runs under the softmax of this one.
//
// Keys behind the last one of a sequence belong to another: their scores are masked, and the V rows among the 16 of the
// last MMA step are zeroed in shared memory (0 x NaN is NaN), the steps behind it left out.
//
// Entries that the plan cut leave (O, m, l) in the workspace; a kernel behind this one joins them, chunk by chunk in their
// order.
//
// Bounded at D = 128 by the chain S, softmax, P V, which two tiles take in turns (tensor cores 72% busy), at D = 64 by
// latency inside the softmax (no unit above half). Measured in a graph, one call after another: 335 us for 8192 tokens of 32
// heads over 8 of 128 channels (1,640 TFLOP/s of useful work), 484 us for 16384 of 16 heads over 4 of 64 (1,140). Called on
// inputs that change from call to call the first takes 367 us (1,500), in long runs under the power cap: 1,340 us for 16384
// tokens (1,640; 1,224 at full clocks).
#include <climits>
#include <type_traits>

#include "packed.cuh"

namespace scfa {
namespace {

constexpr int kThreads = 384;
// registers of a thread of warps 0-3 and of the softmax warps: 128 x 72 + 256 x 216 = 384 x 168, what the CTA starts with
constexpr int kRegsFew = 72, kRegsMany = 216;
constexpr int kSlots = 3;  // items known ahead
constexpr float kGrow = 8.f;
constexpr float kFarScore = 65536.f;

template <int D>
struct PFwdCfg {
  static constexpr int kSubs = D / 64;
  static constexpr int kQ = D == 64 ? 4 : 3;  // Q tiles in the ring
  static constexpr int kKs = D == 64 ? 4 : 2;  // K tiles
  static constexpr int kVs = D == 64 ? 4 : 2;  // V tiles
  static constexpr bool kOwnP = D == 64;
  static constexpr int kIssuers = D == 64 ? 2 : 1;
};

template <int D>
struct __align__(1024) PFwdSmem {
  using C = PFwdCfg<D>;
  uint8_t q[C::kQ][C::kSubs][kPackSub];
  uint8_t k[C::kKs][C::kSubs][kPackSub];
  uint8_t v[C::kVs][C::kSubs][kPackSub];
  PackEntry item[kSlots];
  uint64_t q_full[C::kQ], q_empty[C::kQ], k_full[C::kKs], v_full[C::kVs], k_empty[C::kKs], v_empty[C::kVs];
  uint64_t s_full[2], s_free[2], p_full[2][2], pv_done[2], o_full[2], o_empty[2], drain[2];
  uint64_t tail, item_full[kSlots], item_empty[kSlots];
  uint32_t tmem_base;
  int abort_flag;
};

struct PFwdParams {
  const char* plan;
  long long plan_bytes;
  int N, M, Hq, Hkv, G, tpt;
  float scale_log2;
  uint16_t* o;
  long long ot, oh;
  float* lse;
  int* counter;   // next item
  float* part;    // [slot][Hkv][2][(D + 2) x 128]
  int stall;
  int* status;
};

// Key tiles [a, b) of query tile g of an entry (empty: nothing to compute for it here).
__device__ __forceinline__ void fwd_range(const PackEntry& e, int g, int tpt, int window, int& a, int& b) {
  const int first = e.diag + g * tpt, n = min(tpt, e.n_tok - g * tpt), last = first + n - 1;
  a = b = 0;
  if (n <= 0 || last < 0) return;
  b = min(e.b, last / kTile + 1);
  a = e.a;
  if (window && first - window + 1 > 0) a = max(a, (first - window + 1) / kTile);
  if (a >= b) a = b = 0;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PFwdParams p) {
  using C = PFwdCfg<D>;
  constexpr int kSubs = C::kSubs, kKs = C::kKs, kVs = C::kVs, kQ = C::kQ;
  constexpr bool kOwnP = C::kOwnP;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  PFwdSmem<D>& sm = *reinterpret_cast<PFwdSmem<D>*>(smem_raw + pad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PackHeader* const h = reinterpret_cast<const PackHeader*>(p.plan);
  const int plan_status = pack_plan_status(h, p.plan_bytes, p.N, p.M, p.Hq, p.Hkv);
  if (plan_status != SCFA_OK) {  // the same for every thread
    grid_wait();
    if (threadIdx.x == 0) raise_status(p.status, plan_status);
    return;
  }
  const int window = h->window, n_work = h->n_entries[kListFwd] * p.Hkv;
  const int used = p.G * p.tpt;  // rows of a tile that hold a query
  PackWork work;
  if (warp == 0) work.first(reinterpret_cast<const PackEntry*>(p.plan + h->entries[kListFwd]), n_work, p.Hkv, lane);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQ; ++s) mbar_init(&sm.q_full[s], 1), mbar_init(&sm.q_empty[s], 1);
    for (int s = 0; s < kKs; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], C::kIssuers);
    for (int s = 0; s < kVs; ++s) mbar_init(&sm.v_full[s], 1), mbar_init(&sm.v_empty[s], C::kIssuers);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sm.s_full[g], 1), mbar_init(&sm.s_free[g], 4);
      mbar_init(&sm.p_full[g][0], 4), mbar_init(&sm.p_full[g][1], 4);
      mbar_init(&sm.pv_done[g], 1), mbar_init(&sm.o_full[g], 1), mbar_init(&sm.o_empty[g], 4);
    }
    mbar_init(&sm.tail, 1), mbar_init(&sm.drain[0], 1), mbar_init(&sm.drain[1], 1);
    for (int s = 0; s < kSlots; ++s) mbar_init(&sm.item_full[s], 1), mbar_init(&sm.item_empty[s], C::kIssuers + 8);
    sm.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_v);
  }
  if (used < kTile) {  // rows that no copy writes: zero for good
    for (int s = 0; s < kQ; ++s) zero_tile_rows(sm.q[s][0], kSubs, used, kTile, threadIdx.x, kThreads);
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* const abort_flag = &sm.abort_flag;
  grid_wait();     // the status and the counter are clear
  grid_release();  // the join's CTAs come as these leave

  if (warp < 4) {
  regs_release<kRegsFew>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int q_it = 0, k_it = 0, kv_it = 0, tails = 0, unmarked = -1;  // unmarked: V tile whose zeros an abort kept from being written
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int slot = it % kSlots;
      ok = warp_wait(&sm.item_empty[slot], ((it / kSlots) & 1) ^ 1, abort_flag, p.status);
      if (!ok || !work.publish(&sm.item[slot], &sm.item_full[slot], lane)) break;
      const PackEntry& e = sm.item[slot];
      const int head = e.head;
      int a[2], b[2];
      fwd_range(e, 0, p.tpt, window, a[0], b[0]);
      fwd_range(e, 1, p.tpt, window, a[1], b[1]);
      for (int g = 0; g < 2 && ok; ++g) {
        if (a[g] == b[g]) continue;
        const int s = q_it % kQ;
        ok = warp_wait(&sm.q_empty[s], ((q_it / kQ) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[s], D * used * 2);
          for (int sub = 0; sub < kSubs; ++sub)
            tma_load_3d(sm.q[s][sub], &tm_q, &sm.q_full[s], sub * 64, head * p.G, e.q0 + g * p.tpt);
        }
        ++q_it;
      }
      if (p.stall && k_it == 0 && a[0] + b[0] + a[1] + b[1] > 0) break;  // debug stall: no K / V load ever arrives
      const int j0 = a[0] == b[0] ? a[1] : a[1] == b[1] ? a[0] : min(a[0], a[1]), j1 = max(b[0], b[1]);
      if (j0 == j1) work.next(p.counter, lane);
      for (int j = j0; j < j1 && ok; ++j) {
        const int valid = e.m - j * kTile;  // keys of the sequence in the tile, if below 128
        const bool cut = valid < kTile && (valid & 15) != 0;
        const int ks = k_it % kKs, s = kv_it % kVs;
        ok = warp_wait(&sm.k_empty[ks], ((k_it / kKs) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.k_full[ks], D * kTile * 2);
          for (int sub = 0; sub < kSubs; ++sub) tma_load_3d(sm.k[ks][sub], &tm_k, &sm.k_full[ks], sub * 64, head, e.k0 + j * kTile);
        }
        ++k_it;
        ok = warp_wait(&sm.v_empty[s], ((kv_it / kVs) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) {
          uint64_t* const vb = cut ? &sm.tail : &sm.v_full[s];
          mbar_arrive_expect_tx(vb, D * kTile * 2);
          for (int sub = 0; sub < kSubs; ++sub) tma_load_3d(sm.v[s][sub], &tm_v, vb, sub * 64, head, e.k0 + j * kTile);
        }
        ++kv_it;
        if (cut) {
          ok = warp_wait(&sm.tail, tails & 1, abort_flag, p.status);
          ++tails;
          if (!ok) {
            unmarked = kv_it - 1;
            break;
          }
          zero_tile_rows(sm.v[s][0], kSubs, valid, (valid + 15) & ~15, lane, 32);
          fence_proxy_async_smem();
          warp_arrive(&sm.v_full[s]);
        }
        if (j == j0) work.next(p.counter, lane);  // (under the loads)
      }
    }
    if (lane == 0) {
      // every copy issued has landed before the CTA exits, also after an abort
      if (tails > 0) mbar_wait_drain(&sm.tail, (tails - 1) & 1, p.status);
      for (int d = 1; d <= kKs && d <= k_it; ++d)
        mbar_wait_drain(&sm.k_full[(k_it - d) % kKs], ((k_it - d) / kKs) & 1, p.status);
      for (int d = 1; d <= kVs && d <= kv_it; ++d) {
        const int i = kv_it - d;
        if (i != unmarked) mbar_wait_drain(&sm.v_full[i % kVs], (i / kVs) & 1, p.status);
      }
      for (int d = 1; d <= kQ && d <= q_it; ++d)
        mbar_wait_drain(&sm.q_full[(q_it - d) % kQ], ((q_it - d) / kQ) & 1, p.status);
    }
  } else if (warp <= C::kIssuers) {
    // ------------------------------------------------------------ MMA issuers
    // D = 128: one thread issues for both tiles, in turns: tile 0's products
    // come whole before tile 1's, which keeps one tile's softmax under the
    // other's products. (With a thread for each the two fell into step, both in
    // the softmax, then both waiting for the tensor cores.) D = 64: a thread
    // for each; its MMAs are so short that issuing them counts.
    if (elect_one()) {
      constexpr uint32_t idesc_s = pack_idesc<F16>(kTile, kTile, 0, 0);
      constexpr uint32_t idesc_o = pack_idesc<F16>(kTile, D, 0, 1);
      constexpr uint32_t kTile16 = (kSubs * kPackSub) >> 4;
      const uint32_t qdesc = desc_low(smem_u32(sm.q[0][0]), 16), kdesc = desc_low(smem_u32(sm.k[0][0]), 16);
      const uint32_t vdesc = desc_low(smem_u32(sm.v[0][0]), kPackSub);
      const int g0 = C::kIssuers == 2 ? warp - 1 : 0, g1 = C::kIssuers == 2 ? warp : 2;  // this thread's tiles
      int q_it = 0, kv_it = 0, n_s[2] = {0, 0}, n_p[2] = {0, 0}, n_o[2] = {0, 0};
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % kSlots;
        if (!mbar_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
        const PackEntry& e = sm.item[slot];
        if (sm.item[slot].head < 0) break;
        int a[2], b[2], qi[2];
        fwd_range(e, 0, p.tpt, window, a[0], b[0]);
        fwd_range(e, 1, p.tpt, window, a[1], b[1]);
        const int m_keys = e.m;
        const int j0 = a[0] == b[0] ? a[1] : a[1] == b[1] ? a[0] : min(a[0], a[1]), j1 = max(b[0], b[1]);
        qi[0] = q_it, qi[1] = q_it + (a[0] < b[0]);
        q_it = qi[1] + (a[1] < b[1]);
        bool first[2] = {true, true};
        // S_g of key tile j (number kvi); behind the last one Q_g is free
        auto issue_s = [&](int g, int j, int kvi) -> bool {
          const int s = kvi % kKs, qs = qi[g] % kQ;
          if (j == a[g] && !mbar_wait(&sm.q_full[qs], (qi[g] / kQ) & 1, abort_flag, p.status)) return false;
          if (kOwnP && n_s[g] > 0 && !mbar_wait(&sm.s_free[g], (n_s[g] - 1) & 1, abort_flag, p.status)) return false;
          if (!mbar_wait(&sm.k_full[s], (kvi / kKs) & 1, abort_flag, p.status)) return false;
          tc_fence_after();
          mma_ss_steps<0, D / 16>(tmem + 128u * g, qdesc + qs * kTile16, kdesc + s * kTile16, idesc_s, false);
          tc_commit(&sm.s_full[g]);
          if (j == b[g] - 1) tc_commit(&sm.q_empty[qs]);
          ++n_s[g];
          return true;
        };
        auto issue_pv = [&](int g, int j, int kvi) -> bool {
          const int s = kvi % kVs, steps = min(kTile / 16, (m_keys - j * kTile + 15) >> 4);
          const uint32_t bv = vdesc + s * kTile16;
          const uint32_t dO = tmem + 256u + D * g, aP = kOwnP ? tmem + 384u + 64u * g : tmem + 128u * g;
          if (!mbar_wait(&sm.v_full[s], (kvi / kVs) & 1, abort_flag, p.status)) return false;
          if (first[g] && !mbar_wait(&sm.o_empty[g], (n_o[g] & 1) ^ 1, abort_flag, p.status)) return false;
          if (!mbar_wait(&sm.p_full[g][0], n_p[g] & 1, abort_flag, p.status)) return false;
          tc_fence_after();
          if (steps == 8) mma_ts_steps<0, 4>(dO, aP, bv, idesc_o, !first[g], 8);
          else mma_ts_steps<0, 4>(dO, aP, bv, idesc_o, !first[g], steps);
          if (!mbar_wait(&sm.p_full[g][1], n_p[g] & 1, abort_flag, p.status)) return false;
          tc_fence_after();
          if (steps == 8) mma_ts_steps<4, 8>(dO, aP, bv, idesc_o, true, 8);
          else mma_ts_steps<4, 8>(dO, aP, bv, idesc_o, true, steps);
          if (kOwnP) tc_commit(&sm.pv_done[g]);
          first[g] = false;
          ++n_p[g];
          return true;
        };
        auto in = [&](int g, int j) { return j >= a[g] && j < b[g]; };
        // K_j goes back once both tiles' S of it are issued, long before V_j.
        // A tile that this thread skips goes back once it has landed: a run
        // through such tiles must not give another thread's arrivals too
        auto release_k = [&](bool used, int kvi) -> bool {
          if (C::kIssuers == 2 && !used && !mbar_wait(&sm.k_full[kvi % kKs], (kvi / kKs) & 1, abort_flag, p.status)) return false;
          tc_commit(&sm.k_empty[kvi % kKs]);
          return true;
        };
        if (C::kIssuers == 2) {
          const int g = g0;
          if (j0 < j1) {
            if (in(g, j0)) ok = issue_s(g, j0, kv_it);
            ok = ok && release_k(in(g, j0), kv_it);
          }
          for (int j = j0; j < j1 && ok; ++j, ++kv_it) {
            if (j + 1 < j1) {
              if (in(g, j + 1)) ok = issue_s(g, j + 1, kv_it + 1);
              ok = ok && release_k(in(g, j + 1), kv_it + 1);
            }
            if (ok && in(g, j)) ok = issue_pv(g, j, kv_it);
            else if (ok) ok = mbar_wait(&sm.v_full[kv_it % kVs], (kv_it / kVs) & 1, abort_flag, p.status);
            if (ok) tc_commit(&sm.v_empty[kv_it % kVs]);
          }
        } else {
          for (int g = 0; g < 2 && ok; ++g)
            if (in(g, j0)) ok = issue_s(g, j0, kv_it);
          if (j0 < j1) tc_commit(&sm.k_empty[kv_it % kKs]);
          for (int j = j0; j < j1 && ok; ++j, ++kv_it) {
            for (int g = 0; g < 2 && ok; ++g) {
              if (in(g, j)) ok = issue_pv(g, j, kv_it);
              if (ok && in(g, j + 1)) ok = issue_s(g, j + 1, kv_it + 1);
            }
            tc_commit(&sm.v_empty[kv_it % kVs]);
            if (j + 1 < j1) tc_commit(&sm.k_empty[(kv_it + 1) % kKs]);
          }
        }
        if (!ok) break;
        for (int g = g0; g < g1; ++g)
          if (a[g] < b[g]) {
            tc_commit(&sm.o_full[g]);
            ++n_o[g];
          }
        mbar_arrive(&sm.item_empty[slot]);
      }
      tc_commit(&sm.drain[g0]);
      mbar_wait_drain(&sm.drain[g0], 0, p.status);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    regs_take<kRegsMany>();
    const int g = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tS = lanes + 128u * g, tO = lanes + 256u + D * g, tP = kOwnP ? lanes + 384u + 64u * g : tS;
    const int r_tok = r / p.G, r_head = r - r_tok * p.G;
    int n_s = 0, n_o = 0;
    for (int it = 0;; ++it) {
      const int slot = it % kSlots;
      if (!warp_wait(&sm.item_full[slot], (it / kSlots) & 1, abort_flag, p.status)) break;
      const PackEntry& e = sm.item[slot];
      const int head = e.head;
      if (head < 0) break;
      int a, b;
      fwd_range(e, g, p.tpt, window, a, b);
      const int first = e.diag + g * p.tpt, n_tok = min(p.tpt, e.n_tok - g * p.tpt);
      if (n_tok <= 0) {
        warp_arrive(&sm.item_empty[slot]);
        continue;
      }
      const bool valid = r_tok < n_tok;
      const int hi = valid ? first + r_tok : -1;  // the last key that the row sees
      float m = -INFINITY, l = 0.f;
      float top = -INFINITY;  // largest score so far, log2 units
      // One key tile. There is one copy of this code: with a second for the masked tiles, one or two of an item, that one
      // was fetched anew each time (5,100 cycles for such a tile, 2,400 for the others).
      auto tile = [&](auto may_mask, bool masked, int j) -> bool {
        if (!warp_wait(&sm.s_full[g], n_s & 1, abort_flag, p.status)) return false;
        tc_fence_after();
        uint32_t sr[kTile];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[cc * 32]));
        tmem_wait_ld();
        tmem_ld_fence(sr);
        if (kOwnP) {
          tc_fence_before();
          warp_arrive(&sm.s_free[g]);
        }
        if (decltype(may_mask)::value && masked) {
          // columns lo .. lim are seen: bits of 32 of them at a time
          const int lim = hi - j * kTile, lo = window ? lim - window + 1 : 0;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            const uint32_t bits = bit_range(lo - cc * 32, lim + 1 - cc * 32);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits >> c & 1u)) sr[cc * 32 + c] = 0xff800000u;
          }
        }
        float sl = p.scale_log2;
        // 32 columns of P under the reference `from` (its negative), into TMEM
        uint64_t sum[2];
        auto weigh = [&](int q, uint64_t sl2, uint64_t from) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            f2_split(fma2(f2(__uint_as_float(sr[q * 32 + c]), __uint_as_float(sr[q * 32 + c + 1])), sl2, from), x0, x1);
            x0 = ex2_approx(x0), x1 = ex2_approx(x1);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], f2(x0, x1));
            pk[c >> 1] = c4_pack<F16>(x0, x1);
          }
          tmem_st16(tP + q * 16, pk);
        };
        auto signal = [&](int half) {
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sm.p_full[g][half]);
        };
        auto taken = [&]() {
          float s0, s1;
          f2_split(add2(sum[0], sum[1]), s0, s1);
          l = s0 + s1;
        };
        auto largest = [&]() {
          float mx[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = fmaxf(__uint_as_float(sr[2 * u]), __uint_as_float(sr[2 * u + 1]));
#pragma unroll
          for (int c = 8; c < kTile; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = pack_max3(mx[u], __uint_as_float(sr[c + 2 * u]), __uint_as_float(sr[c + 2 * u + 1]));
          return pack_max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        };
        if (kOwnP && n_s > 0) {
          if (!warp_wait(&sm.pv_done[g], (n_s - 1) & 1, abort_flag, p.status)) return false;
          tc_fence_after();
        }
        float mt;
        if (j > a) {
          // The reference seldom moves behind an item's first tile. So the weights of the first half are made under the old
          // one while the maximum is still being found (on other units); if it moved after all they are made again below
          sum[0] = f2(l, 0.f), sum[1] = 0ull;
          const uint64_t sl2 = f2(sl, sl), from = f2(-m, -m);
          weigh(0, sl2, from);
          weigh(1, sl2, from);
          mt = largest() * sl;
          if (__builtin_expect(!__any_sync(0xffffffffu, mt > m + kGrow || !(fabsf(m) <= kFarScore)), 1)) {
            signal(0);
            top = fmaxf(top, mt);
            weigh(2, sl2, from);
            weigh(3, sl2, from);
            signal(1);
            taken();
            ++n_s;
            return true;
          }
        } else {
          mt = largest() * sl;
        }
        top = fmaxf(top, mt);
        const bool grown = mt > m + kGrow;
        float alpha = 1.f;
        if (grown) {
          alpha = ex2_approx(m - mt);
          m = mt;
        }
        float sub = m == -INFINITY ? 0.f : -m;
        const bool far = fabsf(sub) > kFarScore;
        if (far) {
          // far from zero an fma would give the largest score its product's rounding as a weight: both rounded alike
#pragma unroll
          for (int c = 0; c < kTile; ++c) sr[c] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(sr[c]), sl), sub));
          sl = 1.f, sub = 0.f;
        }
        // O to the new reference. The product before is complete: with P's
        // own columns by the wait above, else because S came behind it
        if (j > a && __any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t oo[16];
            tmem_ld16(tO + cc * 16, oo);
            tmem_wait_ld();
            tmem_ld_fence(oo);
#pragma unroll
            for (int c = 0; c < 16; ++c) oo[c] = __float_as_uint(__uint_as_float(oo[c]) * alpha);
            tmem_st16(tO + cc * 16, oo);
          }
        }
        const uint64_t sl2 = f2(sl, sl), from = f2(sub, sub);
        sum[0] = f2(l * alpha, 0.f), sum[1] = 0ull;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          weigh(q, sl2, from);
          if (q & 1) signal(q >> 1);
        }
        taken();
        ++n_s;
        return true;
      };
      // Tiles [plain, masked) are seen whole by every row: those before hold keys before the last token's first, those
      // behind keys after the first token's last. The plain loop stands by itself, with nothing to jump over.
      const int plain = window ? min(b, max(a, (first + n_tok - window + kTile - 1) / kTile)) : a;
      const int masked = max(plain, min(b, max(0, first + 1) / kTile));
      bool ok = true;
      if (D == 64) {
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
      if (a < b) {
        if (!warp_wait(&sm.o_full[g], n_o & 1, abort_flag, p.status)) break;
        tc_fence_after();
        ++n_o;
      }
      float inv = 1.f;
      const bool cut = e.slot >= 0;
      float* const mine = p.part + (static_cast<long long>(e.slot + e.chunk) * p.Hkv + head) * 2 * kTile * (D + 2) + g * kTile * (D + 2);
      if (cut) {
        reinterpret_cast<float2*>(mine + kTile * D)[r] = make_float2(m, l);
      } else {
        // O is divided by the sum with the largest score's weight as the product saw it, rounded: a row with one key gives
        // that row of V exactly
        const float w = ex2_approx(top - m);
        float w_r;
        if (F16) w_r = __half2float(__float2half_rn(w));
        else w_r = __bfloat162float(__float2bfloat16_rn(w));
        inv = l > 0.f ? 1.f / (l + (w_r - w)) : l == 0.f ? 0.f : l;
      }
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t from = tO + (static_cast<uint32_t>(hf * 16) << 16);
        if (cut) {  // this chunk's share, for the join behind this kernel
          quad_blocks<D>(from, a < b, [&](int c, const uint32_t(&acc)[16]) { leave_part<D>(mine + c, acc, quarter * 32 + hf * 16 + (lane >> 2)); });
          continue;
        }
        uint16_t* row[2];
        float f[2];
        bool live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = hf * 16 + (lane >> 2) + 8 * u, t = __shfl_sync(0xffffffffu, r_tok, at);
          f[u] = __shfl_sync(0xffffffffu, inv, at), live[u] = t < n_tok;
          row[u] = p.o + (e.q0 + g * p.tpt + t) * p.ot + (head * p.G + quarter * 32 + at - t * p.G) * p.oh;
        }
        quad_blocks<D>(from, a < b, [&](int c, const uint32_t(&acc)[16]) {
#pragma unroll
          for (int u = 0; u < 2; ++u) quad_store<F16>(row[u] + c, live[u], acc, u, f[u]);
        });
      }
      if (a < b) {
        tc_fence_before();
        warp_arrive(&sm.o_empty[g]);
      }
      if (valid && !cut) p.lse[(static_cast<long long>(e.q0) + g * p.tpt + r_tok) * p.Hq + head * p.G + r_head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kPackLn2;
      warp_arrive(&sm.item_empty[slot]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// The status and the counter. A kernel, so that the next one sets itself up meanwhile: in a graph 7 short texts take 10.7 us
// so, 14.7 behind a memset (a launch takes the host 1 us more than a memset).
__global__ void packed_clear_kernel(int* words, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) words[i] = 0;
  grid_release();
}

template <int D, bool F16>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PFwdParams& p, int grid, cudaStream_t st) {
  static bool allowed[64] = {};  // by device; setting it twice does no harm
  constexpr size_t smem = sizeof(PFwdSmem<D>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    e = cudaFuncSetAttribute(packed_fwd_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  return launch_behind_with(packed_fwd_kernel<D, F16>, dim3(grid), kThreads, smem, true, st, q, k, v, p);
}

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" scfa_status scfa_packed_fwd(const uint16_t* q, long long q_token, long long q_head, const uint16_t* k, long long k_token,
                                       long long k_head, const uint16_t* v, long long v_token, long long v_head,
                                       const void* plan, size_t plan_bytes, int N, int M, int Hq, int Hkv, int D, float scale,
                                       int dtype, uint16_t* o, long long o_token, long long o_head, float* lse, void* ws,
                                       size_t ws_bytes, unsigned flags, void* stream) {
  if (!plan || !ws || N < 0 || M < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0) return SCFA_ERR_INVALID;
  const float factor = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // to log2 units
  if (!(scale > 0.f && factor < INFINITY)) return SCFA_ERR_INVALID;
  if ((D != 64 && D != 128) || (dtype != SCFA_DTYPE_BF16 && dtype != SCFA_DTYPE_F16) || Hq / Hkv > kTile) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * Hq >= (1ll << 31) - 256 || static_cast<long long>(M) * Hkv >= (1ll << 31) - 256) return SCFA_ERR_UNSUPPORTED;
  const int sms = num_sms();
  const PackWs w = pack_ws(D, sms);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < w.forward) return SCFA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(plan) & 255u) || plan_bytes < sizeof(PackHeader)) return SCFA_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N > 0 && (!lse || !pack_rows_ok(q, q_token, q_head, N, Hq) || !o || (reinterpret_cast<uintptr_t>(o) & 15u) ||
                ((o_token | o_head) & 7) || c4_rows_overlap(o_token, o_head, N, Hq, D)))
    return SCFA_ERR_INVALID;
  if (M > 0 && (!pack_rows_ok(k, k_token, k_head, M, Hkv) || !pack_rows_ok(v, v_token, v_head, M, Hkv))) return SCFA_ERR_INVALID;
  char* c = static_cast<char*>(ws);
  packed_clear_kernel<<<1, 64, 0, st>>>(reinterpret_cast<int*>(c), static_cast<int>(w.clear / sizeof(int)));
  if (cudaGetLastError() != cudaSuccess) return SCFA_ERR_CUDA;
  if (N == 0) return SCFA_OK;
  PFwdParams p = {};
  p.plan = static_cast<const char*>(plan), p.plan_bytes = static_cast<long long>(plan_bytes);
  p.N = N, p.M = M, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.tpt = kTile / p.G, p.scale_log2 = factor;
  p.o = o, p.ot = o_token, p.oh = o_head, p.lse = lse;
  p.counter = reinterpret_cast<int*>(c + w.counters);
  p.part = reinterpret_cast<float*>(c + w.part);
  p.stall = (flags & SCFA_FLAG_DEBUG_STALL) ? 1 : 0, p.status = reinterpret_cast<int*>(c);
  const bool f16 = dtype == SCFA_DTYPE_F16;
  CUtensorMap tq, tk, tv;
  // without keys every row is empty and no K or V is ever copied: any valid map will do
  if (!make_tmap_rows(&tq, q, f16, D, Hq, N, q_head, q_token, p.G, p.tpt)) return SCFA_ERR_INVALID;
  if (M > 0 ? !make_tmap_rows(&tk, k, f16, D, Hkv, M, k_head, k_token, 1, kTile) || !make_tmap_rows(&tv, v, f16, D, Hkv, M, v_head, v_token, 1, kTile)
            : (tk = tv = tq, false))
    return SCFA_ERR_INVALID;
  const cudaError_t e = D == 64 ? (f16 ? launch<64, true>(tq, tk, tv, p, sms, st) : launch<64, false>(tq, tk, tv, p, sms, st))
                                : (f16 ? launch<128, true>(tq, tk, tv, p, sms, st) : launch<128, false>(tq, tk, tv, p, sms, st));
  if (e != cudaSuccess) return SCFA_ERR_CUDA;
  PackJoin j = {};
  j.plan = p.plan, j.plan_bytes = p.plan_bytes, j.N = N, j.M = M, j.Hq = Hq, j.Hkv = Hkv, j.G = p.G, j.tpt = p.tpt;
  j.part = p.part, j.o = o, j.ot = o_token, j.oh = o_head, j.lse = lse, j.status = p.status;
  if (pack_may_cut(N, M, p.tpt, false) && launch_pack_join(j, D, f16, false, sms, st) != cudaSuccess) return SCFA_ERR_CUDA;
  if ((flags & SCFA_FLAG_DEBUG_SYNC) && cudaStreamSynchronize(st) != cudaSuccess) return SCFA_ERR_CUDA;
  return SCFA_OK;
}
