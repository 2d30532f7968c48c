// The plan of attention over packed sequences: from the sequences' starts on the GPU, the lists of work that the
// forward, dQ and dK / dV kernels walk. One launch per batch of sequences, whatever the number of layers.
//
// One CTA builds each list, in four passes over the tiles of one key head: count the tiles of each sequence, find each
// tile's range of tiles on the other side (its units: 128 x 128 score tiles), choose how long a piece of work may be,
// and write the pieces, longest first. Latency is all that counts, a chain of loads and barriers: 16 us for one sequence of
// 8,192 tokens, 56 for one of 131,072, 83 for 5,000 of one token; once a batch, for all its layers.
//
// Cutting. A kernel's CTAs take pieces from a counter, longest first. Where few tiles have long ranges (a long prefix
// under few new tokens, few heads) that leaves SMs idle, so ranges longer than L units are cut into equal chunks whose
// results are joined later, in order. L is the candidate with the least estimate among eighths of the units per SM and
// "no cut". The estimate is a round's length times the rounds that the long pieces take, less what the short ones fill of
// the last round, and three units for leaving and joining a chunk.
// Where all tiles are alike (a window, equal texts) the last round may be nearly empty: 784 equal items on 152 SMs take
// six rounds for 5.2. Then the items of that round alone are cut.
#include "packed.cuh"

namespace scfa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;
constexpr int kCandidates = 16;

struct PlanArgs {
  const int32_t *q_start, *k_start;
  char* plan;
  PackPlanLayout L;
  int N, M, R, Hq, Hkv, tpt, window, sms;
  bool from_0;  // the first sequence has to start at row 0
};

// inclusive scan over the CTA; `total` is the sum
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) s_warp[w] = v;
  __syncthreads();
  int s = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
  return v + (w > 0 ? before : 0);
}

// pre[r] = tiles of the sequences before r; returns their number
__device__ int tile_prefix(const int32_t* start, int R, int tile, int* pre, int* s_warp) {
  int base = 0;
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + threadIdx.x;
    const int n = r < R ? (start[r + 1] - start[r] + tile - 1) / tile : 0;
    int total;
    const int upto = block_scan(n, s_warp, total);
    if (r < R) pre[r] = base + upto - n;
    base += total;
  }
  if (threadIdx.x == 0) pre[R] = base;
  __syncthreads();
  return base;
}

// range [a, b) of tile i of a sequence with n queries and m keys
__device__ __forceinline__ void tile_range(int list, int i, int n, int m, int tpt, int window, int& a, int& b) {
  const long long shift = static_cast<long long>(m) - n;
  a = b = 0;
  if (list == kListDkv) {
    const long long c0 = static_cast<long long>(i) * kTile, c1 = min(static_cast<long long>(m), c0 + kTile) - 1;
    const long long t0 = max(0ll, c0 - shift);
    const long long t1 = window ? min(n - 1ll, c1 - shift + window - 1) : n - 1ll;
    if (t0 > t1) return;
    a = static_cast<int>(t0 / tpt), b = static_cast<int>(t1 / tpt) + 1;
    return;
  }
  const int tile = list == kListFwd ? 2 * tpt : tpt;
  const long long t0 = static_cast<long long>(i) * tile, t1 = min(static_cast<long long>(n), t0 + tile) - 1;
  if (t1 + shift < 0) return;
  const long long lo = window ? t0 + shift - window + 1 : 0;
  a = lo > 0 ? static_cast<int>(lo / kTile) : 0, b = static_cast<int>((t1 + shift) / kTile) + 1;
}

__global__ void __launch_bounds__(kPlanThreads) pack_plan_kernel(const PlanArgs p) {
  __shared__ int s_warp[32];
  __shared__ int s_bin[kBins], s_big[kCandidates], s_cut[kCandidates];
  __shared__ unsigned long long s_units, s_work[kCandidates];  // units of long pieces
  __shared__ int s_most, s_bad, s_limit, s_tail, s_tail_limit, s_slots, s_cuts;
  const int list = blockIdx.x, tid = threadIdx.x;
  PackHeader* h = reinterpret_cast<PackHeader*>(p.plan);
  int* const pre = reinterpret_cast<int*>(p.plan + p.L.pre) + static_cast<long long>(list) * (p.R + 1);
  int* const pre_q = list == kListDkv ? reinterpret_cast<int*>(p.plan + p.L.pre) + 3ll * (p.R + 1) : pre;
  int2* const units = reinterpret_cast<int2*>(p.plan + p.L.units[list]);
  PackEntry* const out = reinterpret_cast<PackEntry*>(p.plan + p.L.entries[list]);
  if (tid == 0) s_units = 0, s_most = 0, s_bad = 0, s_slots = 0, s_cuts = 0;
  if (tid < kCandidates) s_big[tid] = s_cut[tid] = 0, s_work[tid] = 0;
  s_bin[tid] = 0;
  __syncthreads();
  bool bad = p.from_0 && p.q_start[0] != 0;
  for (int r = tid; r < p.R; r += kPlanThreads) {
    const int a = p.q_start[r], b = p.q_start[r + 1], c = p.k_start[r], d = p.k_start[r + 1];
    bad |= a < 0 || b < a || b > p.N || c < 0 || d < c || d > p.M;
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const bool refused = s_bad != 0;
  if (tid == 0) {
    if (list == 0) {
      h->magic = kPackMagic, h->N = p.N, h->M = p.M, h->R = p.R, h->Hq = p.Hq, h->Hkv = p.Hkv, h->window = p.window;
      h->qtiles = static_cast<long long>(p.L.qtiles), h->bytes = static_cast<long long>(p.L.total);
      h->status = refused ? SCFA_ERR_INVALID : SCFA_OK, h->rows = refused ? 0 : p.q_start[p.R];
    }
    h->entries[list] = static_cast<long long>(p.L.entries[list]), h->cuts[list] = static_cast<long long>(p.L.cuts[list]);
    h->n_cuts[list] = 0;
    h->list_status[list] = refused ? SCFA_ERR_INVALID : SCFA_OK;
    if (refused) h->n_entries[list] = 0;
    if (refused && list == kListDq) h->n_qtiles = 0;
  }
  if (refused) return;

  const int tile = list == kListDkv ? kTile : list == kListDq ? p.tpt : 2 * p.tpt;
  const int tiles = tile_prefix(list == kListDkv ? p.k_start : p.q_start, p.R, tile, pre, s_warp);
  if (list == kListDkv) tile_prefix(p.q_start, p.R, p.tpt, pre_q, s_warp);

  // units of each tile
  unsigned long long sum = 0;
  int most = 0;
  for (int g = tid; g < tiles; g += kPlanThreads) {
    int lo = 0, hi = p.R;  // the last sequence that starts at or before tile g (empty ones start where the next does)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= g) lo = mid;
      else hi = mid;
    }
    const int q0 = p.q_start[lo], n = p.q_start[lo + 1] - q0, m = p.k_start[lo + 1] - p.k_start[lo], i = g - pre[lo];
    int a, b;
    tile_range(list, i, n, m, p.tpt, p.window, a, b);
    units[g] = make_int2(b - a, lo);
    sum += b - a, most = max(most, b - a);
    if (list == kListDq)
      reinterpret_cast<int4*>(p.plan + p.L.qtiles)[g] = make_int4(q0 + i * p.tpt, min(p.tpt, n - i * p.tpt), i * p.tpt + m - n, 0);
  }
  most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) atomicAdd(&s_units, sum), atomicMax(&s_most, most);
  __syncthreads();

  // how long a piece may be
  const int longest = max(1, s_most);
  const long long per_sm = (static_cast<long long>(s_units) * p.Hkv + p.sms - 1) / p.sms;
  auto candidate = [&](int c) -> int {  // the last one: no cut
    if (c == kCandidates - 1 || longest <= kPackNeverCut) return longest;
    return static_cast<int>(min(static_cast<long long>(longest), max(2ll, (per_sm * (c + 2) + 7) / 8)));
  };
  int big[kCandidates], cut[kCandidates];
  unsigned long long work[kCandidates];
#pragma unroll
  for (int c = 0; c < kCandidates; ++c) big[c] = cut[c] = 0, work[c] = 0;
  for (int g = tid; g < tiles; g += kPlanThreads) {
    const int u = units[g].x;
#pragma unroll
    for (int c = 0; c < kCandidates; ++c) {
      const int L = candidate(c), n = u > L ? (u + L - 1) / L : 1;
      if (n > 1) cut[c] += n;
      if (u > L / 2) big[c] += n, work[c] += u;
    }
  }
#pragma unroll
  for (int c = 0; c < kCandidates; ++c) {
    const int x = __reduce_add_sync(0xffffffffu, big[c]), y = __reduce_add_sync(0xffffffffu, cut[c]);
    unsigned long long z = work[c];
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((tid & 31) == 0 && z) atomicAdd(&s_work[c], z);
    if ((tid & 31) == 0 && x) atomicAdd(&s_big[c], x);
    if ((tid & 31) == 0 && y) atomicAdd(&s_cut[c], y);
  }
  __syncthreads();
  if (tid < 32) {
    // in quarters of a unit, over all SMs; a candidate by a lane, the last of the cheapest is taken
    const long long room = static_cast<long long>(kPackSlotsPerSm) * p.sms, all = static_cast<long long>(s_units) * p.Hkv;
    const int c = min(tid, kCandidates - 1);
    const long long L = candidate(c), k = static_cast<long long>(s_cut[c]) * p.Hkv;
    long long best;
    {
      const long long n = static_cast<long long>(s_big[c]) * p.Hkv;
      const long long rounds = (n + p.sms - 1) / p.sms, fill = all - static_cast<long long>(s_work[c]) * p.Hkv;
      const long long idle = max(0ll, (rounds * p.sms - n) * L * 3 / 4 - fill);
      best = k > room ? 1ll << 62 : 4 * (all + idle) + 12 * k + (k ? 4ll * p.sms : 0);
    }
    int which = c;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const long long t = __shfl_xor_sync(0xffffffffu, best, o);
      const int w = __shfl_xor_sync(0xffffffffu, which, o);
      if (t < best || (t == best && w > which)) best = t, which = w;
    }
    if (tid == which) s_limit = static_cast<int>(L), s_tail = tiles;
    __syncwarp();
  }
  if (tid == 0) {
    const long long room = static_cast<long long>(kPackSlotsPerSm) * p.sms, all = static_cast<long long>(s_units) * p.Hkv;
    const long long n = static_cast<long long>(s_big[kCandidates - 1]) * p.Hkv, over = n % p.sms;
    if (s_limit >= longest && longest > kPackNeverCut && n > p.sms && over > 0 && 8 * (all - static_cast<long long>(s_work[kCandidates - 1]) * p.Hkv) < all) {
      // the items beyond whole rounds, cut to a share of an SM each
      const long long cut_tiles = (over + p.Hkv - 1) / p.Hkv, share = max(2ll, (cut_tiles * p.Hkv * longest + p.sms - 1) / p.sms);
      const long long chunks = cut_tiles * p.Hkv * ((longest + share - 1) / share);
      const long long t = 4 * p.sms * (n / p.sms * longest + share + 1) + 12 * chunks;
      if (chunks <= room && cut_tiles <= tiles && share < longest && t < 4 * p.sms * ((n + p.sms - 1) / p.sms) * longest)
        s_tail = tiles - static_cast<int>(cut_tiles), s_tail_limit = static_cast<int>(share);
    }
  }
  __syncthreads();
  const int L = s_limit, tail = s_tail, tail_limit = s_tail_limit;
  auto pieces = [&](int g, int u) {  // of tile g
    const int most_units = g >= tail ? tail_limit : L;
    return u > most_units ? (u + most_units - 1) / most_units : 1;
  };
  const int top = max(1, min(longest, L));
  auto bin = [&](int u) { return kBins - 1 - static_cast<int>(static_cast<long long>(min(u, top)) * (kBins - 1) / top); };

  // pieces by length, longest first
  for (int g = tid; g < tiles; g += kPlanThreads) {
    const int u = units[g].x, n = pieces(g, u);
    atomicAdd(&s_bin[bin(u / n)], n);
  }
  __syncthreads();
  int total;
  const int mine = s_bin[tid], upto = block_scan(mine, s_warp, total);
  __syncthreads();
  s_bin[tid] = upto - mine;
  __syncthreads();
  for (int g = tid; g < tiles; g += kPlanThreads) {
    const int2 ur = units[g];
    const int u = ur.x, r = ur.y, n = pieces(g, u), i = g - pre[r];
    const int q0 = p.q_start[r], nq = p.q_start[r + 1] - q0, k0 = p.k_start[r], m = p.k_start[r + 1] - k0;
    int a, b;
    tile_range(list, i, nq, m, p.tpt, p.window, a, b);
    PackEntry e = {};
    e.shift = m - nq, e.chunks = n, e.seq = r;
    if (list == kListDkv) {
      e.q0 = q0, e.k0 = k0 + i * kTile, e.n_tok = min(kTile, m - i * kTile), e.diag = i * kTile, e.m = nq;
      e.tile0 = pre_q[r];
    } else {
      e.q0 = q0 + i * tile, e.k0 = k0, e.n_tok = min(tile, nq - i * tile), e.diag = i * tile + m - nq, e.m = m;
      e.tile0 = g;
    }
    const int at = atomicAdd(&s_bin[bin(u / n)], n);
    e.slot = -1;
    if (n > 1) {
      e.slot = atomicAdd(&s_slots, n);
      reinterpret_cast<PackEntry*>(p.plan + p.L.cuts[list])[atomicAdd(&s_cuts, 1)] = e;
    }
    for (int c = 0; c < n; ++c) {
      e.chunk = c;
      e.a = a + static_cast<int>(static_cast<long long>(u) * c / n);
      e.b = a + static_cast<int>(static_cast<long long>(u) * (c + 1) / n);
      out[at + c] = e;
    }
  }
  __syncthreads();
  if (tid == 0) {
    h->n_cuts[list] = s_cuts;
    h->n_entries[list] = total;
    if (list == kListDq) h->n_qtiles = tiles;
  }
}

scfa_status launch_plan(const int32_t* q_start, const int32_t* k_start, int N, int M, int R, int Hq, int Hkv, int window, bool from_0,
                        void* plan, size_t plan_bytes, void* stream) {
  if (!q_start || !k_start || !plan || N < 0 || M < 0 || R < 1 || window < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0)
    return SCFA_ERR_INVALID;
  PlanArgs p = {};
  p.sms = num_sms();
  if (!pack_plan_layout(N, M, R, Hq, Hkv, p.sms, &p.L)) return SCFA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(plan) & 255u) || plan_bytes < p.L.total) return SCFA_ERR_WORKSPACE;
  p.q_start = q_start, p.k_start = k_start, p.plan = static_cast<char*>(plan);
  p.N = N, p.M = M, p.R = R, p.Hq = Hq, p.Hkv = Hkv, p.tpt = kTile / (Hq / Hkv), p.from_0 = from_0;
  p.window = window < M ? window : 0;  // (one as wide as all keys hides none, and sums with it might leave 32 bits)
  pack_plan_kernel<<<kLists, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
}

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" {

size_t scfa_packed_plan_size(int N, int M, int R, int Hq, int Hkv) {
  PackPlanLayout L;
  return pack_plan_layout(N, M, R, Hq, Hkv, num_sms(), &L) ? L.total : 0;
}

scfa_status scfa_packed_plan(const int32_t* q_start, const int32_t* k_start, int N, int M, int R, int Hq, int Hkv, int window,
                             void* plan, size_t plan_bytes, void* stream) {
  return launch_plan(q_start, k_start, N, M, R, Hq, Hkv, window, false, plan, plan_bytes, stream);
}

scfa_status scfa_packed_plan_self(const int32_t* start, int N, int R, int Hq, int Hkv, int window, void* plan, size_t plan_bytes,
                                  void* stream) {
  return launch_plan(start, start, N, N, R, Hq, Hkv, window, true, plan, plan_bytes, stream);
}

size_t scfa_packed_workspace_size(int backward, int N, int M, int R, int Hq, int Hkv, int D) {
  PackPlanLayout L;
  const int sms = num_sms();
  if ((D != 64 && D != 128) || !pack_plan_layout(N, M, R, Hq, Hkv, sms, &L)) return 0;
  const PackWs w = pack_ws(D, sms);
  if (!backward) return w.forward;
  const int tpt = kTile / (Hq / Hkv);
  return align_up(w.stats + static_cast<size_t>(pack_stats_bytes(N / tpt + static_cast<long long>(R), M, R, Hkv)), 256);
}

}  // extern "C"
