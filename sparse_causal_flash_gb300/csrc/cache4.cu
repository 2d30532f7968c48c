// The paged 4-bit key/value cache: page planning, quantising append and read.
#include <climits>

#include "cache4.cuh"
#include "internal.h"

namespace scfa {
namespace {

// ---------------------------------------------------------------- plan
// Per request, between the request scan and the token fill.
struct PlanReq {
  int32_t len;    // cached tokens before this step
  int32_t first;  // kept tokens of all requests before this one
  int32_t kept;   // kept new tokens
  int32_t taken;  // pages taken by the requests before this one
};
struct PlanArgs {
  const int32_t *len, *new_len;
  const uint8_t* keep;
  const int32_t *free_pages, *n_free;
  int32_t* table;
  int N, R, max_pages, page_size, n_pages;
  int32_t *len_out, *n_free_out, *q_start, *slot, *vis;
  int* status;
  int32_t* free_before;  // n_free as it was (n_free_out may be n_free)
  PlanReq* req;
  uint2* kept;  // per 32 tokens: the kept ones before them, and which of them are kept
};

// exclusive sum over the block; *total gets the sum. `part`: 33 entries.
__device__ __forceinline__ long long block_excl(long long x, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) part[w] = s;
  __syncthreads();
  if (w == 0) {
    long long p = lane < nw ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  const long long before = w > 0 ? part[w - 1] : 0;
  *total = part[nw - 1];
  __syncthreads();
  return before + s - x;
}

// kept tokens before token t; *keep: it is kept
__device__ __forceinline__ int kept_before(const PlanArgs& a, long long t, bool* keep) {
  const uint2 c = a.kept[t >> 5];
  *keep = c.y >> (t & 31) & 1u;
  return static_cast<int>(c.x) + __popc(c.y & ((1u << (t & 31)) - 1u));
}

// Slot, vis and a fresh table entry of token t.
__device__ __forceinline__ void plan_token(const PlanArgs& a, int t) {
  const int total = a.q_start[a.R];
  if (t >= total) {
    a.slot[t] = -1;
    a.vis[t] = 0;
    return;
  }
  int lo = 0, hi = a.R;  // the last request that starts at or before t and is not empty
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const PlanReq q = a.req[lo];
  bool keep = true;
  const int upto = a.keep == nullptr ? t : kept_before(a, t, &keep);
  const int pos = q.len + upto - q.first;
  int slot = -1;
  if (keep) {
    const int pg = pos / a.page_size, have = (q.len + a.page_size - 1) / a.page_size;
    const long long row = static_cast<long long>(lo) * a.max_pages;
    int page;
    if (pg < have) {
      page = a.table[row + pg];
    } else {
      page = a.free_pages[*a.free_before - 1 - (q.taken + pg - have)];
      if (pos % a.page_size == 0) a.table[row + pg] = page;
    }
    if (page >= 0 && page < a.n_pages) slot = page * a.page_size + pos % a.page_size;
    else raise_status(a.status, SCFA_ERR_INVALID);
  }
  a.slot[t] = slot;
  a.vis[t] = pos + (keep ? 1 : 0);
}

// One CTA: kept-token prefix, sums over the requests, the checks, the new
// state; with fill also the tokens (few of them). Latency bound: the requests
// and tokens of a decode step fit one CTA's threads once. 48 requests of one
// token: 3.9 us; 97 prompts, 24,000 tokens and a mask: 5.5 us, and 4.2 us for
// plan_fill_kernel, whose launch hides under it. The prefix leaves 8 bytes per 32
// tokens: an SM that writes every token's count takes 3 us more.
__global__ void __launch_bounds__(1024) plan_kernel(PlanArgs a, int fill) {
  __shared__ long long part[33];
  __shared__ int s_bad;
  const int tid = threadIdx.x, nt = blockDim.x;
  if (tid == 0) s_bad = 0;
  grid_release();
  // (on their way while the mask is counted)
  const int n_free = *a.n_free, len0 = tid < a.R ? a.len[tid] : 0, new0 = tid < a.R ? a.new_len[tid] : 0;
  long long kept_all = 0;
  if (a.keep != nullptr) {
    // 32 tokens a thread and round, by two loads where the mask allows it
    const bool vec = (reinterpret_cast<uintptr_t>(a.keep) & 15u) == 0;
    for (long long base = 0; base < a.N; base += 32ll * nt) {
      const long long t0 = base + 32ll * tid;
      uint32_t bits = 0;  // of the kept ones
      if (vec && t0 + 32 <= a.N) {
        const uint4* const src = reinterpret_cast<const uint4*>(a.keep + t0);
        const uint4 v = src[0], z = src[1];
        const uint32_t x[8] = {v.x, v.y, v.z, v.w, z.x, z.y, z.z, z.w};
#pragma unroll
        for (int i = 0; i < 32; ++i) bits |= ((x[i / 4] >> (8 * (i % 4)) & 255u) != 0u ? 1u : 0u) << i;
      } else {
        for (int i = 0; i < 32 && t0 + i < a.N; ++i) bits |= (a.keep[t0 + i] != 0 ? 1u : 0u) << i;
      }
      long long sum;
      const long long before = kept_all + block_excl(__popc(bits), part, &sum);
      if (t0 < a.N) a.kept[t0 >> 5] = make_uint2(static_cast<uint32_t>(before), bits);
      kept_all += sum;
    }
  }
  __syncthreads();
  long long tokens = 0, taken = 0;
  for (int base = 0; base < a.R; base += nt) {
    const int r = base + tid;
    const bool in = r < a.R;
    const int len = base == 0 ? len0 : in ? a.len[r] : 0, n = base == 0 ? new0 : in ? a.new_len[r] : 0;
    bool bad = len < 0 || n < 0;
    long long sum;
    const long long start = tokens + block_excl(bad ? 0 : n, part, &sum);
    tokens += sum;
    const long long end = start + (bad ? 0 : n);
    long long first = start, last = end;
    if (a.keep != nullptr) {
      bool unused;
      first = start < a.N ? kept_before(a, start, &unused) : kept_all;
      last = end < a.N ? kept_before(a, end, &unused) : kept_all;
    }
    const long long kept = last - first;
    const long long have = (static_cast<long long>(len) + a.page_size - 1) / a.page_size;
    const long long then = (len + kept + a.page_size - 1) / a.page_size;
    bad = bad || end > a.N || then > a.max_pages;
    const long long before = taken + block_excl(bad ? 0 : then - have, part, &sum);
    taken += sum;
    if (in) {
      a.req[r] = {len, static_cast<int32_t>(first), static_cast<int32_t>(kept), static_cast<int32_t>(before)};
      a.q_start[r] = static_cast<int32_t>(start);
      if (bad) s_bad = 1;
    }
  }
  __syncthreads();
  int err = SCFA_OK;
  if (s_bad || n_free < 0 || n_free > a.n_pages || tokens > a.N) err = SCFA_ERR_INVALID;
  else if (taken > n_free) err = SCFA_ERR_WORKSPACE;
  for (int r = tid; r < a.R; r += nt) {
    const PlanReq q = a.req[r];
    a.len_out[r] = q.len + (err == SCFA_OK ? q.kept : 0);
    if (err != SCFA_OK) a.q_start[r] = 0;
  }
  if (tid == 0) {
    a.q_start[a.R] = err == SCFA_OK ? static_cast<int32_t>(tokens) : 0;
    *a.free_before = n_free;
    *a.n_free_out = n_free - (err == SCFA_OK ? static_cast<int32_t>(taken) : 0);
    *a.status = err;
  }
  if (!fill) return;
  __syncthreads();
  for (int t = tid; t < a.N; t += nt) plan_token(a, t);
}

__global__ void __launch_bounds__(256) plan_fill_kernel(PlanArgs a) {
  grid_wait();
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t < a.N) plan_token(a, static_cast<int>(t));
}

// ---------------------------------------------------------------- append / read
struct RowArgs {
  const uint16_t *k, *v;
  uint16_t *k_out, *v_out;
  long long kt, kh, vt, vh;  // strides per token and head
  const int32_t* slot;
  long long rows;  // Hkv times N, rounded up to four
  int N, Hkv, page_size, log_ps;
  long long slots;  // slots of the cache
  uint8_t* cache;
};

// Eight threads per row (one token of one head), the four rows of a warp four
// tokens in a row of one head: tokens appended together mostly follow each
// other in a tile, and the V codes of four such tokens fill whole 32-byte
// sectors. Thread i takes D / 8 consecutive channels of K (D / 64 words) and
// the channels 32 g + 4 i + 0..3 of V, as the tile groups them, so every store
// is a whole word.
struct RowAt {
  long long tok;
  int head, i;
  bool in;
};
__device__ __forceinline__ RowAt row_at(const RowArgs& a) {
  const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const long long quad = row >> 2, four = quad / a.Hkv;
  RowAt r;
  r.tok = four * 4 + (row & 3);
  r.head = static_cast<int>(quad - four * a.Hkv);
  r.i = threadIdx.x & 7;
  r.in = r.tok < a.N;
  return r;
}

// The rows are read once and the codes written once; HBM and the issue slots
// (74% busy: 13.5 lane operations a value, of conversions, rounding and packing,
// but also of the row's place and of scales that its threads repeat) bound it
// alike. 16,384 rows of 8 heads and 128 channels (67 MB in, 18 MB out): 20 us,
// 4.2 TB/s, 63% of the copy rate. A group's largest magnitude is taken on the
// bits, two values at a time (a NaN is then larger than infinity and is seen);
// groups with a value that is not finite or beyond the largest scale take the
// careful way.
template <int D, bool F16>
__global__ void __launch_bounds__(256) append_kernel(RowArgs a) {
  using L = C4<D>;
  constexpr int W = D / 64;  // K words per thread
  constexpr int G = L::kG;
  const RowAt r = row_at(a);
  const int i = r.i;
  const long long slot = r.in ? a.slot[r.tok] : -1;
  const bool live = slot >= 0 && slot < a.slots;
  // every thread stays for the shuffles
  uint32_t kw[4 * W], vw[2 * G];
#pragma unroll
  for (int x = 0; x < 4 * W; ++x) kw[x] = 0;
#pragma unroll
  for (int x = 0; x < 2 * G; ++x) vw[x] = 0;
  if (live) {
    const uint4* ks = reinterpret_cast<const uint4*>(a.k + r.tok * a.kt + r.head * a.kh + i * (8 * W));
#pragma unroll
    for (int x = 0; x < W; ++x) {
      const uint4 u = ks[x];
      kw[4 * x] = u.x, kw[4 * x + 1] = u.y, kw[4 * x + 2] = u.z, kw[4 * x + 3] = u.w;
    }
    const uint16_t* vs = a.v + r.tok * a.vt + r.head * a.vh + 4 * i;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint2 u = *reinterpret_cast<const uint2*>(vs + 32 * g);
      vw[2 * g] = u.x, vw[2 * g + 1] = u.y;
    }
  }
  // bits of the largest magnitude of a group, K and V of up to four groups
  uint32_t kmax = 0;
#pragma unroll
  for (int x = 0; x < 4 * W; ++x) kmax = __vmaxu2(kmax, kw[x] & 0x7FFF7FFFu);
  // (a group of 32 channels of K lies in 32 / (D / 8) threads)
  kmax = __vmaxu2(kmax, __shfl_xor_sync(0xffffffffu, kmax, 1));
  if (W == 1) kmax = __vmaxu2(kmax, __shfl_xor_sync(0xffffffffu, kmax, 2));
  uint32_t vmax[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    vmax[g] = __vmaxu2(vw[2 * g] & 0x7FFF7FFFu, vw[2 * g + 1] & 0x7FFF7FFFu);
    vmax[g] = max(vmax[g] & 0xFFFFu, vmax[g] >> 16);
  }
#pragma unroll
  for (int g = 0; g < G; g += 2) {  // two groups a shuffle
    uint32_t m = vmax[g] | vmax[g + 1] << 16;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    vmax[g] = m & 0xFFFFu, vmax[g + 1] = m >> 16;
  }
  kmax = max(kmax & 0xFFFFu, kmax >> 16);
  // 64512 in bf16 and fp16: from here on codes would leave -7..7
  constexpr uint32_t kMost = F16 ? 0x7BE0u : 0x477Cu;
  bool careful = kmax > kMost;
#pragma unroll
  for (int g = 0; g < G; ++g) careful |= vmax[g] > kMost;
  if (__any_sync(0xffffffffu, careful)) {
    // cut to what the format holds, NaN to 0, and take the maxima again
    auto cut = [](uint32_t w) {
      const float2 f = c4_unpack<F16>(w);
      return c4_pack<F16>(c4_cut(f.x), c4_cut(f.y));
    };
    kmax = 0;
#pragma unroll
    for (int x = 0; x < 4 * W; ++x) {
      kw[x] = cut(kw[x]);
      kmax = __vmaxu2(kmax, kw[x] & 0x7FFF7FFFu);
    }
    kmax = __vmaxu2(kmax, __shfl_xor_sync(0xffffffffu, kmax, 1));
    if (W == 1) kmax = __vmaxu2(kmax, __shfl_xor_sync(0xffffffffu, kmax, 2));
    kmax = max(kmax & 0xFFFFu, kmax >> 16);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      vw[2 * g] = cut(vw[2 * g]), vw[2 * g + 1] = cut(vw[2 * g + 1]);
      uint32_t m = __vmaxu2(vw[2 * g] & 0x7FFF7FFFu, vw[2 * g + 1] & 0x7FFF7FFFu);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      vmax[g] = max(m & 0xFFFFu, m >> 16);
    }
  }
  if (!live) return;
  const int at = static_cast<int>(slot & (a.page_size - 1)), t = at & 15;
  uint8_t* tile = a.cache + c4_tile_base(slot >> a.log_ps, a.Hkv, r.head, a.page_size, at, L::kTileBytes);
  const uint32_t kb = c4_scale_byte(c4_unpack<F16>(kmax).x);
  const float kinv = c4_reciprocal(c4_scale(kb));
#pragma unroll
  for (int x = 0; x < W; ++x) {
    const int word = i * W + x, g = word >> 2, j = word & 3;
    // channels 2 y and 2 y + 1 of the word in bits 4 y and 4 y + 16; the codes' common high bits add up to a constant
    uint32_t c = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float2 f = c4_unpack<F16>(kw[4 * x + y]);
      c += (c4_code(f.x, kinv) << (4 * y)) + (c4_code(f.y, kinv) << (4 * y + 16));
    }
    *reinterpret_cast<uint32_t*>(tile + L::k_row(t) + (j * G + g) * 4) = c - 0x4B400000u * 0x1111u;
    if (j == 0) tile[L::kKScales + t * G + g] = static_cast<uint8_t>(kb);
  }
  uint32_t piece[G / 2], mine = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t b = c4_scale_byte(c4_unpack<F16>(vmax[g]).x);
    const float inv = c4_reciprocal(c4_scale(b));
    const float2 f = c4_unpack<F16>(vw[2 * g]), h = c4_unpack<F16>(vw[2 * g + 1]);
    const uint32_t c = c4_code(f.x, inv) + (c4_code(f.y, inv) << 4) + (c4_code(h.x, inv) << 8) +
                       (c4_code(h.y, inv) << 12);  // right in its low 16 bits
    if (g & 1) piece[g / 2] = __byte_perm(piece[g / 2], c, 0x5410);
    else piece[g / 2] = c;
    if (i == g) mine = b;
  }
  if (G == 4) *reinterpret_cast<uint2*>(tile + L::v_piece(t, i)) = make_uint2(piece[0], piece[G / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(tile + L::v_piece(t, i)) = piece[0];
  if (i < G) tile[L::kVScales + t * G + i] = static_cast<uint8_t>(mine);
}

// The reverse, with the same threads: a thread writes the channels it read
// there. 32,768 rows of 8 heads and 128 channels (36 MB in, 134 MB out): 32 us,
// 5.3 TB/s, 79% of the copy rate, issue slots 65% busy, 10.5 lane operations a value.
template <int D, bool F16>
__global__ void __launch_bounds__(256) read_kernel(RowArgs a) {
  using L = C4<D>;
  constexpr int W = D / 64;
  constexpr int G = L::kG;
  const RowAt r = row_at(a);
  if (!r.in) return;
  const int i = r.i;
  const long long slot = a.slot[r.tok];
  uint16_t* ko = a.k_out + r.tok * a.kt + r.head * a.kh + i * (8 * W);
  uint16_t* vo = a.v_out + r.tok * a.vt + r.head * a.vh + 4 * i;
  if (slot < 0 || slot >= a.slots) {
#pragma unroll
    for (int x = 0; x < W; ++x) reinterpret_cast<uint4*>(ko)[x] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int g = 0; g < G; ++g) *reinterpret_cast<uint2*>(vo + 32 * g) = make_uint2(0u, 0u);
    return;
  }
  const int at = static_cast<int>(slot & (a.page_size - 1)), t = at & 15;
  const uint8_t* tile = a.cache + c4_tile_base(slot >> a.log_ps, a.Hkv, r.head, a.page_size, at, L::kTileBytes);
  uint32_t kc[W], ks[W], vc[G / 2];
#pragma unroll
  for (int x = 0; x < W; ++x) {
    const int word = i * W + x, g = word >> 2, j = word & 3;
    kc[x] = *reinterpret_cast<const uint32_t*>(tile + L::k_row(t) + (j * G + g) * 4);
    ks[x] = tile[L::kKScales + t * G + g];
  }
  uint32_t vs;  // the scale bytes of the groups
  if (G == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(tile + L::v_piece(t, i));
    vc[0] = u.x, vc[G / 2 - 1] = u.y;
    vs = *reinterpret_cast<const uint32_t*>(tile + L::kVScales + t * G);
  } else {
    vc[0] = *reinterpret_cast<const uint32_t*>(tile + L::v_piece(t, i));
    vs = *reinterpret_cast<const uint16_t*>(tile + L::kVScales + t * G);
  }
  // a code's bits under the exponent of 2^23 are 2^23 + (c + 8)
  auto value = [](uint32_t c, float s) { return (__uint_as_float(c | 0x4B000000u) - (8388608.f + 8.f)) * s; };
#pragma unroll
  for (int x = 0; x < W; ++x) {
    const float s = c4_scale(ks[x]);
    uint32_t w[4];
#pragma unroll
    for (int y = 0; y < 4; ++y)
      w[y] = c4_pack<F16>(value(kc[x] >> (4 * y) & 15u, s), value(kc[x] >> (4 * y + 16) & 15u, s));
    reinterpret_cast<uint4*>(ko)[x] = make_uint4(w[0], w[1], w[2], w[3]);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t c = vc[g / 2] >> (16 * (g & 1));
    const float s = c4_scale(vs >> (8 * g) & 255u);
    *reinterpret_cast<uint2*>(vo + 32 * g) = make_uint2(c4_pack<F16>(value(c & 15u, s), value(c >> 4 & 15u, s)),
                                                        c4_pack<F16>(value(c >> 8 & 15u, s), value(c >> 12 & 15u, s)));
  }
}

constexpr int kPlanOneCta = 4096;  // tokens one CTA fills itself

struct PlanWs {
  size_t free_before = sizeof(WsHeader), req = sizeof(WsHeader) + 256, kept = 0, total = 0;
};
bool plan_ws_layout(int N, int R, PlanWs* w) {
  if (N < 1 || R < 1) return false;
  w->kept = align_up(w->req + sizeof(PlanReq) * static_cast<size_t>(R), 256);
  w->total = align_up(w->kept + sizeof(uint2) * (static_cast<size_t>(N) / 32 + 1), 256);
  return true;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// sizes and pointers common to append and read
scfa_status check_rows(const void* k, long long kt, long long kh, const void* v, long long vt, long long vh,
                       const int32_t* slot, int N, int Hkv, int D, int dtype, const void* cache, int page_size,
                       int n_pages) {
  if (!k || !v || !slot || !cache) return SCFA_ERR_INVALID;
  if (N < 1 || Hkv < 1 || n_pages < 1) return SCFA_ERR_INVALID;
  if (dtype != SCFA_DTYPE_BF16 && dtype != SCFA_DTYPE_F16) return SCFA_ERR_UNSUPPORTED;
  if ((D != 64 && D != 128) || !c4_page_size_ok(page_size)) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(n_pages) * page_size >= (1ll << 31)) return SCFA_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return SCFA_ERR_INVALID;
  if ((kt | kh | vt | vh) & 7) return SCFA_ERR_INVALID;
  return SCFA_OK;
}

RowArgs row_args(long long kt, long long kh, long long vt, long long vh, const int32_t* slot, int N, int Hkv,
                 int page_size, int n_pages, const uint8_t* cache) {
  RowArgs a = {};
  a.kt = kt, a.kh = kh, a.vt = vt, a.vh = vh;
  a.slot = slot;
  a.N = N;
  a.rows = (static_cast<long long>(N) + 3) / 4 * 4 * Hkv;
  a.Hkv = Hkv;
  a.page_size = page_size;
  while ((1 << a.log_ps) < page_size) ++a.log_ps;
  a.slots = static_cast<long long>(n_pages) * page_size;
  a.cache = const_cast<uint8_t*>(cache);
  return a;
}

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" {

size_t scfa_cache4_page_bytes(int page_size, int D) {
  if ((D != 64 && D != 128) || !c4_page_size_ok(page_size)) return 0;
  return static_cast<size_t>(page_size) * (D + D / 16);
}

size_t scfa_cache4_plan_workspace_size(int N, int R) {
  PlanWs w;
  return plan_ws_layout(N, R, &w) ? w.total : 0;
}

scfa_status scfa_cache4_plan(const int32_t* len, const int32_t* new_len, const uint8_t* keep,
                             const int32_t* free_pages, const int32_t* n_free, int32_t* table, int N, int R,
                             int max_pages, int page_size, int n_pages, int32_t* len_out, int32_t* n_free_out,
                             int32_t* q_start, int32_t* slot, int32_t* vis, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!len || !new_len || !free_pages || !n_free || !table || !len_out || !n_free_out || !q_start || !slot || !vis ||
      !ws)
    return SCFA_ERR_INVALID;
  if (N < 1 || R < 1 || max_pages < 1 || n_pages < 1) return SCFA_ERR_INVALID;
  if (!c4_page_size_ok(page_size)) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(n_pages) * page_size >= (1ll << 31) ||
      static_cast<long long>(max_pages) * page_size > kC4MostTokens)
    return SCFA_ERR_UNSUPPORTED;
  PlanWs w;
  plan_ws_layout(N, R, &w);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < w.total) return SCFA_ERR_WORKSPACE;
  char* p = static_cast<char*>(ws);
  const PlanArgs a = {len, new_len, keep, free_pages, n_free, table, N, R, max_pages, page_size, n_pages,
                      len_out, n_free_out, q_start, slot, vis, reinterpret_cast<int*>(p),
                      reinterpret_cast<int32_t*>(p + w.free_before), reinterpret_cast<PlanReq*>(p + w.req),
                      reinterpret_cast<uint2*>(p + w.kept)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int fill = N <= kPlanOneCta;
  const int items = fill ? N : keep ? N / 32 + 1 : 1, most = items > R ? items : R;  // of the longest loop
  const int threads = most >= 1024 ? 1024 : (most + 31) / 32 * 32;
  plan_kernel<<<1, threads, 0, st>>>(a, fill);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && !fill) e = launch_behind(plan_fill_kernel, dim3(N / 256 + 1), 256, st, a);
  return e == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
}

scfa_status scfa_cache4_append(const uint16_t* k, long long k_token, long long k_head, const uint16_t* v,
                               long long v_token, long long v_head, const int32_t* slot, int N, int Hkv, int D,
                               int dtype, uint8_t* cache, int page_size, int n_pages, void* stream) {
  const scfa_status s =
      check_rows(k, k_token, k_head, v, v_token, v_head, slot, N, Hkv, D, dtype, cache, page_size, n_pages);
  if (s != SCFA_OK) return s;
  RowArgs a = row_args(k_token, k_head, v_token, v_head, slot, N, Hkv, page_size, n_pages, cache);
  a.k = k, a.v = v;
  const long long grid = (a.rows + 31) / 32;
  if (grid > INT_MAX) return SCFA_ERR_UNSUPPORTED;
  const bool h = dtype == SCFA_DTYPE_F16;
  auto kern = D == 64 ? (h ? append_kernel<64, true> : append_kernel<64, false>)
                      : (h ? append_kernel<128, true> : append_kernel<128, false>);
  kern<<<static_cast<int>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
}

scfa_status scfa_cache4_read(const uint8_t* cache, int page_size, int n_pages, const int32_t* slot, int N, int Hkv,
                             int D, int dtype, uint16_t* k, long long k_token, long long k_head, uint16_t* v,
                             long long v_token, long long v_head, void* stream) {
  const scfa_status s =
      check_rows(k, k_token, k_head, v, v_token, v_head, slot, N, Hkv, D, dtype, cache, page_size, n_pages);
  if (s != SCFA_OK) return s;
  if (c4_rows_overlap(k_token, k_head, N, Hkv, D) || c4_rows_overlap(v_token, v_head, N, Hkv, D))
    return SCFA_ERR_INVALID;
  RowArgs a = row_args(k_token, k_head, v_token, v_head, slot, N, Hkv, page_size, n_pages, cache);
  a.k_out = k, a.v_out = v;
  const long long grid = (a.rows + 31) / 32;
  if (grid > INT_MAX) return SCFA_ERR_UNSUPPORTED;
  const bool h = dtype == SCFA_DTYPE_F16;
  auto kern = D == 64 ? (h ? read_kernel<64, true> : read_kernel<64, false>)
                      : (h ? read_kernel<128, true> : read_kernel<128, false>);
  kern<<<static_cast<int>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
}

}  // extern "C"
