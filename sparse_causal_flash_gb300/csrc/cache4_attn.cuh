// What the two attention kernels over the paged 4-bit cache share: how the
// work is cut, the walk of a CTA over its piece, the copies of a unit's pages,
// and the join of what was cut.
//
// An item is a block of query rows (token, head) of one request that share a
// key head; its cached tokens are walked in units of 128. The units of all
// items, in one long line, are cut into equal pieces, one per CTA of a grid
// that fills the GPU: a ragged batch and one long request are spread alike.
// An item that falls into several pieces leaves partial rows (O, m, l in
// fp32), which the join kernel sums in the order of the tokens, so results do
// not depend on scheduling.
#pragma once

#include <climits>

#include "cache4.cuh"
#include "internal.h"

namespace scfa {

constexpr int kCh = 128;  // tokens per unit
constexpr int kChTiles = kCh / kC4Tile;
// Running maximum before any key: below every score there can be (2^120 in log2 units), and finite, so that differences
// stay defined. Scores are rounded to fp32 before the maximum comes off (a multiplication and an addition, no fma):
// past 2^24, where a step of fp32 is more than a softmax is wide, the largest then still has a weight near one.
constexpr float kNoMax = -3e38f;

// What a CTA reports, and the item that begins in its piece and goes on behind
// it. One per CTA, written by every call.
struct C4Desc {
  int err;    // SCFA_OK or the CTA's first error
  int parts;  // > 0: the item ends `parts` CTAs later
  int tok0, rows, row0, head;
  int pad[2];
};

struct C4AttnArgs {
  const uint16_t* q;
  long long qt, qh;
  const uint8_t* cache;
  int page_size, log_ps, n_pages;
  const int32_t* table;
  int max_pages;
  const int32_t *q_start, *vis;
  int N, R, Hq, Hkv, G;
  float factor;  // scale * log2(e)
  uint16_t* o;
  long long ot, oh;
  float* lse;
  int* status;
  C4Desc* desc;
  float* part;  // [cta][2][rows][D]: the tail of an item begun before the piece; an item that goes on behind it
  float* ml;    // [cta][2][rows][2]
  int stall;
  // 16, 128 and fp16 512 twice, as values the compiler does not know: a
  // multiplication then stays on the FMA pipe (a shift-and-add is ALU work,
  // which is what is short), and an AND-OR stays one instruction
  uint32_t k16, k128, magic;
};

// What a unit's stage holds.
struct C4Stage {
  int tok0, rows, row0, head;  // first token of the request, its rows, first row of the item, key head
  int base;                    // position of the unit's first token
  int tiles;                   // bit t: tile t was copied
  int flags;
  int seen;                    // tokens that the item's last row sees
  int qslot;                   // where its queries are
  int pad[3];
};
// of the item, in this piece: first and last unit; it began before, it goes on behind
enum { kFirst = 1, kLast = 2, kOpenStart = 4, kOpenEnd = 8 };

__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Eight codes of a word, four in each half, as fp16 c s (exact): pairs of bits
// 0-3 and 16-19, 4-7 and 20-23, 8-11 and 24-27, 12-15 and 28-31. sc2: twice
// the scales of the two halves. The bits of c + 8 under the exponent of 512
// are 512 + (c + 8) / 2 at the bottom and 512 + 8 (c + 8) four bits up.
__device__ __forceinline__ uint4 c4_unpack8(uint32_t x, uint32_t sc2, uint32_t magic) {
  const uint32_t y = x >> 8, sc_hi = mul_f16x2(sc2, 0x2C002C00u);  // s / 8
  const uint32_t lo = 0xE008E008u, hi = 0xE080E080u;               // -516, -576
  return make_uint4(mul_f16x2(add_f16x2(and_or(x, 0x000F000Fu, magic), lo), sc2),
                    mul_f16x2(add_f16x2(and_or(x, 0x00F000F0u, magic), hi), sc_hi),
                    mul_f16x2(add_f16x2(and_or(y, 0x000F000Fu, magic), lo), sc2),
                    mul_f16x2(add_f16x2(and_or(y, 0x00F000F0u, magic), hi), sc_hi));
}

// The rare part of a wait, out of line: the roles of a CTA share the schedulers'
// instruction caches.
static __device__ __noinline__ bool c4_gave_up(uint32_t t0, volatile int* abort_flag, int* status) {
  if (*abort_flag) return true;
  if (static_cast<uint32_t>(global_timer_ns()) - t0 <= static_cast<uint32_t>(kWaitLimitNs)) return false;
  raise_status(status, SCFA_ERR_TIMEOUT);
  *abort_flag = 1;
  return true;
}
// Bounded wait of a whole warp, whose lanes go on, or give up, together: looks at
// the abort flag and the clock once in 16 polls.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    const uint32_t t0 = static_cast<uint32_t>(global_timer_ns());
    uint32_t polls = 0;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
      if ((++polls & 15u) == 0 && __any_sync(0xffffffffu, c4_gave_up(t0, abort_flag, status))) return false;
  }
  return true;
}

// a / b, in 32 bits where they hold it
__device__ __forceinline__ long long c4_div(long long a, int b) {
  return a >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Row blocks of a request and the units of one of them.
struct C4Req {
  int tok0, rows, blocks;
};
template <int ROWS>
__device__ __forceinline__ C4Req c4_request(const C4AttnArgs& a, int r) {
  C4Req q;
  // (indices are clamped: nothing is read out of bounds whatever q_start holds)
  q.tok0 = min(max(a.q_start[r], 0), a.N);
  const int end = min(max(a.q_start[r + 1], q.tok0), a.N);
  q.rows = (end - q.tok0) * a.G;
  q.blocks = (q.rows + ROWS - 1) / ROWS;
  return q;
}
// tokens that the last row of block b sees (vis does not decrease within a request)
template <int ROWS>
__device__ __forceinline__ int c4_seen(const C4AttnArgs& a, const C4Req& q, int b) {
  const int last = min((b + 1) * ROWS, q.rows) - 1;
  const long long cap = static_cast<long long>(a.max_pages) << a.log_ps;
  return static_cast<int>(min(cap, static_cast<long long>(max(0, a.vis[q.tok0 + last / a.G]))));
}
__device__ __forceinline__ int c4_chunks(int seen) { return max(1, (seen + kCh - 1) / kCh); }

// The piece of this CTA: its units, and the request in which it begins.
struct C4Span {
  long long per, u0;  // units per piece; first unit
  long long prefix;   // units before the request
  int units, req;
  C4Req q;   // that request,
  int seen;  // and, if it is of one block, the tokens it sees
};
template <int THREADS>
struct C4SpanSmem {
  long long sum[THREADS / 32], prefix;
  int req;
};
// Up to 32 requests: by each warp for itself, a lane per request. Nothing else
// can start before this has, so it waits for memory once: the count that a
// lane's request sees is fetched with the request's bounds, at the place where
// it is if every request brings one token.
template <int ROWS>
__device__ __forceinline__ bool c4_span_warp(const C4AttnArgs& a, C4Span& span) {
  const int lane = threadIdx.x & 31;
  const bool in = lane < a.R;
  const int guess = a.vis[min(lane, a.N - 1)];
  C4Req q = {0, 0, 0};
  if (in) q = c4_request<ROWS>(a, lane);
  long long mine = 0;
  int seen = 0;
  if (q.blocks == 1) {
    const int tok = q.tok0 + (q.rows <= a.G ? 0 : (q.rows - 1) / a.G);
    const long long cap = static_cast<long long>(a.max_pages) << a.log_ps;
    seen = static_cast<int>(min(cap, static_cast<long long>(max(0, tok == lane ? guess : a.vis[tok]))));
    mine = c4_chunks(seen);
  }
  uint32_t big = __ballot_sync(0xffffffffu, q.blocks > 1);
  while (big) {  // requests of several blocks: the warp together
    const int src = __ffs(big) - 1;
    big &= big - 1;
    C4Req p;
    p.tok0 = __shfl_sync(0xffffffffu, q.tok0, src);
    p.rows = __shfl_sync(0xffffffffu, q.rows, src);
    p.blocks = __shfl_sync(0xffffffffu, q.blocks, src);
    long long x = 0;
    for (int b = lane; b < p.blocks; b += 32) x += c4_chunks(c4_seen<ROWS>(a, p, b));
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == src) mine = x;
  }
  mine *= a.Hkv;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  span.per = c4_div(total + gridDim.x - 1, gridDim.x);
  span.u0 = span.per * blockIdx.x;
  const long long u1 = min(total, span.u0 + span.per);
  if (span.u0 >= u1) return false;
  span.units = static_cast<int>(u1 - span.u0);
  const int src = __ffs(__ballot_sync(0xffffffffu, span.u0 < upto)) - 1;
  span.req = src;
  span.prefix = __shfl_sync(0xffffffffu, upto - mine, src);
  span.q.tok0 = __shfl_sync(0xffffffffu, q.tok0, src);
  span.q.rows = __shfl_sync(0xffffffffu, q.rows, src);
  span.q.blocks = __shfl_sync(0xffffffffu, q.blocks, src);
  span.seen = __shfl_sync(0xffffffffu, seen, src);
  return true;
}
// By the whole CTA (the caller's barrier comes behind); false: an empty piece.
template <int ROWS, int THREADS>
__device__ __forceinline__ bool c4_span(const C4AttnArgs& a, C4SpanSmem<THREADS>& sm, C4Span& span) {
  if (a.R <= 32) return c4_span_warp<ROWS>(a, span);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  auto request_units = [&](int r) {
    C4Req q = {0, 0, 0};
    if (r < a.R) q = c4_request<ROWS>(a, r);
    long long sum = 0;
    if (q.blocks <= 4) {
      for (int b = 0; b < q.blocks; ++b) sum += c4_chunks(c4_seen<ROWS>(a, q, b));
    }
    // requests of many blocks: the warp together
    uint32_t big = __ballot_sync(0xffffffffu, q.blocks > 4);
    while (big) {
      const int src = __ffs(big) - 1;
      big &= big - 1;
      C4Req p;
      p.tok0 = __shfl_sync(0xffffffffu, q.tok0, src);
      p.rows = __shfl_sync(0xffffffffu, q.rows, src);
      p.blocks = __shfl_sync(0xffffffffu, q.blocks, src);
      long long x = 0;
      for (int b = lane; b < p.blocks; b += 32) x += c4_chunks(c4_seen<ROWS>(a, p, b));
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == src) sum = x;
    }
    return sum * a.Hkv;
  };
  // inclusive sum over the block; *total gets the sum
  auto block_incl = [&](long long x, long long* total) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm.sum[w] = x;
    __syncthreads();
    long long all = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i == w) x += all;
      all += sm.sum[i];
    }
    *total = all;
    return x;
  };
  long long total = 0, mine = 0, upto = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    long long sum;
    mine = request_units(base + tid);
    upto = block_incl(mine, &sum);
    total += sum;
  }
  span.per = c4_div(total + gridDim.x - 1, gridDim.x);
  span.u0 = span.per * blockIdx.x;
  const long long u1 = min(total, span.u0 + span.per);
  if (span.u0 >= u1) return false;
  span.units = static_cast<int>(u1 - span.u0);
  long long before = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    long long sum = total;
    if (a.R > THREADS) {
      mine = request_units(base + tid);
      upto = before + block_incl(mine, &sum);
    }
    if (span.u0 < upto && span.u0 >= upto - mine) {
      sm.req = base + tid;
      sm.prefix = upto - mine;
    }
    before += sum;
    if (span.u0 < before) break;  // (uniform)
  }
  __syncthreads();
  span.req = sm.req;
  span.prefix = sm.prefix;
  span.q = c4_request<ROWS>(a, span.req);
  span.seen = span.q.blocks == 1 ? c4_seen<ROWS>(a, span.q, 0) : 0;
  return true;
}

// The walk of one warp over the units of the piece.
template <int ROWS>
struct C4Walk {
  C4Req q;
  int r, b, h, ch, seen, chunks;  // request, row block, key head, unit of the item
  __device__ __forceinline__ void begin(const C4AttnArgs& a, const C4Span& span, int lane) {
    r = span.req;
    b = 0;
    q = span.q;
    long long rem = span.u0 - span.prefix;
    for (; q.blocks > 1; b += 32) {  // the block: 32 at a time
      const int mb = b + lane;
      const int c = mb < q.blocks ? c4_chunks(c4_seen<ROWS>(a, q, mb)) : 0;
      const long long own = static_cast<long long>(c) * a.Hkv;
      long long x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, rem < x);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b += src;
        rem -= __shfl_sync(0xffffffffu, x - own, src);
        break;
      }
      rem -= __shfl_sync(0xffffffffu, x, 31);
      if (b + 32 >= q.blocks) break;  // (does not happen: the piece begins in this request)
    }
    seen = q.blocks > 1 ? c4_seen<ROWS>(a, q, b) : span.seen;
    chunks = c4_chunks(seen);
    h = static_cast<int>(c4_div(rem, chunks));
    ch = static_cast<int>(rem - static_cast<long long>(h) * chunks);
  }
  __device__ __forceinline__ void next(const C4AttnArgs& a, bool more) {
    if (++ch < chunks) return;
    ch = 0;
    if (++h < a.Hkv) return;
    h = 0;
    if (!more) return;
    if (++b == q.blocks) {
      b = 0;
      do {
        q = c4_request<ROWS>(a, ++r);
      } while (q.blocks == 0 && r + 1 < a.R);
    }
    seen = c4_seen<ROWS>(a, q, b);
    chunks = c4_chunks(seen);
  }
  // the stage of unit u of the piece, all but its tiles and query slot; by one lane, which also notes an item that
  // begins here and goes on behind the piece
  __device__ __forceinline__ void describe(const C4Span& span, int u, C4Desc* desc, C4Stage& d) const {
    const bool last = ch + 1 == chunks, began = ch <= u, goes_on = !last && u + 1 == span.units;
    d.tok0 = q.tok0;
    d.rows = q.rows;
    d.row0 = b * ROWS;
    d.head = h;
    d.base = ch * kCh;
    d.seen = seen;
    d.flags = (ch == 0 || u == 0 ? kFirst : 0) | (last || goes_on ? kLast : 0) | (began ? 0 : kOpenStart) |
              (goes_on ? kOpenEnd : 0);
    if (goes_on && began) {
      const long long end = span.u0 + u + (chunks - 1 - ch);  // the item's last unit
      desc->parts = static_cast<int>(c4_div(end, static_cast<int>(span.per)) - blockIdx.x);
      desc->tok0 = q.tok0;
      desc->rows = q.rows;
      desc->row0 = b * ROWS;
      desc->head = h;
    }
  }
};

// The pages of a unit and their copies, by one warp: a lane for each page that
// the unit's tokens lie in (or one for the part of a longer page).
struct C4Pages {
  int have_r = -1, have_p = 0, page = -1;  // the 32 pieces whose pages the lanes hold
  int psub, npc;                           // tokens of a unit per page; pages
  int tiles, pg;                           // this lane's piece of the unit
  __device__ __forceinline__ explicit C4Pages(const C4AttnArgs& a) : psub(min(a.page_size, kCh)), npc(kCh / psub) {}
  // returns the mask of the tiles to copy; a page id out of range has none and is reported
  template <int ROWS>
  __device__ __forceinline__ uint32_t look_up(const C4AttnArgs& a, const C4Walk<ROWS>& w, int lane, int* err) {
    const int p0 = w.ch * npc;
    if (have_r != w.r || p0 < have_p || p0 + npc > have_p + 32) {
      have_r = w.r;
      have_p = p0;
      const long long pos = static_cast<long long>(p0 + lane) * psub;
      page = -1;
      if (pos < (static_cast<long long>(a.max_pages) << a.log_ps))
        page = a.table[static_cast<long long>(w.r) * a.max_pages + (pos >> a.log_ps)];
    }
    pg = __shfl_sync(0xffffffffu, page, (p0 - have_p + lane) & 31);
    const int n = min(kCh, w.seen - w.ch * kCh) - lane * psub;  // tokens of this lane's piece
    tiles = lane < npc && n > 0 ? (min(n, psub) + kC4Tile - 1) / kC4Tile : 0;
    if (tiles > 0 && (pg < 0 || pg >= a.n_pages)) {
      raise_status(err, SCFA_ERR_INVALID);
      tiles = 0;
    }
    return __reduce_or_sync(0xffffffffu, tiles > 0 ? ((1u << tiles) - 1u) << (lane * (psub / kC4Tile)) : 0u);
  }
  template <int D, int ROWS>
  __device__ __forceinline__ void copy(const C4AttnArgs& a, const C4Walk<ROWS>& w, int lane, uint8_t* dst,
                                       uint64_t* bar) const {
    if (tiles == 0) return;
    constexpr int TB = C4<D>::kTileBytes;
    const long long pos = static_cast<long long>(w.ch * npc + lane) * psub;
    const uint8_t* src =
        a.cache + c4_tile_base(pg, a.Hkv, w.h, a.page_size, static_cast<int>(pos & (a.page_size - 1)), TB);
    bulk_load(dst + lane * (psub / kC4Tile) * TB, src, tiles * TB, bar);
  }
};

// cache4_wide.cu: blocks of rp = 32, 64 or 128 query rows, one CTA per SM
cudaError_t launch_cache4_wide(int D, bool f16, int rp, int grid, const C4AttnArgs& a, cudaStream_t st);

namespace {
// Joins the partial rows of the items that were cut, in the order of their
// chunks, and gathers the CTAs' errors. A CTA per eight or 16 rows of a piece,
// the one in which an item begins. Lanes first weigh the parts, then each takes
// four channels of every part, kFly parts at a time. Few rows (long items, up to
// hundreds of parts): two warps per row, each for half the parts. Blocks of 32
// rows and more have few parts each and there are many of them: one warp per
// row and fewer registers, so that more CTAs are resident. Latency bound: the
// descriptor, then maxima and parts. 57 parts of 8 rows for each of 8 heads
// 7 us, two or three parts of 128 rows for each of 152 pieces 9 us.
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
template <int ROWS>
struct C4Join {
  static constexpr int kWarpsPerRow = ROWS <= 16 ? 2 : 1, kFly = ROWS <= 16 ? 8 : 4, kCtas = ROWS <= 16 ? 2 : 3;
  static constexpr int kRows = kJoinWarps / kWarpsPerRow;  // per CTA
};
template <int D, bool F16, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, C4Join<ROWS>::kCtas) cache4_join_kernel(C4AttnArgs a, int n_desc) {
  using J = C4Join<ROWS>;
  __shared__ float4 s_o[J::kRows][32];
  __shared__ float s_l[J::kRows];
  __shared__ int s_err[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  grid_wait();
  const C4Desc d = a.desc[blockIdx.x];
  if (blockIdx.x + blockIdx.y == 0) {
    int err = 0;
    for (int i = tid; i < n_desc; i += kJoinThreads) err = max(err, a.desc[i].err);
    err = __reduce_max_sync(0xffffffffu, err);
    if (lane == 0) s_err[w] = err;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < kJoinWarps; ++i) err = max(err, s_err[i]);
      *a.status = err;
    }
  }
  if (d.parts <= 0 || d.row0 + static_cast<int>(blockIdx.y) * J::kRows >= d.rows) return;
  constexpr int LPP = D / 4;     // lanes per part
  constexpr int PPW = 32 / LPP;  // parts side by side in a warp
  const int n = d.parts + 1, sub = lane / LPP, ch0 = lane % LPP * 4;
  const int half = J::kWarpsPerRow == 2 ? w & 1 : 0, mid = J::kWarpsPerRow == 2 ? (n + 1) / 2 : n;
  const int i0 = half ? mid : 0, i1 = half ? n : mid, slot = w / J::kWarpsPerRow;
  const int row = blockIdx.y * J::kRows + slot;
  const bool in = d.row0 + row < d.rows;
  // index of part i of the row: [cta][2][ROWS], below 2^31
  auto at = [&](int i) { return ((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + row; };
  float mt = kNoMax, lt = 0.f;
  float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f), v[J::kFly / PPW];
  const float* const part = a.part + ch0;
  auto load = [&](int i) {  // parts i to i + kFly - 1
#pragma unroll
    for (int y = 0; y < J::kFly / PPW; ++y)
      v[y] = *reinterpret_cast<const float4*>(part + at(min(i + y * PPW + sub, i1 - 1)) * D);
  };
  if (in) {
    load(i0);  // (under the wait for the maxima)
    for (int i = lane; i < n; i += 32) mt = fmaxf(mt, a.ml[2 * at(i)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    for (int base = i0; base < i1; base += 32) {
      float f = 0.f;  // weight of part base + lane
      if (base + lane < i1) {
        const float2 ml = *reinterpret_cast<const float2*>(a.ml + 2 * at(base + lane));
        f = ex2_approx(ml.x - mt);
        lt = fmaf(ml.y, f, lt);
      }
      const int cnt = min(32, i1 - base);
      for (int i = 0; i < cnt; i += J::kFly) {
        if (base + i != i0) load(base + i);
#pragma unroll
        for (int y = 0; y < J::kFly / PPW; ++y) {
          const float fi = __shfl_sync(0xffffffffu, f, i + y * PPW + sub);  // 0 behind the last part
          o4.x = fmaf(v[y].x, fi, o4.x), o4.y = fmaf(v[y].y, fi, o4.y);
          o4.z = fmaf(v[y].z, fi, o4.z), o4.w = fmaf(v[y].w, fi, o4.w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
    if (PPW == 2) {
      o4.x += __shfl_xor_sync(0xffffffffu, o4.x, 16), o4.y += __shfl_xor_sync(0xffffffffu, o4.y, 16);
      o4.z += __shfl_xor_sync(0xffffffffu, o4.z, 16), o4.w += __shfl_xor_sync(0xffffffffu, o4.w, 16);
    }
  }
  if (J::kWarpsPerRow == 2) {
    if (half) {
      s_o[slot][lane] = o4;
      if (lane == 0) s_l[slot] = lt;
    }
    __syncthreads();
    if (half) return;
    const float4 z = s_o[slot][lane];
    o4.x += z.x, o4.y += z.y, o4.z += z.z, o4.w += z.w;
    lt += s_l[slot];
  }
  if (in) {
    const int grow = d.row0 + row, tok = d.tok0 + grow / a.G, head = d.head * a.G + grow % a.G;
    const float inv = lt != 0.f ? 1.f / lt : 0.f;
    if (sub == 0)
      *reinterpret_cast<uint2*>(a.o + tok * a.ot + head * a.oh + ch0) =
          make_uint2(c4_pack<F16>(o4.x * inv, o4.y * inv), c4_pack<F16>(o4.z * inv, o4.w * inv));
    if (lane == 0)
      a.lse[static_cast<long long>(tok) * a.Hq + head] =
          lt != 0.f ? (mt + log2f(lt)) * 0.69314718055994531f : -INFINITY;
  }
}

// The main kernel (its dynamic shared memory allowed once per device) and
// behind it the join, whose launch hides under the main kernel's end.
template <int D, bool F16, int ROWS, typename Kernel>
cudaError_t launch_and_join(Kernel kern, int grid, int threads, size_t smem, const C4AttnArgs& a, cudaStream_t st) {
  static bool allowed[64] = {};  // by device; setting it twice does no harm
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  kern<<<grid, threads, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_behind(cache4_join_kernel<D, F16, ROWS>,
                       dim3(grid, (ROWS + C4Join<ROWS>::kRows - 1) / C4Join<ROWS>::kRows), kJoinThreads, st, a, grid);
}

}  // namespace
}  // namespace scfa
