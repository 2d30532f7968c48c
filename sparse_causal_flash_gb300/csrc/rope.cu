// Rotary positions of query and key rows, with the root-mean-square norm that may stand before them, and the gradients.
//
// A row x of D channels at position p: with a norm, n = x / sqrt(mean(x^2) + eps) and x becomes n w. Of the first `rot`
// channels pair i turns by p f[i] radians: (a, b) -> factor (a cos - b sin, b cos + a sin). A rotation's transpose turns
// back, so with g = the gradient turned back (times factor), dw = sum over rows of g n and
// dx = (g w - n mean(g w n)) / sqrt(mean(x^2) + eps).
//
// Angles. f[i] comes as a whole number F of 2^-64 turns, so p F mod 2^64 is the angle modulo one turn with no error at
// all; its high 32 bits (2^-32 of a turn) become an fp32 angle in [-pi, pi) for the hardware's sine and cosine (error
// below 2^-20), below the rounding of the 16-bit rows. With fp32 angles position 10^6 would be off by 0.06 radians.
//
// One row is held by D / 16 threads, each with two 16-byte pieces such that both halves of its eight pairs are its own:
// a norm is a few shuffles, and a row may be turned in place. What bounds it is HBM: each row is read once and written
// once (gradients with a norm: two read, one written). A thread turns up to four heads of a token with one set of sines
// (they cost 100 lane operations, a row's other work some 80), all loads before the first use.
#include "cache4.cuh"
#include "internal.h"

namespace scfa {
namespace {

constexpr int kRopeThreads = 256, kRopeStages = 2;
enum { kHalf = 0, kInterleaved = 1, kHalfOdd = 2 };  // kHalfOdd: halves that do not fall on 16-byte pieces

struct RopeSide {
  const uint16_t *x, *dy;  // forward: x only; backward without a norm: the gradient as x
  uint16_t* y;
  long long xt, xh, dyt, dyh, yt, yh;
  const float* w;
  float* dw;
  int H, slices, blocks;  // heads; units per token; CTAs of this side
};
struct RopeArgs {
  RopeSide side[2];
  const int32_t* pos;
  const int32_t* count;  // null, or how many of the N tokens there are
  const uint64_t* table;
  float* part;  // [CTA][D] partial dw
  int N, rot;
  float factor, eps, turn;  // turn: +-2 pi / 2^32
};

__device__ __forceinline__ int rope_tokens(const RopeArgs& g) { return g.count ? max(0, min(g.N, __ldg(g.count))) : g.N; }

// The eight pairs of thread t of a row: slot(i) numbers them, 0 .. rot / 2 are turned; a(i), b(i) are their channels.
template <int D, int KIND>
struct RopeMap {
  int t, rot;
  __device__ __forceinline__ int piece(int j) const {  // 16-byte piece j of the thread's two
    constexpr int T = D / 16;
    if (KIND == kInterleaved) return t + j * T;
    const int n = rot >> 4;  // pieces of a half
    return t < n ? t + j * n : 2 * t + j;
  }
  __device__ __forceinline__ int slot(int i) const {
    constexpr int T = D / 16;
    if (KIND == kInterleaved) return piece(i >> 2) * 4 + (i & 3);
    if (KIND == kHalfOdd) return t + i * T;
    return t * 8 + i;
  }
  __device__ __forceinline__ int a(int i) const {
    const int s = slot(i), h = rot >> 1;
    if (KIND == kInterleaved) return 2 * s;
    if (KIND == kHalfOdd) return s < h ? s : 2 * s;
    return piece(0) * 8 + i;
  }
  __device__ __forceinline__ int b(int i) const {
    const int s = slot(i), h = rot >> 1;
    if (KIND == kInterleaved) return 2 * s + 1;
    if (KIND == kHalfOdd) return s < h ? s + h : 2 * s + 1;
    return piece(1) * 8 + i;
  }
};

struct RopeRaw {
  uint32_t w[8];
};

template <int D, bool F16, int KIND>
__device__ __forceinline__ RopeRaw rope_load(const uint16_t* row, const RopeMap<D, KIND>& m) {
  RopeRaw r;
  if (KIND == kHalfOdd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = row[m.a(i)] | static_cast<uint32_t>(row[m.b(i)]) << 16;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(row + m.piece(0) * 8);
    const uint4 v = *reinterpret_cast<const uint4*>(row + m.piece(1) * 8);
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w, r.w[4] = v.x, r.w[5] = v.y, r.w[6] = v.z, r.w[7] = v.w;
  }
  return r;
}
// words of (channel, next channel) or, for halves on pieces, of (pair, next pair) -> pairs
template <int D, bool F16, int KIND>
__device__ __forceinline__ void rope_unpack(const RopeRaw& r, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = c4_unpack<F16>(r.w[i]);
    if (KIND == kHalf) {
      float* z = i < 4 ? a : b;
      z[(i & 3) * 2] = f.x, z[(i & 3) * 2 + 1] = f.y;
    } else {
      a[i] = f.x, b[i] = f.y;
    }
  }
}
template <int D, bool F16, int KIND>
__device__ __forceinline__ void rope_store(uint16_t* row, const RopeMap<D, KIND>& m, const float (&a)[8], const float (&b)[8]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float* z = i < 4 ? a : b;
    w[i] = KIND == kHalf ? c4_pack<F16>(z[(i & 3) * 2], z[(i & 3) * 2 + 1]) : c4_pack<F16>(a[i], b[i]);
  }
  if (KIND == kHalfOdd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) row[m.a(i)] = static_cast<uint16_t>(w[i]), row[m.b(i)] = static_cast<uint16_t>(w[i] >> 16);
  } else {
    *reinterpret_cast<uint4*>(row + m.piece(0) * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + m.piece(1) * 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The weights of a thread's channels, from global or shared memory.
template <int D, int KIND>
__device__ __forceinline__ void rope_weights(const float* w, const RopeMap<D, KIND>& m, float (&a)[8], float (&b)[8]) {
  if constexpr (KIND == kHalfOdd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = w[m.a(i)], b[i] = w[m.b(i)];
  } else {
    float v[16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(&v[4 * j]) = *reinterpret_cast<const float4*>(w + m.piece(j >> 1) * 8 + (j & 1) * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (KIND == kHalf) a[i] = v[i], b[i] = v[8 + i];
      else a[i] = v[2 * i], b[i] = v[2 * i + 1];
    }
  }
}

// (a, b) -> (a c - b s, b c + a s) for those of a thread's eight pairs that turn, two at a time; the others stay as they are.
// (Cosine 1 and sine 0 would not do: a 1 - b 0 is NaN beside an infinite b.) ALL: every pair turns.
template <int D, int KIND, bool ALL>
__device__ __forceinline__ void rope_turn_some(const RopeMap<D, KIND>& m, float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t x = f2(a[i], a[i + 1]), y = f2(b[i], b[i + 1]), co = f2(c[i], c[i + 1]);
    float p[2], q[2];
    f2_split(fma2(x, co, mul2(y, f2(-s[i], -s[i + 1]))), p[0], p[1]);
    f2_split(fma2(y, co, mul2(x, f2(s[i], s[i + 1]))), q[0], q[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)  // slots rise with i; of halves on pieces all eight turn or none
      if (ALL || m.slot(KIND == kHalf ? 7 : i + j) < m.rot >> 1) a[i + j] = p[j], b[i + j] = q[j];
  }
}
// With a branch around it where all turn or none: right for the forward (with selects alone 28.4 instead of 27.2 us in a
// graph for 8192 tokens of 32 and 8 heads of 128 channels), not for the gradient below (43.4 instead of 41.9).
template <int D, int KIND>
__device__ __forceinline__ void rope_turn(const RopeMap<D, KIND>& m, float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
  if (m.slot(7) < m.rot >> 1) rope_turn_some<D, KIND, true>(m, a, b, c, s);
  else if (KIND != kHalf) rope_turn_some<D, KIND, false>(m, a, b, c, s);
}
// sum over the thread's channels of x y
__device__ __forceinline__ float rope_dot(const float (&xa)[8], const float (&xb)[8], const float (&ya)[8], const float (&yb)[8]) {
  uint64_t t[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    t[0] = fma2(f2(xa[i], xa[i + 1]), f2(ya[i], ya[i + 1]), t[0]);
    t[1] = fma2(f2(xb[i], xb[i + 1]), f2(yb[i], yb[i + 1]), t[1]);
  }
  float lo, hi;
  f2_split(add2(t[0], t[1]), lo, hi);
  return lo + hi;
}

template <int D>
__device__ __forceinline__ float rope_row_sum(float x) {
#pragma unroll
  for (int o = D / 32; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// 2^-64ths of a turn per position of pairs i and i + 1, zero where they are not turned
template <int D, int KIND>
__device__ __forceinline__ void rope_turns(const RopeArgs& g, const RopeMap<D, KIND>& m, int i, uint64_t* f) {
  const int h = g.rot >> 1, k = m.slot(i);
  if (KIND == kHalf || (KIND == kInterleaved && k + 1 < h)) {  // two neighbours, both turned or neither
    const ulonglong2 u = k < h ? __ldg(reinterpret_cast<const ulonglong2*>(g.table + k)) : make_ulonglong2(0, 0);
    f[0] = u.x, f[1] = u.y;
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      f[j] = m.slot(i + j) < h ? __ldg(reinterpret_cast<const unsigned long long*>(g.table) + m.slot(i + j)) : 0;
  }
}
// cosine and sine of pairs i and i + 1, times factor (no matter which where a pair is not turned)
template <int D, int KIND>
__device__ __forceinline__ void rope_angles(const RopeArgs& g, const RopeMap<D, KIND>& m, int i, const uint64_t* f, int pos,
                                            float (&c)[8], float (&s)[8]) {
  const uint32_t p = static_cast<uint32_t>(pos), below = pos < 0 ? 0xffffffffu : 0u;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = static_cast<uint32_t>(f[j]), hi = static_cast<uint32_t>(f[j] >> 32);
    // bits 32..63 of the signed position times f
    const uint32_t z = p * hi + (below * lo + __umulhi(p, lo));
    const float t = static_cast<float>(static_cast<int32_t>(z)) * g.turn;
    c[i + j] = __cosf(t) * g.factor;
    s[i + j] = __sinf(t) * g.factor;
  }
}

// 16 bytes to shared memory, asynchronously; wait until at most `left` of this thread's groups are on their way
__device__ __forceinline__ void rope_fetch(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
template <int LEFT>
__device__ __forceinline__ void rope_fetched() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// One row: norm, turn, store.
template <int D, bool F16, int KIND, bool NORM>
__device__ __forceinline__ void rope_row(const RopeArgs& g, const RopeMap<D, KIND>& m, const RopeRaw& raw, const float (&wa)[8],
                                         const float (&wb)[8], const float (&c)[8], const float (&s)[8], uint16_t* to, bool live) {
  float a[8], b[8];
  rope_unpack<D, F16, KIND>(raw, a, b);
  if (NORM) {
    const float r = rsqrtf(fmaf(rope_row_sum<D>(rope_dot(a, b, a, b)), 1.f / D, g.eps));
    const uint64_t r2 = f2(r, r);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      f2_split(mul2(f2(a[i], a[i + 1]), mul2(f2(wa[i], wa[i + 1]), r2)), a[i], a[i + 1]);
      f2_split(mul2(f2(b[i], b[i + 1]), mul2(f2(wb[i], wb[i + 1]), r2)), b[i], b[i + 1]);
    }
  }
  rope_turn(m, a, b, c, s);
  if (live) rope_store<D, F16, KIND>(to, m, a, b);
}

// Forward, and the gradient without a norm (turn < 0). One unit is HP heads of one token. (Five CTAs per SM: with the six
// registers more that the compiler would take, 275,280 interleaved rows of 64 channels took 18.4 us instead of 17.1.)
template <int D, bool F16, int KIND, bool NORM, int HP>
__global__ void __launch_bounds__(kRopeThreads, HP > 1 ? 2 : NORM || KIND == kHalfOdd ? 1 : 5) rope_kernel(const __grid_constant__ RopeArgs g) {
  constexpr int T = D / 16;
  const int si = static_cast<int>(blockIdx.x) >= g.side[0].blocks;
  const RopeSide& sd = g.side[si];
  const int block = blockIdx.x - (si ? g.side[0].blocks : 0);
  // (units are fewer than 2^31: N Hq is)
  const uint32_t unit = static_cast<uint32_t>(block) * (kRopeThreads / T) + threadIdx.x / T;
  const int tok_ = static_cast<int>(unit / static_cast<uint32_t>(sd.slices)), h0 = static_cast<int>(unit - static_cast<uint32_t>(tok_) * sd.slices) * HP;
  const bool live = tok_ < rope_tokens(g);
  const int tok = min(tok_, g.N - 1);
  RopeMap<D, KIND> m;
  m.t = threadIdx.x % T, m.rot = g.rot;
  RopeRaw raw[HP];
#pragma unroll
  for (int u = 0; u < HP; ++u)
    raw[u] = rope_load<D, F16, KIND>(sd.x + tok * sd.xt + min(h0 + u, sd.H - 1) * sd.xh, m);
  float c[8], s[8], wa[8], wb[8];
  const int pos = __ldg(g.pos + tok);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint64_t f[2];
    rope_turns(g, m, i, f);
    rope_angles(g, m, i, f, pos, c, s);
  }
  if (NORM) rope_weights<D, KIND>(sd.w, m, wa, wb);
#pragma unroll
  for (int u = 0; u < HP; ++u)
    rope_row<D, F16, KIND, NORM>(g, m, raw[u], wa, wb, c, s, sd.y + tok * sd.yt + (h0 + u) * sd.yh, live && h0 + u < sd.H);
}

// The same for many units of four heads: a CTA takes every side.blocks-th, and while a thread works on one its pieces of the
// next are on their way to shared memory. It reads back what it fetched itself, so it waits for its own copies alone.
// 29.5 us for 8192 tokens of 32 and 8 heads of 128 channels with norms, 5.7 TB/s (34.9 with loads into registers, in units
// that come and go; 32.3 with three CTAs per SM; 30.4 with two units ahead). Single heads are better off without: 16.9 us for
// 275,280 rows of 64 channels, staged 19.8 and more.
constexpr int kFwdHeads = 4, kFwdStages = 2;
template <int D, bool F16, int KIND, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_staged_kernel(const __grid_constant__ RopeArgs g) {
  constexpr int T = D / 16, HP = kFwdHeads, STAGES = kFwdStages;
  extern __shared__ uint4 s_raw[];  // [stage][head][piece][thread]
  const int si = static_cast<int>(blockIdx.x) >= g.side[0].blocks;
  const RopeSide& sd = g.side[si];
  const int block = blockIdx.x - (si ? g.side[0].blocks : 0);
  RopeMap<D, KIND> m;
  m.t = threadIdx.x % T, m.rot = g.rot;
  const int tokens = rope_tokens(g);
  const uint32_t units = static_cast<uint32_t>(tokens) * sd.slices, step = static_cast<uint32_t>(sd.blocks) * (kRopeThreads / T);
  auto slot = [&](int stage, int u, int piece) { return s_raw + ((stage * HP + u) * 2 + piece) * kRopeThreads + threadIdx.x; };
  auto fetch = [&](uint32_t unit, int stage) {
    if (unit < units) {
      const int tok = static_cast<int>(unit / static_cast<uint32_t>(sd.slices)), h0 = static_cast<int>(unit - static_cast<uint32_t>(tok) * sd.slices) * HP;
#pragma unroll
      for (int u = 0; u < HP; ++u) {
        const uint16_t* const x = sd.x + tok * sd.xt + min(h0 + u, sd.H - 1) * sd.xh;
#pragma unroll
        for (int j = 0; j < 2; ++j) rope_fetch(slot(stage, u, j), x + m.piece(j) * 8);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float wa[8], wb[8];
  if (NORM) rope_weights<D, KIND>(sd.w, m, wa, wb);
  uint64_t f[8];  // (loaded once: 46.4 -> 43.8 us for the gradient below, 31.3 -> 29.5 for the forward)
#pragma unroll
  for (int i = 0; i < 8; i += 2) rope_turns(g, m, i, f + i);
  uint32_t unit = static_cast<uint32_t>(block) * (kRopeThreads / T) + threadIdx.x / T;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(unit + i * step, i);
  int stage = 0;
  // (whole warps stay together: rows are summed across their lanes)
  for (uint32_t first = unit - threadIdx.x % 32 / T; first < units; first += step, unit += step) {
    const int tok_ = static_cast<int>(unit / static_cast<uint32_t>(sd.slices)), h0 = static_cast<int>(unit - static_cast<uint32_t>(tok_) * sd.slices) * HP;
    const bool live = tok_ < tokens;
    const int tok = min(tok_, g.N - 1);
    fetch(unit + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    float c[8], s[8];
    const int pos = __ldg(g.pos + tok);
#pragma unroll
    for (int i = 0; i < 8; i += 2) rope_angles(g, m, i, f + i, pos, c, s);
    rope_fetched<STAGES - 1>();
#pragma unroll
    for (int u = 0; u < HP; ++u) {
      const uint4 x = *slot(stage, u, 0), y = *slot(stage, u, 1);
      rope_row<D, F16, KIND, NORM>(g, m, RopeRaw{{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}}, wa, wb, c, s,
                                   sd.y + tok * sd.yt + (h0 + u) * sd.yh, live && h0 + u < sd.H);
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
}

// Gradients with a norm. A CTA takes every side.blocks-th unit and keeps its sum of dw in registers, which it leaves in
// `part`: rows are summed in an order that the sizes alone decide. A thread's pieces of its next unit are on their way to
// shared memory while it works on one; it reads back what it fetched itself, so it waits for its own copies alone.
// Bounded by HBM and, near it, by latency: 43.9 us for 8192 tokens of 32 and 8 heads of 128 channels, 5.7 TB/s (with loads
// into registers, all that fit, 61; at 46.4, two units ahead cost 2 more, one head a thread and three CTAs per SM 10).
template <int D, bool F16, int KIND, int HP>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_bwd_kernel(const __grid_constant__ RopeArgs g) {
  constexpr int T = D / 16;
  constexpr bool kStaged = KIND != kHalfOdd;
  extern __shared__ uint4 s_raw[];  // [stage][head][x, dy][piece][thread]
  __shared__ float s_dw[kRopeThreads / 32][D];
  const int si = static_cast<int>(blockIdx.x) >= g.side[0].blocks;
  const RopeSide& sd = g.side[si];
  const int block = blockIdx.x - (si ? g.side[0].blocks : 0);
  RopeMap<D, KIND> m;
  m.t = threadIdx.x % T, m.rot = g.rot;
  __shared__ __align__(16) float s_w[D];  // (sixteen registers less)
  if (threadIdx.x < D) s_w[threadIdx.x] = __ldg(sd.w + threadIdx.x);
  __syncthreads();
  float da[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) da[i] = db[i] = 0.f;
  const int tokens = rope_tokens(g);
  const uint32_t units = static_cast<uint32_t>(tokens) * sd.slices;  // (fewer than 2^31: N Hq is)
  const uint32_t step = static_cast<uint32_t>(sd.blocks) * (kRopeThreads / T);
  auto where = [&](uint32_t first, int& tok, int& h0) {
    const uint32_t unit = first + threadIdx.x / T;
    tok = static_cast<int>(unit / static_cast<uint32_t>(sd.slices)), h0 = static_cast<int>(unit - static_cast<uint32_t>(tok) * sd.slices) * HP;
  };
  auto slot = [&](int stage, int u, int which, int piece) { return s_raw + (((stage * HP + u) * 2 + which) * 2 + piece) * kRopeThreads + threadIdx.x; };
  auto fetch = [&](uint32_t first, int stage) {
    if (first < units) {
      int tok, h0;
      where(first, tok, h0);
      tok = min(tok, g.N - 1);
#pragma unroll
      for (int u = 0; u < HP; ++u) {
        const int h = min(h0 + u, sd.H - 1);
        const uint16_t* const x = sd.x + tok * sd.xt + h * sd.xh;
        const uint16_t* const dy = sd.dy + tok * sd.dyt + h * sd.dyh;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          rope_fetch(slot(stage, u, 0, j), x + m.piece(j) * 8), rope_fetch(slot(stage, u, 1, j), dy + m.piece(j) * 8);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetched = [&](int stage, int u, int which) {
    const uint4 x = *slot(stage, u, which, 0), y = *slot(stage, u, which, 1);
    return RopeRaw{{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
  };
  uint64_t f[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) rope_turns(g, m, i, f + i);
  uint32_t first = static_cast<uint32_t>(block) * (kRopeThreads / T);
  if (kStaged) {
#pragma unroll
    for (int i = 0; i < kRopeStages - 1; ++i) fetch(first + i * step, i);
  }
  int stage = 0;
  for (; first < units; first += step) {
    int tok_, h0;
    where(first, tok_, h0);
    const bool live = tok_ < tokens;
    const int tok = min(tok_, g.N - 1);
    const int pos = __ldg(g.pos + tok);
    RopeRaw rx[HP], rd[HP];
    if (kStaged) {
      rope_fetched<kRopeStages - 2>();
#pragma unroll
      for (int u = 0; u < HP; ++u) rx[u] = fetched(stage, u, 0), rd[u] = fetched(stage, u, 1);
      fetch(first + (kRopeStages - 1) * step, stage == 0 ? kRopeStages - 1 : stage - 1);
      stage = stage == kRopeStages - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int u = 0; u < HP; ++u) {
        const int h = min(h0 + u, sd.H - 1);
        rx[u] = rope_load<D, F16, KIND>(sd.x + tok * sd.xt + h * sd.xh, m);
        rd[u] = rope_load<D, F16, KIND>(sd.dy + tok * sd.dyt + h * sd.dyh, m);
      }
    }
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) rope_angles(g, m, i, f + i, pos, c, s);
#pragma unroll
    for (int u = 0; u < HP; ++u) {
      float xa[8], xb[8], ga[8], gb[8], wa[8], wb[8];
      rope_weights<D, KIND>(s_w, m, wa, wb);
      rope_unpack<D, F16, KIND>(rx[u], xa, xb);
      rope_unpack<D, F16, KIND>(rd[u], ga, gb);
      rope_turn_some<D, KIND, false>(m, ga, gb, c, s);
      const float r = rsqrtf(fmaf(rope_row_sum<D>(rope_dot(xa, xb, xa, xb)), 1.f / D, g.eps));
      const uint64_t r2 = f2(r, r);
      const bool in = live && h0 + u < sd.H;
      // n = x r in place of x; dw += g n; then g w in place of g
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t na = mul2(f2(xa[i], xa[i + 1]), r2), nb = mul2(f2(xb[i], xb[i + 1]), r2);
        const uint64_t a2 = f2(ga[i], ga[i + 1]), b2 = f2(gb[i], gb[i + 1]);
        if (in) {
          f2_split(fma2(a2, na, f2(da[i], da[i + 1])), da[i], da[i + 1]);
          f2_split(fma2(b2, nb, f2(db[i], db[i + 1])), db[i], db[i + 1]);
        }
        f2_split(mul2(a2, f2(wa[i], wa[i + 1])), ga[i], ga[i + 1]);
        f2_split(mul2(b2, f2(wb[i], wb[i + 1])), gb[i], gb[i + 1]);
        f2_split(na, xa[i], xa[i + 1]);
        f2_split(nb, xb[i], xb[i + 1]);
      }
      const float k = rope_row_sum<D>(rope_dot(ga, gb, xa, xb)) * (-1.f / D);
      const uint64_t k2 = f2(k, k);
      if (in) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          f2_split(mul2(r2, fma2(f2(xa[i], xa[i + 1]), k2, f2(ga[i], ga[i + 1]))), ga[i], ga[i + 1]);
          f2_split(mul2(r2, fma2(f2(xb[i], xb[i + 1]), k2, f2(gb[i], gb[i + 1]))), gb[i], gb[i + 1]);
        }
        rope_store<D, F16, KIND>(sd.y + tok * sd.yt + (h0 + u) * sd.yh, m, ga, gb);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = T; o < 32; o <<= 1) {
      da[i] += __shfl_xor_sync(0xffffffffu, da[i], o);
      db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
    }
    if ((threadIdx.x & 31) < T) s_dw[threadIdx.x >> 5][m.a(i)] = da[i], s_dw[threadIdx.x >> 5][m.b(i)] = db[i];
  }
  __syncthreads();
  for (int ch = threadIdx.x; ch < D; ch += kRopeThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) v += s_dw[i][ch];
    g.part[static_cast<long long>(blockIdx.x) * D + ch] = v;
  }
  __syncthreads();
  grid_release();
}

// dw[ch] = sum of the CTAs' partial sums: CTA (x, side) takes 8 channels, 32 threads share a channel's column.
template <int D>
__global__ void __launch_bounds__(256) rope_dw_kernel(const __grid_constant__ RopeArgs g) {
  const RopeSide& sd = g.side[blockIdx.y];
  __shared__ float s_v[32][9];
  const int ch = blockIdx.x * 8 + threadIdx.x % 8, lane = threadIdx.x / 8;
  grid_wait();
  const float* part = g.part + static_cast<long long>(blockIdx.y ? g.side[0].blocks : 0) * D + ch;
  float v = 0.f;
  for (int i = lane; i < sd.blocks; i += 32) v += part[static_cast<long long>(i) * D];
  s_v[lane][threadIdx.x % 8] = v;
  __syncthreads();
  if (threadIdx.x < 8 && sd.H > 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s_v[i][threadIdx.x];
    sd.dw[ch] = v;
  }
}

// CTAs of a side of H heads, HP a thread: its part of `most`, which is what runs at once (no CTA may wait for another's
// end), and no more than there is work for.
int rope_ctas(const RopeArgs& g, int H, int HP, int D, int most) {
  if (H == 0) return 0;
  const long long n = (static_cast<long long>(g.N) * ((H + HP - 1) / HP) * (D / 16) + kRopeThreads - 1) / kRopeThreads;
  return static_cast<int>(min(n, max(1ll, static_cast<long long>(most) * H / (g.side[0].H + g.side[1].H))));
}
// Gradients with a norm: two CTAs per SM (launching four, two of which wait: 6 us more for the call above).
constexpr int kBwdHeads = 2;
int rope_most_ctas() { return 2 * num_sms(); }

template <typename Kernel>
cudaError_t rope_allow(Kernel kern, int smem, bool (&allowed)[64]) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !allowed[dev])) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) allowed[dev] = true;
  }
  return e;
}

template <int D, bool F16, int KIND, bool NORM, int HP>
cudaError_t rope_launch_direct(RopeArgs& g, cudaStream_t st) {
  for (RopeSide& s : g.side) {
    s.slices = (s.H + HP - 1) / HP;
    s.blocks = static_cast<int>((static_cast<long long>(g.N) * s.slices * (D / 16) + kRopeThreads - 1) / kRopeThreads);
  }
  rope_kernel<D, F16, KIND, NORM, HP><<<g.side[0].blocks + g.side[1].blocks, kRopeThreads, 0, st>>>(g);
  return cudaGetLastError();
}

template <int D, bool F16, int KIND, bool NORM>
cudaError_t rope_launch_staged(RopeArgs& g, cudaStream_t st) {
  constexpr int HP = kFwdHeads, smem = kFwdStages * HP * 2 * kRopeThreads * 16;
  static bool allowed[64] = {};
  const cudaError_t e = rope_allow(rope_staged_kernel<D, F16, KIND, NORM>, smem, allowed);
  if (e != cudaSuccess) return e;
  for (RopeSide& s : g.side) s.slices = (s.H + HP - 1) / HP, s.blocks = rope_ctas(g, s.H, HP, D, 2 * num_sms());
  rope_staged_kernel<D, F16, KIND, NORM><<<g.side[0].blocks + g.side[1].blocks, kRopeThreads, smem, st>>>(g);
  return cudaGetLastError();
}
template <int D, bool F16, int KIND>
cudaError_t rope_launch(RopeArgs& g, bool bwd, bool norm, cudaStream_t st) {
  constexpr int T = D / 16;
  if (bwd && norm) {
    for (RopeSide& s : g.side) s.slices = (s.H + kBwdHeads - 1) / kBwdHeads, s.blocks = rope_ctas(g, s.H, kBwdHeads, D, rope_most_ctas());
    constexpr int smem = KIND == kHalfOdd ? 0 : kRopeStages * kBwdHeads * 4 * kRopeThreads * 16;
    static bool allowed[64] = {};
    cudaError_t e = rope_allow(rope_bwd_kernel<D, F16, KIND, kBwdHeads>, smem, allowed);
    if (e != cudaSuccess) return e;
    rope_bwd_kernel<D, F16, KIND, kBwdHeads><<<g.side[0].blocks + g.side[1].blocks, kRopeThreads, smem, st>>>(g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_behind(rope_dw_kernel<D>, dim3(D / 8, g.side[1].H ? 2 : 1), 256, st, g);
  }
  // Four heads a thread once one head each fills the GPU twice over, and where there are as many; from shared memory where
  // rows are 16-byte pieces.
  const bool many = g.side[0].H > 2 && static_cast<long long>(g.N) * (g.side[0].H + g.side[1].H) * T > 2ll * 2048 * num_sms();
  if constexpr (KIND == kHalfOdd) {
    if (many) return norm ? rope_launch_direct<D, F16, KIND, true, kFwdHeads>(g, st) : rope_launch_direct<D, F16, KIND, false, kFwdHeads>(g, st);
  } else {
    if (many) return norm ? rope_launch_staged<D, F16, KIND, true>(g, st) : rope_launch_staged<D, F16, KIND, false>(g, st);
  }
  return norm ? rope_launch_direct<D, F16, KIND, true, 1>(g, st) : rope_launch_direct<D, F16, KIND, false, 1>(g, st);
}

template <int D>
cudaError_t rope_launch_d(RopeArgs& g, bool bwd, bool norm, bool f16, int interleaved, cudaStream_t st) {
  if (interleaved) return f16 ? rope_launch<D, true, kInterleaved>(g, bwd, norm, st) : rope_launch<D, false, kInterleaved>(g, bwd, norm, st);
  if (g.rot % 16) return f16 ? rope_launch<D, true, kHalfOdd>(g, bwd, norm, st) : rope_launch<D, false, kHalfOdd>(g, bwd, norm, st);
  return f16 ? rope_launch<D, true, kHalf>(g, bwd, norm, st) : rope_launch<D, false, kHalf>(g, bwd, norm, st);
}

scfa_status rope_rows(const void* p, long long token, long long head) {
  return !p || (reinterpret_cast<uintptr_t>(p) & 15u) || ((token | head) & 7) ? SCFA_ERR_INVALID : SCFA_OK;
}

// what both directions check
scfa_status rope_check(const void* pos, const void* table, int N, int Hq, int Hkv, int D, int rot, int interleaved, float factor,
                       float eps, int dtype) {
  if ((!pos && N > 0) || N < 0 || Hq < 1 || Hkv < 0 || rot < 0 || rot > D || (rot & 1) || (rot > 0 && !table)) return SCFA_ERR_INVALID;
  if (interleaved != 0 && interleaved != 1) return SCFA_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(table) & 15u) return SCFA_ERR_INVALID;
  if (!(factor > -INFINITY && factor < INFINITY) || !(eps >= 0.f && eps < INFINITY)) return SCFA_ERR_INVALID;
  if (D != 64 && D != 128) return SCFA_ERR_UNSUPPORTED;
  if (dtype != SCFA_DTYPE_BF16 && dtype != SCFA_DTYPE_F16) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * (static_cast<long long>(Hq) + Hkv) >= (1ll << 31) - 256) return SCFA_ERR_UNSUPPORTED;
  return SCFA_OK;
}

RopeArgs rope_args(const int32_t* pos, const int32_t* count, const uint64_t* table, int N, int rot, float factor, float eps, bool back) {
  RopeArgs g = {};
  g.pos = pos, g.count = count, g.table = table, g.N = N, g.rot = rot, g.factor = factor, g.eps = eps;
  g.turn = (back ? -1.f : 1.f) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  return g;
}

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" {

scfa_status scfa_rope_fwd(const uint16_t* q, long long q_token, long long q_head, const uint16_t* k, long long k_token,
                          long long k_head, const int32_t* pos, const int32_t* count, const uint64_t* table, int N, int Hq,
                          int Hkv, int D, int rot, int interleaved, float factor, const float* wq, const float* wk, float eps, int dtype,
                          uint16_t* q_out, long long qo_token, long long qo_head, uint16_t* k_out, long long ko_token,
                          long long ko_head, void* stream) {
  if (scfa_status e = rope_check(pos, table, N, Hq, Hkv, D, rot, interleaved, factor, eps, dtype)) return e;
  const bool norm = wq != nullptr;
  if (norm ? Hkv > 0 && !wk : wk != nullptr) return SCFA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(wq) | reinterpret_cast<uintptr_t>(wk)) & 15u) return SCFA_ERR_INVALID;
  if (N == 0) return SCFA_OK;
  if (rope_rows(q, q_token, q_head) || rope_rows(q_out, qo_token, qo_head) || c4_rows_overlap(qo_token, qo_head, N, Hq, D))
    return SCFA_ERR_INVALID;
  if (Hkv > 0 && (rope_rows(k, k_token, k_head) || rope_rows(k_out, ko_token, ko_head) || c4_rows_overlap(ko_token, ko_head, N, Hkv, D)))
    return SCFA_ERR_INVALID;
  RopeArgs g = rope_args(pos, count, table, N, rot, factor, eps, false);
  g.side[0] = {q, nullptr, q_out, q_token, q_head, 0, 0, qo_token, qo_head, wq, nullptr, Hq, 0, 0};
  g.side[1] = {k, nullptr, k_out, k_token, k_head, 0, 0, ko_token, ko_head, wk, nullptr, Hkv, 0, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = dtype == SCFA_DTYPE_F16;
  const cudaError_t e = D == 64 ? rope_launch_d<64>(g, false, norm, f16, interleaved, st)
                                : rope_launch_d<128>(g, false, norm, f16, interleaved, st);
  return e == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
}

size_t scfa_rope_workspace_size(int N, int Hq, int Hkv, int D) {
  if (N < 0 || Hq < 1 || Hkv < 0 || (D != 64 && D != 128)) return 0;
  return align_up(static_cast<size_t>(rope_most_ctas() + 2) * D * sizeof(float), 256);
}

scfa_status scfa_rope_bwd(const uint16_t* dq, long long dq_token, long long dq_head, const uint16_t* dk, long long dk_token,
                          long long dk_head, const uint16_t* q, long long q_token, long long q_head, const uint16_t* k,
                          long long k_token, long long k_head, const int32_t* pos, const int32_t* count,
                          const uint64_t* table, int N, int Hq, int Hkv, int D, int rot, int interleaved, float factor, const float* wq, const float* wk, float eps,
                          int dtype, uint16_t* dq_out, long long dqo_token, long long dqo_head, uint16_t* dk_out,
                          long long dko_token, long long dko_head, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                          void* stream) {
  if (scfa_status e = rope_check(pos, table, N, Hq, Hkv, D, rot, interleaved, factor, eps, dtype)) return e;
  const bool norm = wq != nullptr;
  if (norm ? !dwq || (Hkv > 0 && (!wk || !dwk)) : wk || dwq || dwk) return SCFA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(wq) | reinterpret_cast<uintptr_t>(wk)) & 15u) return SCFA_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    if (!norm) return SCFA_OK;
    cudaError_t e = cudaMemsetAsync(dwq, 0, D * sizeof(float), st);
    if (e == cudaSuccess && Hkv > 0) e = cudaMemsetAsync(dwk, 0, D * sizeof(float), st);
    return e == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
  }
  if (rope_rows(dq, dq_token, dq_head) || rope_rows(dq_out, dqo_token, dqo_head) || c4_rows_overlap(dqo_token, dqo_head, N, Hq, D))
    return SCFA_ERR_INVALID;
  if (Hkv > 0 && (rope_rows(dk, dk_token, dk_head) || rope_rows(dk_out, dko_token, dko_head) || c4_rows_overlap(dko_token, dko_head, N, Hkv, D)))
    return SCFA_ERR_INVALID;
  RopeArgs g = rope_args(pos, count, table, N, rot, factor, eps, true);
  if (norm) {
    if (rope_rows(q, q_token, q_head) || (Hkv > 0 && rope_rows(k, k_token, k_head))) return SCFA_ERR_INVALID;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < scfa_rope_workspace_size(N, Hq, Hkv, D)) return SCFA_ERR_WORKSPACE;
    g.side[0] = {q, dq, dq_out, q_token, q_head, dq_token, dq_head, dqo_token, dqo_head, wq, dwq, Hq, 0, 0};
    g.side[1] = {k, dk, dk_out, k_token, k_head, dk_token, dk_head, dko_token, dko_head, wk, dwk, Hkv, 0, 0};
    g.part = static_cast<float*>(ws);
  } else {
    g.side[0] = {dq, nullptr, dq_out, dq_token, dq_head, 0, 0, dqo_token, dqo_head, nullptr, nullptr, Hq, 0, 0};
    g.side[1] = {dk, nullptr, dk_out, dk_token, dk_head, 0, 0, dko_token, dko_head, nullptr, nullptr, Hkv, 0, 0};
  }
  const bool f16 = dtype == SCFA_DTYPE_F16;
  const cudaError_t e = D == 64 ? rope_launch_d<64>(g, true, norm, f16, interleaved, st)
                                : rope_launch_d<128>(g, true, norm, f16, interleaved, st);
  return e == cudaSuccess ? SCFA_OK : SCFA_ERR_CUDA;
}

}  // extern "C"
